"""Refusals and sizes of the 4-bit weights' entry points (no GPU: every call
returns before it touches the device), and the checks of their classes."""
import ctypes
import dataclasses
import os
import re

import numpy as np
import pytest
import torch

import mixture_experts_layer_offsets_amd as m
import w4_oracle as wo
from mixture_experts_layer_offsets_amd import _lib

FAKE = 1 << 40
INVALID, UNSUPPORTED = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED
MX = m.W4Shape(2, 48, 256)
INT = m.W4Shape(2, 48, 256, m.MOE_W4_INT4, 64, m.MOE_SCALE_F16, 1)
LAYER = m.Shape(4, 256, 8, 2, 128)
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe.h")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_layer_offsets_amd import build
        build.build(verbose=False)
    return _lib.load()


def every_call(lib, shape, p=FAKE, zeros=None):
    s = None if shape is None else ctypes.byref(shape.c())
    return [lib.moe_w4_pack(s, p, p, zeros, p, None), lib.moe_w4_quantize(s, p, p, None),
            lib.moe_w4_unpack(s, p, p, None),
            lib.moe_w4_linear(s, 3, p, 1 << 21, p, p, p, 1 << 21, None)]


@pytest.mark.parametrize("base,change,code", [
    (MX, dict(groups=0), INVALID), (MX, dict(n=0), INVALID), (MX, dict(k=0), INVALID),
    (MX, dict(format=2), INVALID), (MX, dict(group_size=0), INVALID), (MX, dict(zeros=1), INVALID),
    (MX, dict(scale_type=2), INVALID), (MX, dict(group_size=64), UNSUPPORTED),
    (MX, dict(k=240), UNSUPPORTED), (MX, dict(groups=1025), UNSUPPORTED),
    (MX, dict(n=(1 << 20) + 1), UNSUPPORTED), (MX, dict(k=1 << 21), UNSUPPORTED),
    (MX, dict(groups=1024, n=1 << 20, k=1 << 15), UNSUPPORTED),
    (INT, dict(zeros=2), INVALID), (INT, dict(group_size=96), UNSUPPORTED),
    (INT, dict(k=224), UNSUPPORTED),
])
def test_shapes_outside_the_limits(lib, base, change, code):
    shape = dataclasses.replace(base, **change)
    assert set(every_call(lib, shape, zeros=FAKE if shape.zeros else None)) == {code}
    assert m.moe_w4_bytes(shape) == 0


def test_missing_pointers(lib):
    assert set(every_call(lib, None)) == {INVALID}
    assert set(every_call(lib, MX, p=None)) == {INVALID}
    s, i = ctypes.byref(MX.c()), ctypes.byref(INT.c())
    # zero points exactly where the shape has them
    assert lib.moe_w4_pack(s, FAKE, FAKE, FAKE, FAKE, None) == INVALID
    assert lib.moe_w4_pack(i, FAKE, FAKE, None, FAKE, None) == INVALID
    # several groups need offsets; strides shorter than a row; negative rows
    for args in ((3, FAKE, 256, None, FAKE, FAKE, 48), (3, FAKE, 255, FAKE, FAKE, FAKE, 48),
                 (3, FAKE, 256, FAKE, FAKE, FAKE, 47), (-1, FAKE, 256, FAKE, FAKE, FAKE, 48),
                 (3, None, 256, FAKE, FAKE, FAKE, 48), (3, FAKE, 256, FAKE, None, FAKE, 48),
                 (3, FAKE, 256, FAKE, FAKE, None, 48)):
        assert lib.moe_w4_linear(s, *args, None) == INVALID, args
    assert lib.moe_w4_linear(s, 3, FAKE, (1 << 32) + 1, FAKE, FAKE, FAKE, 48, None) == UNSUPPORTED
    # more rows than the kernels index; out over x
    assert lib.moe_w4_linear(s, (1 << 30) + 1, FAKE, 256, FAKE, FAKE, FAKE, 48, None) == UNSUPPORTED
    assert lib.moe_w4_linear(s, 3, FAKE, 256, FAKE, FAKE, FAKE, 48, None) == INVALID


def test_sizes(lib):
    # 2 groups x 3 output tiles x 2 steps of 1 KB, and 4 scale bytes per output and step
    assert m.moe_w4_bytes(MX) == 12 * 1024 + 12 * 64
    assert m.moe_w4_bytes(INT) == 12 * 1024 + 12 * 64 + 512
    # ragged n and k round up to whole tiles
    assert m.moe_w4_bytes(m.W4Shape(1, 1, 32)) == 1024 + 256
    big = m.W4Shape(48, 2048, 7168)
    assert m.moe_w4_bytes(big) == 48 * 2048 * 7168 * 17 // 32


def decode_rc(lib, shape, experts, x=FAKE, wr=None, bias=None, idx=FAKE, w=FAKE, out=FAKE, ws=FAKE,
              n=1 << 40):
    return lib.moe_w4_decode_fwd(None if shape is None else ctypes.byref(shape.c()),
                                 None if experts is None else ctypes.byref(experts), x, wr, bias,
                                 idx, w, out, ws, n, None)


def experts(fmt=m.MOE_W4_MXFP4, group=32, scale=0, zeros=0, first=0, routed=FAKE, shared=None):
    return _lib.MoeW4Experts(fmt, group, scale, zeros, first, routed, routed, routed, shared, shared,
                             shared)


def test_decode_refusals(lib):
    e = experts()
    for kw in (dict(x=None), dict(out=None), dict(ws=None), dict(wr=FAKE), dict(idx=None),
               dict(w=None), dict(idx=None, w=None)):
        assert decode_rc(lib, LAYER, e, **kw) == INVALID, kw
    assert decode_rc(lib, None, e) == INVALID and decode_rc(lib, LAYER, None) == INVALID
    assert decode_rc(lib, LAYER, experts(routed=None)) == INVALID
    # the shared expert's matrices exactly when the shape has one
    assert decode_rc(lib, LAYER, experts(shared=FAKE)) == INVALID
    assert decode_rc(lib, dataclasses.replace(LAYER, shared_inter=64), e) == INVALID
    # a router: over the experts here, at most E slots, whole 16-byte router rows
    r = dict(wr=FAKE, idx=None, w=None)
    assert decode_rc(lib, LAYER, experts(first=8), **r) == INVALID
    assert decode_rc(lib, dataclasses.replace(LAYER, top_k=9), e, **r) == INVALID
    assert decode_rc(lib, dataclasses.replace(LAYER, experts=12), e, **r) == UNSUPPORTED
    for change in (dict(dtype=m.MOE_MXFP8), dict(dtype=m.MOE_MXFP8_W4), dict(hidden=96),
                   dict(tokens=2049), dict(top_k=17), dict(experts=1025)):
        shape = dataclasses.replace(LAYER, **change)
        assert decode_rc(lib, shape, e) == UNSUPPORTED, change
        assert m.moe_w4_decode_workspace_bytes(shape) == 0
    for change in (dict(tokens=0), dict(dtype=9), dict(inter=0), dict(shared_inter=-64)):
        assert decode_rc(lib, dataclasses.replace(LAYER, **change), e) == INVALID
    # the format against H and I
    assert decode_rc(lib, dataclasses.replace(LAYER, inter=64),
                     experts(m.MOE_W4_INT4, 128)) == UNSUPPORTED
    assert decode_rc(lib, LAYER, experts(5)) == INVALID
    assert decode_rc(lib, LAYER, experts(m.MOE_W4_INT4, 48)) == UNSUPPORTED
    need = m.moe_w4_decode_workspace_bytes(LAYER)
    assert need > 0 and decode_rc(lib, LAYER, e, n=need - 1) == _lib.MOE_ERR_WORKSPACE


def test_structs_match_header(lib):
    text = open(HEADER).read()
    for name, ct in (("moe_w4_shape", _lib.MoeW4Shape), ("moe_w4_experts", _lib.MoeW4Experts)):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), text, re.S).group(1)
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
        fields = [re.findall(r"\w+|\*", d) for d in body.split(";")[:-1]]
        want = [(d[-1], ctypes.c_void_p if "*" in d else ctypes.c_int32) for d in fields]
        assert want == ct._fields_


def test_classes_check_their_tensors():
    shape = m.W4Shape(2, 5, 64, m.MOE_W4_INT4, 32, m.MOE_SCALE_BF16, 1)
    codes = torch.zeros((2, 5, 32), dtype=torch.uint8)
    scales = torch.zeros((2, 5, 2), dtype=torch.bfloat16)
    z = torch.zeros((2, 5, 2), dtype=torch.uint8)
    lin = m.W4Linear(shape, torch.empty(m.moe_w4_bytes(shape), dtype=torch.uint8))
    x, off = torch.zeros((3, 64), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    bad = [lambda: m.W4Linear.pack(shape, codes[:, :4], scales, z),
           lambda: m.W4Linear.pack(shape, codes.int(), scales, z),
           lambda: m.W4Linear.pack(shape, codes, scales.float(), z),
           lambda: m.W4Linear.pack(shape, codes, scales, None),
           lambda: m.W4Linear.pack(shape, codes, scales, z[:, :, :1]),
           lambda: m.W4Linear.pack(shape, codes, scales.transpose(0, 1).contiguous().transpose(0, 1), z),
           lambda: m.W4Linear.pack(dataclasses.replace(shape, k=60), codes, scales, z),
           lambda: m.W4Linear.quantize(torch.zeros((64, 5), dtype=torch.bfloat16)),
           lambda: m.W4Linear.quantize(torch.zeros((1, 64, 5))),
           lambda: m.W4Linear.quantize(torch.zeros((1, 33, 5), dtype=torch.bfloat16)),
           lambda: lin(x), lambda: lin(x[0], off), lambda: lin(x[:, :32], off),
           lambda: lin(x.float(), off), lambda: lin(x, off.long()), lambda: lin(x, off[:2]),
           lambda: lin(x.t().contiguous().t(), off), lambda: lin(x, off, out=x),
           lambda: lin(torch.zeros((1, 64), dtype=torch.bfloat16).expand(3, 64), off),
           lambda: lin(torch.empty_like(x, device="meta"), off)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i}")


def test_decoder_checks_its_experts():
    layer = m.Shape(4, 256, 8, 2, 128)
    up, down = m.W4Shape(8, 128, 256), m.W4Shape(8, 256, 128)
    buf = {s: torch.empty(m.moe_w4_bytes(s), dtype=torch.uint8) for s in (up, down)}
    lin = {s: m.W4Linear(s, buf[s]) for s in buf}
    e = m.W4Experts.of(lin[up], lin[up], lin[down])
    dec = m.W4Decoder(layer, e)
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    idx, w = torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2))
    other = m.W4Linear(dataclasses.replace(down, format=m.MOE_W4_INT4), buf[down])
    bad = [lambda: m.W4Experts.of(lin[up], lin[up], other),
           lambda: m.W4Decoder(dataclasses.replace(layer, hidden=512), e),
           lambda: m.W4Decoder(dataclasses.replace(layer, tokens=0), e),
           lambda: m.W4Decoder(dataclasses.replace(layer, shared_inter=64), e),
           lambda: m.W4Decoder(layer, m.W4Experts(buf[up], buf[up], buf[down], buf[up], buf[up], buf[down])),
           lambda: dec(x[:3], topk_idx=idx, topk_w=w), lambda: dec(x.float(), topk_idx=idx, topk_w=w),
           lambda: dec(x, topk_idx=idx.long(), topk_w=w), lambda: dec(x, topk_idx=idx, topk_w=w[:, :1]),
           lambda: dec(x, w_router=torch.zeros((256, 4), dtype=torch.bfloat16)),
           lambda: dec(x, topk_idx=idx, topk_w=w, out=x[:2])]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i}")


def test_plain_forms():
    """The tests' own plain forms on values worked by hand."""
    codes = np.array([[[0x10, 0x32, 0xF8] + [0] * 13]], np.uint8)      # 0 1 2 3 8 15 0 ..
    v, s = wo.values(codes, np.array([[[128]]], np.uint8), None, "mxfp4", 32)
    assert v[0, 0, :6].tolist() == [0, 1, 2, 3, 0, -12] and s[0, 0, 0] == 2
    v, s = wo.values(codes, np.array([[[0.5]]], np.float32), np.array([[[3]]], np.uint8), "int4", 32)
    assert v[0, 0, :6].tolist() == [-1.5, -1, -.5, 0, 2.5, 6]
    v, _ = wo.values(codes, np.array([[[-2.0]]], np.float32), None, "int4", 32)
    assert v[0, 0, :6].tolist() == [16, 14, 12, 10, 0, -14]
