"""Refusals and sizes of the 8-bit products' entry points (no GPU: every call returns
before it touches the device), and the checks of their classes."""
import contextlib
import ctypes
import dataclasses
import os
import re

import numpy as np
import pytest
import torch

import f8_oracle as fo
import mixture_experts_layer_offsets_amd as m
from mixture_experts_layer_offsets_amd import _lib

FAKE, OTHER = 1 << 40, 1 << 44
INVALID, UNSUPPORTED = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED
S = m.F8Shape(2, 48, 256)
LAYER = m.Shape(4, 256, 8, 2, 128)
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe.h")


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_layer_offsets_amd import build
        build.build(verbose=False)
    return _lib.load()


def every_call(lib, shape, p=FAKE):
    s = None if shape is None else ctypes.byref(shape.c())
    far = None if p is None else OTHER
    return [lib.moe_f8_pack(s, p, p, p, None), lib.moe_f8_quantize(s, p, 0, p, None),
            lib.moe_f8_unpack(s, p, p, None), lib.moe_f8_transpose(s, p, far, None),
            lib.moe_f8_quantize_rows(s, 3, p, 1 << 21, p, p, None),
            lib.moe_f8_linear(s, 3, p, 1 << 21, p, p, far, 1 << 21, p, 1 << 60, None),
            lib.moe_f8_linear_codes(s, 3, p, p, p, p, far, 1 << 21, None),
            lib.moe_f8_wgrad(s, 3, p, 1 << 21, p, 1 << 21, p, far, p, 1 << 60, None)]


@pytest.mark.parametrize("change,code", [
    (dict(groups=0), INVALID), (dict(n=0), INVALID), (dict(k=0), INVALID), (dict(row_type=3), INVALID),
    (dict(row_type=-1), INVALID), (dict(row_type=m.MOE_ROW_F32), UNSUPPORTED),
    (dict(groups=1025), UNSUPPORTED), (dict(n=(1 << 20) + 1), UNSUPPORTED), (dict(k=1 << 21), UNSUPPORTED)])
def test_shapes_outside_the_limits(lib, change, code):
    shape = dataclasses.replace(S, **change)
    assert set(every_call(lib, shape)) == {code}
    assert m.moe_f8_bytes(shape) == 0
    assert m.moe_f8_linear_workspace_bytes(shape, 5) == 0 and m.moe_f8_wgrad_workspace_bytes(shape, 5) == 0


def test_missing_pointers(lib):
    assert set(every_call(lib, None)) == {INVALID}
    assert set(every_call(lib, S, p=None)) == {INVALID}


def linear(lib, shape=S, rows=3, x=FAKE, xs=256, off=FAKE, packed=FAKE, out=OTHER, os_=48, ws=FAKE, n=1 << 60):
    return lib.moe_f8_linear(ctypes.byref(shape.c()), rows, x, xs, off, packed, out, os_, ws, n, None)


def wgrad(lib, shape=S, rows=3, x=FAKE, xs=256, dy=FAKE, ys=48, off=FAKE, dw=OTHER, ws=FAKE, n=1 << 60):
    return lib.moe_f8_wgrad(ctypes.byref(shape.c()), rows, x, xs, dy, ys, off, dw, ws, n, None)


def test_linear_refusals(lib):
    for kw in (dict(off=None), dict(xs=255), dict(os_=47), dict(rows=-1), dict(x=None), dict(out=None),
               dict(packed=None), dict(packed=FAKE + 8), dict(rows=30000, ws=None), dict(rows=30000, ws=FAKE + 8)):
        assert linear(lib, **kw) == INVALID, kw
    for kw in (dict(xs=(1 << 32) + 1), dict(os_=(1 << 32) + 1), dict(rows=(1 << 30) + 1),
               dict(shape=m.F8Shape(2, 1 << 20, 256), rows=1 << 26, os_=1 << 20)):
        assert linear(lib, **kw) == UNSUPPORTED, kw
    # the tiles' threads are less than 2^32: 2^23 tiles of 512
    for rows, rc in (((1 << 30) - 256, 0), (1 << 30, UNSUPPORTED)):
        assert linear(lib, shape=m.F8Shape(1, 256, 256), rows=rows, os_=256, out=1 << 50, n=0) == \
            (rc or _lib.MOE_ERR_WORKSPACE), rows
    need = m.moe_f8_linear_workspace_bytes(S, 30000)
    assert need >= 30000 * 256 + 30000 * 8 and linear(lib, rows=30000, n=need - 1) == _lib.MOE_ERR_WORKSPACE
    assert linear(lib, rows=0, x=None, out=None, ws=None, n=0) == _lib.MOE_OK
    assert m.moe_f8_linear_workspace_bytes(S, -1) == 0
    codes = lambda **k: lib.moe_f8_linear_codes(*{**dict(s=ctypes.byref(S.c()), rows=3, c=FAKE, sc=FAKE, off=FAKE,  # noqa: E731
                                                         p=FAKE, o=OTHER, os=48, st=None), **k}.values())
    for kw in (dict(c=None), dict(sc=None), dict(o=None), dict(p=None), dict(off=None), dict(os=47),
               dict(c=FAKE + 4), dict(rows=-1)):
        assert codes(**kw) == INVALID, kw
    assert codes(os=(1 << 32) + 1) == UNSUPPORTED and codes(rows=0, c=None, sc=None, o=None) == _lib.MOE_OK


def test_outputs_over_inputs(lib):
    """A value of out on one of x: refused.  Rows of one stride may interleave."""
    at = lambda values: FAKE + 2 * values  # noqa: E731
    for o in (0, 255, -47, 300 * 2 + 10, 300 - 47, -300 * 2):
        assert linear(lib, xs=300, os_=300, out=at(o)) == INVALID, o
    assert linear(lib, xs=256, os_=300, out=at(200)) == INVALID
    assert linear(lib, rows=1, out=at(255)) == INVALID and linear(lib, rows=1, out=at(-47)) == INVALID
    assert linear(lib, rows=2, xs=300, os_=301, out=at(256)) == INVALID
    # between the rows, and behind the last one: past the check (to the workspace's)
    big = dict(rows=30000, n=0)
    for o in (256, 304 - 48, 256 + 304 * 5, 29999 * 304 + 256, -48):
        assert linear(lib, xs=304, os_=304, out=at(o), **big) == _lib.MOE_ERR_WORKSPACE, o
    assert wgrad(lib, dw=at(2 * 256 + 255)) == INVALID and wgrad(lib, dw=at(-1)) == INVALID
    assert wgrad(lib, dy=OTHER, dw=OTHER) == INVALID
    assert wgrad(lib, dw=at(3 * 256), n=0) == _lib.MOE_ERR_WORKSPACE


def test_wgrad_refusals(lib):
    for kw in (dict(off=None), dict(xs=255), dict(ys=47), dict(rows=-1), dict(x=None), dict(dy=None), dict(dw=None),
               dict(ws=None), dict(ws=FAKE + 8)):
        assert wgrad(lib, **kw) == INVALID, kw
    for kw in (dict(xs=(1 << 32) + 1), dict(ys=(1 << 32) + 1), dict(rows=65534 * 128)):
        assert wgrad(lib, **kw) == UNSUPPORTED, kw
    for k, rc in (((1 << 20) - 128, _lib.MOE_ERR_WORKSPACE), (1 << 20, UNSUPPORTED)):
        assert wgrad(lib, shape=m.F8Shape(1024, 256, k), xs=k, ys=256, dw=1 << 50, n=0) == rc, k
    assert m.moe_f8_wgrad_workspace_bytes(S, 65534 * 128) == 0
    assert m.moe_f8_wgrad_workspace_bytes(S, 65533 * 128 + 127) > 0
    wide = m.F8Shape(1024, 1 << 20, 1 << 20)
    assert m.moe_f8_wgrad_workspace_bytes(wide, 5) == 0
    need = m.moe_f8_wgrad_workspace_bytes(S, 300)
    assert need >= (300 // 128 + 2) * 128 * (256 + 48) and wgrad(lib, rows=300, n=need - 1) == _lib.MOE_ERR_WORKSPACE


def test_other_refusals(lib):
    s = ctypes.byref(S.c())
    assert lib.moe_f8_quantize(s, FAKE, 3, FAKE, None) == INVALID
    assert lib.moe_f8_pack(s, FAKE, FAKE, FAKE + 8, None) == INVALID
    assert lib.moe_f8_transpose(s, FAKE, FAKE, None) == INVALID
    assert lib.moe_f8_quantize_rows(s, 3, FAKE, 255, FAKE, FAKE, None) == INVALID
    assert lib.moe_f8_quantize_rows(s, -1, FAKE, 256, FAKE, FAKE, None) == INVALID
    assert lib.moe_f8_quantize_rows(s, 3, FAKE, 256, FAKE + 4, FAKE, None) == INVALID
    assert lib.moe_f8_quantize_rows(s, 3, FAKE, (1 << 32) + 1, FAKE, FAKE, None) == UNSUPPORTED


def test_sizes():
    # 2 groups x 3 tiles x 2 steps of 2 KB, and a scale each
    assert m.moe_f8_bytes(S) == 12 * 2048 + 256
    assert m.moe_f8_bytes(m.F8Shape(1, 1, 1)) == 2048 + 256
    assert m.moe_f8_bytes(m.F8Shape(48, 2048, 7168)) == 48 * 128 * 56 * (2048 + 4)


def experts(first=0, routed=FAKE, shared=None):
    return _lib.MoeF8Experts(first, routed, routed, routed, shared, shared, shared)


def decode_rc(lib, shape, e, x=FAKE, wr=None, bias=None, idx=FAKE, w=FAKE, out=FAKE, ws=FAKE, n=1 << 40):
    return lib.moe_f8_decode_fwd(None if shape is None else ctypes.byref(shape.c()),
                                 None if e is None else ctypes.byref(e), x, wr, bias, idx, w, out, ws, n, None)


def test_decode_refusals(lib):
    e = experts()
    for kw in (dict(x=None), dict(out=None), dict(ws=None), dict(wr=FAKE), dict(idx=None), dict(w=None)):
        assert decode_rc(lib, LAYER, e, **kw) == INVALID, kw
    assert decode_rc(lib, None, e) == INVALID and decode_rc(lib, LAYER, None) == INVALID
    assert decode_rc(lib, LAYER, experts(routed=None)) == INVALID
    assert decode_rc(lib, LAYER, experts(shared=FAKE)) == INVALID
    assert decode_rc(lib, dataclasses.replace(LAYER, shared_inter=64), e) == INVALID
    assert decode_rc(lib, LAYER, experts(first=8), wr=FAKE, idx=None, w=None) == INVALID
    for change in (dict(dtype=m.MOE_MXFP8), dict(hidden=96), dict(inter=32), dict(tokens=2049), dict(top_k=17),
                   dict(experts=1025)):
        shape = dataclasses.replace(LAYER, **change)
        assert decode_rc(lib, shape, e) == UNSUPPORTED, change
        assert m.moe_f8_decode_workspace_bytes(shape) == 0
    need = m.moe_f8_decode_workspace_bytes(LAYER)
    assert need > 0 and decode_rc(lib, LAYER, e, n=need - 1) == _lib.MOE_ERR_WORKSPACE


def test_structs_match_header():
    text = open(HEADER).read()
    kinds = {"int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64}
    for name, ct in (("moe_f8_shape", _lib.MoeF8Shape), ("moe_f8_experts", _lib.MoeF8Experts),
                     ("moe_grad_tensor", _lib.MoeGradTensor)):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), text, re.S).group(1)
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
        fields = [re.findall(r"\w+|\*", d) for d in body.split(";")[:-1]]
        assert [(d[-1], ctypes.c_void_p if "*" in d else kinds[d[0]]) for d in fields] == ct._fields_


def test_classes_check_their_tensors():
    shape = m.F8Shape(2, 5, 64)
    codes, scales = torch.zeros((2, 5, 64), dtype=torch.uint8), torch.zeros((2, 1, 1))
    lin = m.F8Linear(shape, torch.empty(m.moe_f8_bytes(shape), dtype=torch.uint8))
    x, dy, off = (torch.zeros((3, 64), dtype=torch.bfloat16), torch.zeros((3, 5), dtype=torch.bfloat16),
                  torch.zeros(3, dtype=torch.int32))
    short = m.F8Linear(shape, lin.packed[:-1])
    bad = [lambda: m.F8Linear.pack(shape, codes[:, :4], scales),
           lambda: m.F8Linear.pack(shape, codes.int(), scales),
           lambda: m.F8Linear.pack(shape, codes, scales.half()),
           lambda: m.F8Linear.pack(shape, codes, torch.zeros((2, 5, 1))),
           lambda: m.F8Linear.pack(dataclasses.replace(shape, row_type=m.MOE_ROW_F32), codes, scales),
           lambda: m.F8Linear.quantize(torch.zeros((64, 5), dtype=torch.bfloat16)),
           lambda: m.F8Linear.quantize(torch.zeros((1, 64, 5), dtype=torch.float64)),
           lambda: m.F8Linear.quantize(torch.zeros((1, 5, 64), dtype=torch.bfloat16).transpose(1, 2)),
           lambda: lin(x), lambda: lin(x[0], off), lambda: lin(x[:, :32], off), lambda: lin(x.half(), off),
           lambda: lin(x, off.long()), lambda: lin(x, off[:2]), lambda: lin(x.t().contiguous().t(), off),
           lambda: lin(x, off, out=x), lambda: lin(x[:1].expand(3, 64), off),
           lambda: lin(torch.empty_like(x, device="meta"), off), lambda: lin(x, off, out=dy.half()),
           lambda: lin.weight_gradient(x, dy), lambda: lin.weight_gradient(x, dy[:2], off),
           lambda: lin.weight_gradient(dy, x, off), lambda: lin.weight_gradient(x, dy.float(), off),
           lambda: lin.weight_gradient(x, dy, off, out=torch.zeros((2, 64, 5))),
           lambda: lin.weight_gradient(x, dy, off, out=torch.zeros((2, 5, 64), dtype=torch.bfloat16)),
           lambda: short(x, off), short.values, short.transposed]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i}")


def test_calls_that_fit_are_taken(monkeypatch):
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    calls = []
    for name in ("moe_f8_linear", "moe_f8_unpack", "moe_f8_wgrad", "moe_f8_transpose"):
        monkeypatch.setattr(_lib, name, lambda *a, name=name: calls.append(name))
    shape = m.F8Shape(2, 5, 64, m.MOE_ROW_F16)
    lin = m.F8Linear(shape, torch.empty(m.moe_f8_bytes(shape), dtype=torch.uint8))
    x, dy, off = (torch.zeros((3, 64), dtype=torch.half), torch.zeros((3, 5), dtype=torch.half),
                  torch.zeros(3, dtype=torch.int32))
    assert lin(x, off).shape == (3, 5) and lin.values().shape == (2, 64, 5)
    assert lin.weight_gradient(x, dy, off).shape == (2, 64, 5)
    assert lin.transposed().shape == m.F8Shape(2, 64, 5, m.MOE_ROW_F16)
    assert calls == ["moe_f8_linear", "moe_f8_unpack", "moe_f8_wgrad", "moe_f8_transpose"]


def test_decoder_checks_its_experts():
    layer = m.Shape(4, 256, 8, 2, 128, 128)
    mats = {s: m.F8Linear(s, torch.zeros(m.moe_f8_bytes(s), dtype=torch.uint8)) for s in (
        m.F8Shape(8, 128, 256), m.F8Shape(8, 256, 128), m.F8Shape(4, 256, 256),
        m.F8Shape(1, 128, 256), m.F8Shape(1, 256, 128))}
    up, down, up4, up1, down1 = mats.values()
    dec = m.F8Decoder(layer, m.F8Experts.of(up, up, down, up1, up1, down1))
    m.F8Decoder(layer, m.F8Experts(*[i.packed for i in (up, up, down, up1, up1, down1)]))
    for wrong in ((down, up, down, up1, up1, down1), (up, up, up, up1, up1, down1), (up4, up4, down, up1, up1, down1),
                  (up, up, down, down1, up1, down1), (up, up, down, None, None, None)):
        with pytest.raises(ValueError, match="experts"):
            m.F8Decoder(layer, m.F8Experts.of(*wrong))
    with pytest.raises(ValueError, match="limits"):
        m.F8Decoder(dataclasses.replace(layer, hidden=100), m.F8Experts.of(up, up, down, up1, up1, down1))
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    idx, w = torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2))
    for call in (lambda: dec(x[:3], topk_idx=idx, topk_w=w), lambda: dec(x.float(), topk_idx=idx, topk_w=w),
                 lambda: dec(x, topk_idx=idx.long(), topk_w=w), lambda: dec(x, topk_idx=idx, topk_w=w, out=x[:2])):
        with pytest.raises(ValueError):
            call()


def test_plain_forms():
    """The tests' own plain forms on values worked by hand."""
    x = np.zeros((1, 130), np.float32)
    x[0, 0], x[0, 1], x[0, 2], x[0, 129] = 448, 17, -17, 0.5
    codes, s, v = fo.rows_quantised(x)
    # 17 lies between 16 and 18, a tie: the even code, 16
    assert s[0, 0] == 1 and v[0, 1] == 16 and v[0, 2] == -16
    assert abs(v[0, 129] - 0.5) <= 2.0 ** -24 and codes[0, 1, 1] == 0x7E
    assert fo.decode(np.array([0x7E, 0x01, 0x08, 0x80], np.uint8)).tolist() == [448, 2.0 ** -9, 2.0 ** -6, 0]
    zero = fo.rows_quantised(np.zeros((2, 5), np.float32))
    assert np.all(zero[1] == np.float32(2.0 ** -100)) and np.all(zero[2] == 0)
    w = fo.weight_values(np.full((1, 130, 3), 0x38, np.uint8), np.array([[[2.0], [3.0]]], np.float32))
    assert w[0, 127, 0] == 2 and w[0, 128, 2] == 3
    y, bound = fo.product(np.array([[1.0, 2.0]]), np.array([[3.0, -1.0]]))
    assert y[0, 0] == 1 and bound[0, 0] >= fo.CUT * 6
