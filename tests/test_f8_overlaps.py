"""8-bit entry points whose output lies on what it is computed from, or whose weights lie
askew, refuse (no GPU: the refusals come first, and nothing else is called)."""
import ctypes
import os

import pytest

import mixture_experts_layer_offsets_amd as m
from mixture_experts_layer_offsets_amd import _lib

A = 1 << 40
INVALID = _lib.MOE_ERR_INVALID_ARG
S = m.F8Shape(2, 48, 256)       # packed: 12 tiles of 2 KB and 256 bytes of scales
PACKED = 12 * 2048 + 256
TURNED = 2 * 16 * 2048 + 256    # [256 / 16][1] tiles of a group
N = 2 * 48 * 256


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_layer_offsets_amd import build
        build.build(verbose=False)
    return _lib.load()


def test_sizes(lib):
    assert m.moe_f8_bytes(S) == PACKED and m.moe_f8_bytes(m.F8Shape(2, 256, 48)) == TURNED


def edges(out_bytes, in_bytes):
    """Places of an output beside an input at A: the first and last that meet it, and some
    between (16-byte steps)."""
    return [A, A + (in_bytes - 1) // 16 * 16, A - (out_bytes - 1) // 16 * 16, A + in_bytes // 2 // 16 * 16]


def test_weights(lib):
    s, far = ctypes.byref(S.c()), 1 << 44
    for at in edges(PACKED, N):
        assert lib.moe_f8_pack(s, A, far, at, None) == INVALID, hex(at)
    for at in edges(PACKED, 2 * 1 * 2 * 4):
        assert lib.moe_f8_pack(s, far, A, at, None) == INVALID, hex(at)
    for kind, size in ((m.MOE_ROW_BF16, 2), (m.MOE_ROW_F32, 4)):
        for at in edges(PACKED, N * size):
            assert lib.moe_f8_quantize(s, A, kind, at, None) == INVALID, hex(at)
    for at in edges(N * 4, PACKED):
        assert lib.moe_f8_unpack(s, A, at, None) == INVALID, hex(at)
    for at in edges(TURNED, PACKED):
        assert lib.moe_f8_transpose(s, A, at, None) == INVALID, hex(at)


def test_rows(lib):
    s, far = ctypes.byref(S.c()), 1 << 44
    rows, stride = 7, 300
    x, codes, scales = 2 * (6 * stride + 256), 2 * rows * 128, 2 * rows * 4
    for at in edges(codes, x):
        assert lib.moe_f8_quantize_rows(s, rows, A, stride, at, far, None) == INVALID, hex(at)
    for at in edges(scales, x):
        assert lib.moe_f8_quantize_rows(s, rows, A, stride, far, at, None) == INVALID, hex(at)
    for at in edges(codes, scales):
        assert lib.moe_f8_quantize_rows(s, rows, far, stride, at, A, None) == INVALID, hex(at)
    out = 2 * (6 * stride + 48)
    for at in edges(out, codes):
        assert lib.moe_f8_linear_codes(s, rows, A, far, far, far, at, stride, None) == INVALID, hex(at)
    for at in edges(out, scales):
        assert lib.moe_f8_linear_codes(s, rows, far, A, far, far, at, stride, None) == INVALID, hex(at)
    # without rows there is nothing to meet
    assert lib.moe_f8_linear_codes(s, 0, A, far, far, far, A, stride, None) == _lib.MOE_OK


@pytest.mark.parametrize("which", ["gate", "up", "down", "shared_gate", "shared_up", "shared_down"])
def test_experts_are_aligned(lib, which):
    """Packed matrices lie on 16 bytes, as every other entry point asks of them."""
    layer = m.Shape(4, 256, 8, 2, 128, 128)
    for off, rc in ((0, _lib.MOE_ERR_WORKSPACE), (8, INVALID), (1, INVALID)):
        e = _lib.MoeF8Experts(0, *[A] * 6)
        setattr(e, which, A + off)
        assert lib.moe_f8_decode_fwd(ctypes.byref(layer.c()), ctypes.byref(e), A, None, None, A, A, A, A, 0,
                                     None) == rc, off
