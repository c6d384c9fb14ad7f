"""8-bit products where a tile, a buffer or a number's range ends, against plain 64-bit
forms and the bounds derived in f8_oracle.py."""
import os

import numpy as np
import pytest
import torch

import f8_oracle as fo
import mixture_experts_layer_offsets_amd as m
from gpu_util import note

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
ROW = {BF: m.MOE_ROW_BF16, FP: m.MOE_ROW_F16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mixture_experts_layer_offsets_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_layer_offsets_amd import build
        build.build(verbose=False)
    m.load()


def f64(t):
    return t.detach().cpu().double().numpy()


def rows(rng, M, k, dtype=BF):
    x = rng.standard_normal((M, k)) * np.exp(rng.standard_normal(k))
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


def within(name, got, want, tol):
    err = np.abs(f64(got) - want)
    assert np.all(err <= tol), (name, float((err - tol).max()), float((err / np.maximum(tol, 1e-300)).max()))


@pytest.mark.parametrize("groups,k", [(1, 272), (40, 520)], ids=["128", "256"])
@pytest.mark.parametrize("n", [257, 272, 400])
def test_weight_gradient_whose_last_columns_end_early(n, groups, k):
    """The last tile's second half has no scales of its own, in the last stage of a
    workspace of the smallest size; tiles of 128 and 256 rows of dw."""
    rng = np.random.default_rng([n, k])
    M = 1000
    shape = m.F8Shape(groups, n, k)
    x, dy = rows(rng, M, k), rows(rng, M, n)
    off = torch.tensor([0] * groups + [M], dtype=torch.int32, device="cuda")
    ws = torch.empty(m.moe_f8_wgrad_workspace_bytes(shape, M), dtype=torch.uint8, device="cuda")
    dw = torch.full((groups, k, n), 7.0, dtype=BF, device="cuda")
    note(f"f8 weight gradient groups={groups} k={k} n={n}")
    m.moe_f8_wgrad(shape, x.cuda(), dy.cuda(), off, dw, ws)
    want, bound = fo.weight_gradient(x.float().numpy(), dy.float().numpy())
    within("dw", dw[-1], want, fo.rounded(want, bound, BF))
    assert torch.all(dw[:-1] == 0)


# (rows, end of every group's rows, outputs, contraction): each kernel of the products, and
# the sizes on both sides of the choice between rows quantised on the way and before
SAME = [
    (1, None, 2048, 2048), (8, None, 2560, 7936), (8, None, 10240, 2560), (16, None, 2048, 4096),
    (16, None, 4096, 4096), (200, None, 256, 390), (33, None, 1280, 520), (1000, None, 256, 512),
    (4000, None, 256, 128), (5000, None, 16, 520), (500, [100, 100, 101, 499], 256, 130),
    (160, list(range(10, 161, 10)), 1000, 512), (300, [0, 7, 7, 290], 1001, 1000),
    (16000, list(range(160, 16001, 160)), 16, 200), (24, [0, 1, 23], 3584, 2560),
    (60, None, 15360, 390), (600, None, 10240, 390), (2000, [5, 70, 1999], 7168, 520)]


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("M,ends,n,k", SAME)
def test_codes_give_the_bits_of_their_rows(M, ends, n, k, dtype):
    """A product from rows, and from the same rows quantised before."""
    rng = np.random.default_rng([M, n, k])
    ends = [M] if ends is None else ends
    groups = len(ends)
    codes, scales, _ = fo.random_codes(rng, groups, n, k)
    shape = m.F8Shape(groups, n, k, ROW[dtype])
    lin = m.F8Linear.pack(shape, torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    x = rows(rng, M, k, dtype).cuda()
    off = torch.tensor([0] + ends, dtype=torch.int32, device="cuda")
    note(f"f8 codes rows={M} groups={groups} n={n} k={k} {dtype}")
    ks = -(-k // 128)
    xc = torch.empty((ks, M, 128), dtype=torch.uint8, device="cuda")
    xs = torch.empty((ks, M), device="cuda")
    m.moe_f8_quantize_rows(shape, x, xc, xs)
    a, b = (torch.zeros((M, n), dtype=dtype, device="cuda") for _ in range(2))
    lin(x, off, out=a)
    m.moe_f8_linear_codes(shape, xc, xs, off, lin.packed, b)
    assert torch.equal(a, b)


# Two blocks' scales meet as one fp32 product.  Below 2^-126 that is held in steps of 2^-149:
# off by 2^-150 times a sum of code products, at most 128 448^2 < 2^25 of them, each block.
SMALL = 2.0 ** -125


@pytest.mark.parametrize("sx,sw", [(-60, -63), (-97, -20), (-70, -70), (-75, -50), (-99, -99)])
@pytest.mark.parametrize("M", [3, 20, 300, 600])
def test_small_scales_on_both_sides(M, sx, sw):
    """Down to a scales' product of 2^-126 as precise as anywhere; below, to SMALL a block."""
    rng = np.random.default_rng([M, -sx, -sw])
    n, k = (10240, 390) if M == 600 else (200, 390)
    codes, _, _ = fo.random_codes(rng, 1, n, k)
    scales = np.full((1, -(-n // 128), 4), 2.0 ** sw, np.float32)
    lin = m.F8Linear.pack(m.F8Shape(1, n, k), torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    x = rng.standard_normal((M, k))
    x[:, ::128] = 448 / 2                         # scales between 2^(sx - 1) and 2^sx
    x = torch.from_numpy((x * 2.0 ** sx).astype(np.float32)).to(BF)
    note(f"f8 small scales rows={M} 2^{sx} 2^{sw}")
    part = slice(0, 200)
    w = fo.weight_values(codes[:, part], scales[:, :2])[0]
    y, bound = fo.product(fo.rows_quantised(x.float().numpy())[2], w)
    tol = fo.rounded(y, bound, BF) + (4 * SMALL if sx - 1 + sw < -126 else 0.0)
    within("y", lin(x.cuda())[:, part], y, tol)


@pytest.mark.parametrize("M", [200, 3000], ids=["one launch", "two"])
@pytest.mark.parametrize("sx,sy", [(-60, -63), (-70, -70), (-75, -50)])
def test_small_scales_of_a_weight_gradient(M, sx, sy):
    rng = np.random.default_rng([M, -sx, -sy])
    k, n = 40, 300
    x, dy = rng.standard_normal((M, k)), rng.standard_normal((M, n))
    x[::128], dy[::128] = 448 / 2, 448 / 2
    x, dy = (torch.from_numpy((v * 2.0 ** s).astype(np.float32)).to(BF) for v, s in ((x, sx), (dy, sy)))
    lin = m.F8Linear(m.F8Shape(1, n, k), torch.empty(0, dtype=torch.uint8, device="cuda"))
    want, bound = fo.weight_gradient(x.float().numpy(), dy.float().numpy())
    tol = fo.rounded(want, bound, BF) + (-(-M // 128) * SMALL if sx - 1 + sy - 1 < -126 else 0.0)
    within("dw", lin.weight_gradient(x.cuda(), dy.cuda())[0], want, tol)
