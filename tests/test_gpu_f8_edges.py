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


# Whole codes up to 15, and a 448 that gives every block the scale 1: a block's products are
# whole numbers below 2^13 and their sums below 2^17, which the matrix unit keeps.  What is
# left are the fp32 roundings of the scaled sums, without the bound's share of the unit.

def whole(rng, *shape):
    return rng.integers(-15, 16, shape).astype(np.float32)


def exact_within(name, got, blocks, scales, dtype):
    """blocks: sums of a block's products [..][block], scales the same shape."""
    terms = blocks * scales
    y, size = terms.sum(-1), np.abs(terms).sum(-1)
    within(name, got, y, fo.rounded(y, (blocks.shape[-1] + 24) * fo.ULP * size, dtype))


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("M,n,k", [(1, 40, 7168), (8, 300, 2000), (24, 5120, 390), (60, 15360, 390), (200, 256, 390),
                                   (300, 512, 7168), (600, 5120, 2560), (3000, 2304, 390)])
def test_whole_codes(M, n, k, dtype):
    rng = np.random.default_rng([M, n, k])
    x, w = whole(rng, M, k), whole(rng, n, k)
    x[:, ::128] = 448
    scales = np.exp(rng.uniform(-12, -10, (-(-n // 128), -(-k // 128)))).astype(np.float32)
    codes = torch.from_numpy(w).to(torch.float8_e4m3fn).view(torch.uint8)
    lin = m.F8Linear.pack(m.F8Shape(1, n, k, ROW[dtype]), codes[None].cuda(), torch.from_numpy(scales)[None].cuda())
    note(f"f8 whole codes rows={M} n={n} k={k} {dtype}")
    got = lin(torch.from_numpy(x).to(dtype).cuda())
    part = rng.permutation(M)[:32]
    sums = np.matmul(fo.blocks(x[part], 1).transpose(1, 0, 2).astype(np.float64),
                     fo.blocks(w, 1).transpose(1, 2, 0).astype(np.float64)).transpose(1, 2, 0)
    exact_within("y", got[torch.from_numpy(part).cuda()], sums,
                 np.repeat(scales.astype(np.float64), 128, 0)[:n][None], dtype)


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("M,n,k", [(300, 64, 64), (420, 2304, 520), (1000, 300, 272), (1000, 20000, 300), (9000, 130, 300)])
def test_whole_codes_of_a_weight_gradient(M, n, k, dtype):
    """Rows 0 and 1 of every block hold the 448s, where the other operand has zeros."""
    rng = np.random.default_rng([M, n, k, 1])
    x, dy = whole(rng, M, k), whole(rng, M, n)
    x[::128], dy[::128], x[1::128], dy[1::128] = 448, 0, 0, 448
    sx, sy = (2.0 ** -rng.integers(4, 8, c) for c in (k, n))  # a column's own scale
    lin = m.F8Linear(m.F8Shape(1, n, k, ROW[dtype]), torch.empty(0, dtype=torch.uint8, device="cuda"))
    note(f"f8 whole codes, weight gradient {M} rows n={n} k={k} {dtype}")
    got = lin.weight_gradient(*(torch.from_numpy((v * s).astype(np.float32)).to(dtype).cuda()
                                for v, s in ((x, sx), (dy, sy))))[0]
    cols = rng.permutation(n)[:128]
    xb, yb = (fo.blocks(v.T, 1).transpose(1, 0, 2).astype(np.float64) for v in (x, dy[:, cols]))
    sums = np.matmul(xb, yb.transpose(0, 2, 1)).transpose(1, 2, 0)
    exact_within("dw", got[:, torch.from_numpy(cols).cuda()], sums, (sx[:, None] * sy[cols])[..., None], dtype)
