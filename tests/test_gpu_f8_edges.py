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
