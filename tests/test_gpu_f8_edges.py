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
