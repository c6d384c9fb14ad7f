"""Rows of the few-token 4-bit layer that routings make in other ways than by
independent draws (against the 64-bit form and bounds of w4_oracle.py)."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_offsets_amd as m
import test_gpu_w4 as base
import w4_oracle as wo
from gpu_util import note

pytestmark = pytest.mark.gpu
_built = base._built

# name: T, k, E, H, I, shared I
SHAPES = {
    # every lane's list and weights come from other lanes' slots
    "twice-64": (16, 4, 3, 128, 64, 0),
    "twice-256": (64, 4, 3, 128, 64, 64),
    "twice-256-many-experts": (64, 4, 300, 64, 64, 0),
    "k16": (16, 16, 5, 128, 64, 0),
    "k3-straddles-waves": (85, 3, 4, 128, 64, 0),
    "one-token": (1, 16, 4, 128, 64, 0),
    "planned": (90, 4, 3, 128, 64, 0),
}


def matrices(rng, E, H, I, Is, f):
    lins, vals = [], []
    for groups, n, kk in [(E, I, H), (E, I, H), (E, H, I)] + ([(1, Is, H), (1, Is, H), (1, H, Is)]
                                                             if Is else []):
        codes, scales, zeros = wo.random_weights(rng, groups, n, kk, f[0], f[1], f[3])
        if f[0] == "mxfp4":
            scales = np.clip(scales.astype(int) // 8 + 127 - 20, 1, 254).astype(np.uint8)
        else:
            scales = np.ldexp(scales, -6).astype(np.float32)
        sc = torch.from_numpy(scales).cuda()
        if f[0] != "mxfp4":
            sc = sc.to(torch.float16 if f[2] == "f16" else torch.bfloat16)
            scales = sc.float().cpu().numpy()
        lins.append(m.W4Linear.pack(base.shape_of(groups, n, kk, f), torch.from_numpy(codes).cuda(), sc,
                                    None if zeros is None else torch.from_numpy(zeros).cuda()))
        vals.append(wo.values(codes, scales, zeros, f[0], f[1]))
    experts = [tuple((v[0][e], v[1][e]) for v in vals[:3]) for e in range(E)]
    shared = tuple((v[0][0], v[1][0]) for v in vals[3:]) if Is else None
    return lins, experts, shared


def check(name, shape, f, lins, experts, shared, idx, rng):
    T, k, H = shape.tokens, shape.top_k, shape.hidden
    wt = rng.random((T, k)).astype(np.float32)
    x = base.bf16(rng.standard_normal((T, H)))
    dec = m.W4Decoder(shape, m.W4Experts.of(*lins))
    args = dict(topk_idx=torch.from_numpy(idx).cuda(), topk_w=torch.from_numpy(wt).cuda())
    out = dec(x.cuda(), **args)
    want, tol = wo.layer(base.f64(x), idx, wt, experts, 0, f[0], f[1], shared)
    base.within(name, out, want, tol)
    for _ in range(5):
        assert torch.equal(out, dec(x.cuda(), **args))


@pytest.mark.parametrize("f", [base.FORMATS[0], base.FORMATS[4]], ids=[base.IDS[0], base.IDS[4]])
@pytest.mark.parametrize("name", list(SHAPES))
def test_tokens_that_name_an_expert_more_than_once(name, f):
    """Their weights add up in one row, wherever in the token the slots lie."""
    T, k, E, H, I, Is = SHAPES[name]
    rng = np.random.default_rng([T, k, E])
    note(f"w4 layer, repeated experts: {name} {f}")
    idx = rng.integers(0, E, (T, k))
    idx[:, -1] = idx[:, 0]                     # the first and the last slot
    idx[::3] = idx[::3, :1]                    # one expert for all
    idx[1::5, k // 2] = -1                     # a masked slot between
    lins, experts, shared = matrices(rng, E, H, I, Is, f)
    check(name, m.Shape(T, H, E, k, I, Is), f, lins, experts, shared, idx.astype(np.int32), rng)


# name: T, k, E, H, I, shared I: few routed rows an expert, all tokens the shared one
SHARED = {
    "in-the-workgroups": (32, 8, 128, 128, 64, 128),
    "planned": (64, 8, 256, 128, 64, 192),
    "staged-routed": (300, 4, 60, 64, 64, 64),
    "one-slot": (1000, 1, 256, 64, 64, 64),
}


@pytest.mark.parametrize("f", [base.FORMATS[0], base.FORMATS[4]], ids=[base.IDS[0], base.IDS[4]])
@pytest.mark.parametrize("name", list(SHARED))
def test_shared_expert_of_many_tokens_beside_many_experts(name, f):
    """The routed experts' average picks the kernels; the shared expert's rows,
    many times that average, go through the same ones."""
    T, k, E, H, I, Is = SHARED[name]
    rng = np.random.default_rng([T, k, E, Is])
    note(f"w4 layer, shared expert: {name} {f}")
    lins, experts, shared = matrices(rng, E, H, I, Is, f)
    idx = rng.integers(-1, E, (T, k)).astype(np.int32)
    check(name, m.Shape(T, H, E, k, I, Is), f, lins, experts, shared, idx, rng)
