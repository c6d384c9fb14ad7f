"""The few-token layer on 8-bit experts (moe_f8_decode_fwd) against its 64-bit form.

A step's 128 products are summed in fp32 by the matrix unit and the scale multiplies
that sum: every one of them is off by at most 2^-23 of the step's absolute sum, which
is the form that w4_oracle's bound of group-scaled weights has (its 62 times the
group's scale is the largest value there; here |w| stands for it)."""
import os

import numpy as np
import pytest
import torch

import f8_oracle as fo
import mixture_experts_layer_offsets_amd as m
import w4_oracle as wo
from gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mixture_experts_layer_offsets_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_layer_offsets_amd import build
        build.build(verbose=False)
    m.load()


def f64(t):
    return t.detach().cpu().double().numpy()


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)


# name: T, k, E (here), first, ids drawn from [lo, hi), H, I, shared I
LAYERS = {
    "one-token": (1, 8, 12, 0, 0, 12, 512, 256, 0),
    "one-slot": (1, 1, 1, 0, 0, 1, 64, 64, 0),
    "one-shared": (1, 4, 6, 0, 0, 6, 256, 128, 192),
    "one-elsewhere": (1, 2, 4, 100, 0, 50, 128, 64, 0),
    "one-elsewhere-shared": (1, 2, 4, 100, 0, 50, 128, 64, 64),
    # hidden rows too long to be staged together
    "one-token-wide": (1, 16, 16, 0, 0, 16, 128, 2176, 0),
    "few": (5, 4, 16, 0, 0, 16, 384, 128, 0),
    "share": (9, 6, 8, 16, 0, 40, 256, 192, 0),
    "all-elsewhere": (3, 2, 4, 100, 0, 50, 128, 64, 0),
    "heavy-expert": (40, 4, 2, 0, 0, 2, 256, 128, 0),
    "middle": (30, 4, 5, 0, 0, 5, 256, 128, 0),
    # contractions that end inside a tile, with few rows an expert and with many
    "tails": (6, 3, 5, 0, 0, 5, 192, 320, 64),
    "heavy-tails": (40, 4, 2, 0, 0, 2, 192, 320, 0),
    # more slots than a workgroup looks through: planned, at each average
    "planned": (100, 4, 64, 5, 0, 80, 128, 64, 64),
    "planned-more": (80, 4, 16, 0, 0, 16, 128, 192, 0),
    "planned-heavy": (90, 4, 4, 0, 0, 4, 128, 192, 0),
    "slots-256": (64, 4, 40, 0, 0, 44, 128, 64, 0),
    "slots-257": (257, 1, 40, 0, 0, 44, 128, 64, 0),
    "shared-heavy": (70, 2, 6, -3, -3, 6, 128, 64, 64),
    "k16-E1024": (6, 16, 1024, 0, 0, 1024, 64, 64, 0),
    "long": (3, 3, 5, 0, 0, 5, 7168, 2048, 0),
}


def layer_case(name, seed=0):
    T, k, E, first, lo, hi, H, I, Is = LAYERS[name]
    rng = np.random.default_rng([seed, sorted(LAYERS).index(name)])
    lins, vals = [], []
    for groups, n, kk in [(E, I, H), (E, I, H), (E, H, I)] + ([(1, Is, H), (1, Is, H), (1, H, Is)]
                                                             if Is else []):
        codes, scales, _ = fo.random_codes(rng, groups, n, kk)
        scales = (scales * np.float32(3 / np.sqrt(kk))).astype(np.float32)
        lins.append(m.F8Linear.pack(m.F8Shape(groups, n, kk), torch.from_numpy(codes).cuda(),
                                    torch.from_numpy(scales).cuda()))
        w = fo.weight_values(codes, scales)
        vals.append((w, np.abs(w) / 62))
    idx = rng.integers(lo, hi, (T, k)).astype(np.int32)
    wt = rng.random((T, k)).astype(np.float32)
    x = bf16(rng.standard_normal((T, H)))
    experts = [tuple((v[0][e], v[1][e]) for v in vals[:3]) for e in range(E)]
    shared = tuple((v[0][0], v[1][0]) for v in vals[3:]) if Is else None
    return m.Shape(T, H, E, k, I, Is), lins, x, idx, wt, experts, shared, first


@pytest.mark.parametrize("name", list(LAYERS))
def test_decode_layer(name):
    shape, lins, x, idx, wt, experts, shared, first = layer_case(name)
    note(f"f8 decode {name}")
    dec = m.F8Decoder(shape, m.F8Experts.of(*lins, first_expert=first))
    wn = wt.copy()
    wn[(idx < first) | (idx >= first + shape.experts)] = np.nan   # masked slots: unused weights
    args = dict(topk_idx=torch.from_numpy(idx).cuda(), topk_w=torch.from_numpy(wn).cuda())
    out = dec(x.cuda(), **args)
    want, tol = wo.layer(f64(x), idx, wt, experts, first, "int4", 128, shared)
    err = np.abs(f64(out) - want)
    assert np.all(err <= tol), (name, float((err / tol).max()))
    dec.ws.fill_(255)                                            # nothing is kept in the workspace
    assert torch.equal(out, dec(x.cuda(), **args))


def test_decode_with_a_router():
    """The router path is the layer's routing followed by the supplied path."""
    shape, lins, x, *_ = layer_case("few")
    rng = np.random.default_rng(3)
    wr = bf16(rng.standard_normal((shape.hidden, shape.experts)) * 0.1).cuda()
    bias = torch.from_numpy(rng.standard_normal(shape.experts).astype(np.float32)).cuda()
    dec = m.F8Decoder(shape, m.F8Experts.of(*lins))
    out = dec(x.cuda(), w_router=wr, bias=bias)
    logits = torch.empty((shape.tokens, shape.experts), device="cuda")
    ws = torch.empty(m.moe_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
    m.moe_router_logits(shape, x.cuda(), wr, bias, logits, ws)
    idx = torch.empty((shape.tokens, shape.top_k), dtype=torch.int32, device="cuda")
    w = torch.empty((shape.tokens, shape.top_k), device="cuda")
    m.moe_route(shape, logits, idx, w)
    assert torch.equal(out, dec(x.cuda(), topk_idx=idx, topk_w=w))


@pytest.mark.parametrize("name", ["one-token", "planned", "heavy-expert", "share"])
def test_each_way_of_the_layer_captured(name):
    """One token, planned, staged and few-row layers in a graph, replayed with new
    inputs, routings and a spoiled workspace between the replays."""
    shape, lins, x0, idx0, wt0, *_, first = layer_case(name, 7)
    experts = m.F8Experts.of(*lins, first_expert=first)
    dec, eager = m.F8Decoder(shape, experts), m.F8Decoder(shape, experts)
    x, idx, wt = x0.cuda(), torch.from_numpy(idx0).cuda(), torch.from_numpy(wt0).cuda()
    out = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dec(x, topk_idx=idx, topk_w=wt, out=out)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        dec(x, topk_idx=idx, topk_w=wt, out=out)
    _, _, _, _, lo, hi, *_ = LAYERS[name]
    for seed in range(4):
        rng = np.random.default_rng(seed)
        x.copy_(bf16(rng.standard_normal(x0.shape)))
        idx.copy_(torch.from_numpy(rng.integers(lo - 1, hi + 1, idx0.shape).astype(np.int32)))
        wt.copy_(torch.from_numpy(rng.random(wt0.shape).astype(np.float32)))
        dec.ws.fill_(seed)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager(x, topk_idx=idx, topk_w=wt))


def test_nan_weights_of_unused_experts():
    """Experts that no slot names are not read."""
    shape, lins, x, idx, wt, *_, first = layer_case("few")
    want = m.F8Decoder(shape, m.F8Experts.of(*lins))(
        x.cuda(), topk_idx=torch.from_numpy(idx % 3).cuda(), topk_w=torch.from_numpy(wt).cuda())
    for lin in lins:
        per = lin.shape.n // 16 * -(-lin.shape.k // 128) * 2048
        lin.packed[3 * per:shape.experts * per] = 0x7F
    got = m.F8Decoder(shape, m.F8Experts.of(*lins))(
        x.cuda(), topk_idx=torch.from_numpy(idx % 3).cuda(), topk_w=torch.from_numpy(wt).cuda())
    assert torch.equal(got, want)
