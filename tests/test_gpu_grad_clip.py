"""Global gradient norm and clipping (moe_grad_*) against 64-bit sums.

The norm: squares and sums in 64 bits, so that its one rounding to fp32 remains (half
a step, 2^-24, and as much again for the 64-bit sums and root).  Outputs: the
coefficient is off by 2^-24 and as much again, the product rounded once to the type."""
import math
import os

import numpy as np
import pytest
import torch

import mixture_experts_layer_offsets_amd as m
from gpu_util import note

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
LEAST = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
NORMS = [m.MOE_NORM_2, m.MOE_NORM_INF]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mixture_experts_layer_offsets_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_layer_offsets_amd import build
        build.build(verbose=False)
    m.load()


def f64(t):
    return t.detach().cpu().double().numpy()


def norm_of(values, norm_type):
    if norm_type == m.MOE_NORM_INF:
        return max((float(np.abs(v).max()) for v in values if v.size), default=0.0)
    return math.sqrt(math.fsum(float((v ** 2).sum()) for v in values))


def tensors(rng, sizes, dtypes, scale=1.0):
    """Tensors of one buffer each, at odd places in it."""
    out = []
    for i, n in enumerate(sizes):
        t = torch.from_numpy((rng.standard_normal(n + 3) * scale).astype(np.float32)).to(dtypes[i % len(dtypes)])
        out.append(t.cuda()[i % 3:i % 3 + n])
    return out


def check(grads, outs, before, norm, norm_type, max_norm):
    true = norm_of(before, norm_type)
    assert abs(float(norm) - true) <= true * 2.0 ** -23 + 2.0 ** -149
    coef = min(1.0, max_norm / (true + 1e-6))
    for x, o, b in zip(grads, outs, before):
        tol = np.abs(b) * coef * (HALF[x.dtype] + 2.0 ** -23) + LEAST[x.dtype]
        err = np.abs(f64(o) - b * coef)
        assert np.all(err <= tol), float((err / tol).max())


F32, BF, FP = torch.float32, torch.bfloat16, torch.float16
SETS = {
    "one-value": ([1], [F32]),
    "small": ([5, 64, 1, 1000], [F32, BF, FP]),
    "ragged": ([1, 7, 8, 9, 16383, 16384, 16385, 32768, 32769, 100003], [F32, BF, FP]),
    "empty-ones": ([0, 10, 0, 0, 33, 0], [BF, F32]),
    "a-launch": ([100 + i for i in range(128)], [F32, BF]),
    "more-than-a-launch": ([37 * i % 5000 for i in range(300)], [FP, F32, BF]),
    "many": ([i % 40 for i in range(3000)], [F32, BF]),
    "large": ([9000001, 1, 4000000], [F32, BF]),
}


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("norm_type", NORMS)
@pytest.mark.parametrize("name", list(SETS))
def test_clip(name, norm_type, in_place):
    sizes, dtypes = SETS[name]
    rng = np.random.default_rng(len(sizes))
    for max_norm in (0.5, 1e9):
        grads = tensors(rng, sizes, dtypes)
        before = [f64(t) for t in grads]
        outs = grads if in_place else [torch.full_like(t, 7.0) for t in grads]
        note(f"clip {name} norm {norm_type} max {max_norm} in place {in_place}")
        clip = m.GradClip(m.GradSet(grads, None if in_place else outs), norm_type)
        norm = clip(max_norm)
        check(grads, outs, before, norm, norm_type, max_norm)
        if not in_place:
            assert all(np.array_equal(f64(t), b) for t, b in zip(grads, before))
        if max_norm == 1e9:
            assert all(np.array_equal(f64(o), b) for o, b in zip(outs, before))


@pytest.mark.parametrize("sizes", [
    [1000] * 16, [1000] * 17, [16384] * 3, [16384, 16384, 16384, 1], [16383, 16385, 16384], [0] * 20 + [3] * 16],
    ids=["16", "17", "48-chunks", "49-chunks", "49-by-one", "16-and-empty"])
@pytest.mark.parametrize("norm_type", NORMS)
def test_where_one_workgroup_ends(norm_type, sizes):
    """Sets on both sides of what one workgroup takes."""
    rng = np.random.default_rng(len(sizes))
    for dtype in (F32, BF):
        grads = tensors(rng, [n if dtype == F32 else 2 * n for n in sizes], [dtype])
        before = [f64(t) for t in grads]
        note(f"clip {len(sizes)} tensors norm {norm_type} {dtype}")
        norm = m.GradClip(m.GradSet(grads), norm_type)(0.5)
        check(grads, grads, before, norm, norm_type, 0.5)


def test_past_the_partial_sums():
    """So many launches that their partial sums are added up before the scaling."""
    n = 128 * 40
    flat = torch.randn(n * 20000 // 10, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    grads = list(flat.view(n, -1))
    before = flat.double()
    note(f"clip {n} tensors of {grads[0].numel()}")
    for big in (False, True):
        if big:   # every launch as many workgroups as it may have: 128 tensors of 4 chunks and more
            flat = torch.randn(n * 40000, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
            grads, before = list(flat.view(n, -1)), flat.double()
        norm = m.GradClip(m.GradSet(grads))(1.0)
        true = float(before.square().sum().sqrt())
        assert abs(float(norm) - true) <= true * 2.0 ** -22
        assert torch.all((flat.double() - before / (true + 1e-6)).abs() <= before.abs() / true * 2.0 ** -22 + 2.0 ** -149)


def test_two_halves_are_the_whole():
    """Two ranks' parts: totals added, each part scaled by the sum."""
    rng = np.random.default_rng(4)
    for norm_type in NORMS:
        parts = [tensors(rng, [100, 5000], [F32, BF]) for _ in range(2)]
        before = [f64(t) for p in parts for t in p]
        clips = [m.GradClip(m.GradSet(p), norm_type) for p in parts]
        totals = [c.total() for c in clips]
        both = totals[0] + totals[1] if norm_type == m.MOE_NORM_2 else torch.maximum(*totals)
        norms = [c.scale(both, 0.25) for c in clips]
        for n in norms:
            check([t for p in parts for t in p], [t for p in parts for t in p], before, n, norm_type, 0.25)


def test_extremes():
    """Squares that fp32 does not hold; values that are not finite; none at all."""
    big = torch.full((1000,), 1e30, device="cuda")
    small = torch.full((1000,), 1e-30, device="cuda")
    for t, v in ((big, 1e30), (small, 1e-30)):
        t0 = t.clone()
        norm = m.GradClip(m.GradSet([t]))(1.0)
        true = float(t0.double().square().sum().sqrt())
        assert abs(float(norm) - true) <= true * 2.0 ** -23
        coef = min(1.0, 1 / (true + 1e-6))
        assert torch.all((t.double() - t0.double() * coef).abs() <= t0.double() * coef * 2.0 ** -22 + 2.0 ** -149)
    for norm_type in NORMS:
        t = torch.tensor([1.0, float("inf"), -2.0], device="cuda")
        norm = m.GradClip(m.GradSet([t]), norm_type)(1.0)
        assert float(norm) == math.inf and torch.equal(torch.isnan(t).cpu(), torch.tensor([False, True, False]))
        assert float(t[0]) == 0 and float(t[2]) == 0
        t = torch.tensor([1.0, float("nan"), float("-inf")], device="cuda")
        norm = m.GradClip(m.GradSet([t]), norm_type)(1.0)
        assert math.isnan(float(norm)) and torch.all(torch.isnan(t))
        t = torch.zeros(40, device="cuda")
        norm = m.GradClip(m.GradSet([t]), norm_type)(0.0)
        assert float(norm) == 0 and torch.all(t == 0)
        t = torch.empty(0, device="cuda")
        norm = m.GradClip(m.GradSet([t]), norm_type)(1.0)
        assert float(norm) == 0
        total = m.GradClip(m.GradSet([t]), norm_type).total()
        assert float(total) == 0
    t = torch.ones(100, device="cuda")
    m.GradClip(m.GradSet([t]))(math.inf)
    assert torch.all(t == 1)
    m.GradClip(m.GradSet([t]))(0.0)
    assert torch.all(t == 0)


def test_views_and_an_out_of_its_own():
    """Dense tensors in any order of their axes; the others are refused."""
    t = torch.randn(40, 30, 7, generator=torch.Generator().manual_seed(2)).cuda().permute(2, 0, 1)
    before = f64(t)
    norm = m.GradClip(m.GradSet([t]))(0.5)
    check([t], [t], [before], norm, m.MOE_NORM_2, 0.5)
    with pytest.raises(ValueError, match="dense"):
        m.GradSet([t[:, ::2]])
    with pytest.raises(ValueError, match="overlap"):
        m.GradSet([t, t])
    flat = torch.zeros(100, device="cuda")
    with pytest.raises(ValueError, match="overlap"):
        m.GradSet([flat[:50]], [flat[10:60]])
    with pytest.raises(ValueError, match="overlap"):
        m.GradSet([flat[:20], flat[50:70]], [flat[20:40], flat[60:80]])


def test_captured_replayed_and_repeated():
    """Captured on a side stream and replayed with new gradients; every replay and
    every eager call gives the same bits."""
    rng = np.random.default_rng(5)
    sizes = [100000, 3, 4097] * 60
    grads = tensors(rng, sizes, [F32, BF])
    outs = [torch.empty_like(t) for t in grads]
    want = [torch.empty_like(t) for t in grads]
    captured, eager = m.GradClip(m.GradSet(grads, outs)), m.GradClip(m.GradSet(grads, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        captured(1.0)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured(1.0)
    for seed in range(4):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for t in grads:
            t.copy_(torch.randn(t.shape, generator=gen, device="cuda") * 10 ** (seed - 2))
        captured.ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        norm = eager(1.0)
        torch.cuda.synchronize()
        assert torch.equal(norm, captured.norm)
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_clips_at_once_on_three_streams():
    rng = np.random.default_rng(6)
    sets = [tensors(rng, [200000 + i, 50, 3333], [F32, FP]) for i in range(3)]
    outs = [[torch.empty_like(t) for t in s] for s in sets]
    clips = [m.GradClip(m.GradSet(s, o)) for s, o in zip(sets, outs)]
    for c in clips:
        c(1.0)
    torch.cuda.synchronize()
    want = [(c.norm.clone(), [t.clone() for t in o]) for c, o in zip(clips, outs)]
    streams = [torch.cuda.Stream() for _ in clips]
    for _ in range(10):
        for s, c in zip(streams, clips):
            with torch.cuda.stream(s):
                c(1.0)
        torch.cuda.synchronize()
        for c, o, (n, w) in zip(clips, outs, want):
            assert torch.equal(c.norm, n) and all(torch.equal(a, b) for a, b in zip(o, w))
