"""Tokens sorted by expert and back (moe_sort_*, moe_unsort_*) against plain
64-bit forms.

Layouts and copies are exact.  Sums: every term and partial sum is rounded
once in fp32 (at most 2^-24 relative to the terms' absolute sum S, k terms and
one addend: (k + 1) 2^-24 S), then the result once to the row type (half a
step: eps / 2 of its value, and half the smallest subnormal).  dw is a sum of
`width` products: at most width 2^-24 of the products' absolute sum.
"""
import os

import numpy as np
import pytest
import torch

import mixture_experts_layer_offsets_amd as m
import rows_oracle as ro
from gpu_util import note

pytestmark = pytest.mark.gpu

TYPES = {"bf16": (m.MOE_ROW_BF16, torch.bfloat16), "f16": (m.MOE_ROW_F16, torch.float16),
         "f32": (m.MOE_ROW_F32, torch.float32)}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mixture_experts_layer_offsets_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_layer_offsets_amd import build
        build.build(verbose=False)
    m.load()


# name: T, k, E, width, type, align, first_expert, token gap, row gap, masked share
CASES = {
    "one-token": (1, 8, 256, 7168, "bf16", 1, 0, 0, 0, 0.0),
    "one-slot": (1, 1, 1, 8, "bf16", 1, 0, 0, 0, 0.0),
    "all-masked": (9, 4, 6, 72, "bf16", 16, 0, 0, 0, 1.0),
    "half-masked-f32": (131, 7, 30, 1111, "f32", 1, 15, 5, 0, 0.5),
    "aligned-f16": (77, 3, 16, 1000, "f16", 16, 16, 24, 8, 0.3),
    "align-not-pow2": (50, 2, 5, 136, "bf16", 24, 0, 0, 0, 0.1),
    "k16": (33, 16, 24, 264, "bf16", 1, 0, 0, 0, 0.2),
    "k9-align128": (40, 9, 3, 520, "f32", 128, -1, 0, 4, 0.2),
    "odd-width": (65, 8, 12, 77, "bf16", 8, 0, 0, 0, 0.2),
    "odd-stride": (65, 8, 12, 96, "f16", 1, 0, 3, 1, 0.2),
    "width-1": (70, 4, 5, 1, "bf16", 4, 0, 2, 1, 0.2),
    "width-3-f32": (300, 2, 7, 3, "f32", 1, 0, 0, 0, 0.2),
    "width-7": (19, 3, 7, 7, "f16", 2, 0, 0, 0, 0.0),
    "few-chunks": (500, 4, 9, 24, "bf16", 1, 0, 0, 0, 0.1),
    "E1024": (300, 5, 1024, 64, "bf16", 2, 0, 0, 0, 0.1),
    "two-chunks": (700, 3, 17, 40, "f32", 1, 0, 0, 0, 0.1),
    "many-chunks": (9000, 16, 6, 16, "bf16", 32, 0, 0, 0, 0.1),
    # few slots: in one launch, or layout and rows apart
    "slots-64": (8, 8, 12, 600, "bf16", 4, 0, 0, 0, 0.3),
    "slots-1024": (128, 8, 40, 512, "bf16", 1, 3, 0, 0, 0.2),
    "slots-1024-align": (64, 16, 9, 520, "bf16", 128, -2, 8, 0, 0.1),
    "slots-1025": (205, 5, 40, 512, "bf16", 1, 0, 0, 0, 0.2),
    "small-E1024": (16, 16, 1024, 1000, "f16", 16, 0, 0, 0, 0.1),
    # rows of many chunks at odd byte offsets (tokens and sorted rows)
    "wide-odd": (21, 5, 6, 1031, "bf16", 4, 2, 0, 0, 0.3),
    "wide-odd-stride": (21, 16, 6, 1030, "f16", 1, 0, 3, 5, 0.5),
    "wide-f32": (40, 12, 9, 515, "f32", 2, 0, 0, 2, 0.2),
    "wide": (3, 2, 4, 20000, "bf16", 1, 0, 0, 0, 0.0),
    # one-launch sorts at their limits (x: the others keep their inputs)
    "x-slots-512": (64, 8, 40, 2056, "bf16", 1, 3, 0, 0, 0.2),
    "x-slots-513": (171, 3, 40, 512, "bf16", 1, 0, 0, 0, 0.2),
    "x-slots-256-align": (64, 4, 9, 520, "bf16", 128, -2, 8, 0, 0.1),
    "x-slots-272-align": (17, 16, 9, 520, "f32", 128, -2, 8, 0, 0.1),
}


def make(name, seed=0):
    T, k, E, D, ty, align, first, tgap, rgap, masked = CASES[name]
    rng = np.random.default_rng([seed, sorted(CASES).index(name)])
    idx = rng.integers(0, E, (T, k)).astype(np.int64) + first
    drop = rng.random((T, k)) < masked
    bad = np.array([first - 1, first + E, -1 if not 0 <= -1 - first < E else first - 7,
                    2**31 - 1, -2**31])
    idx[drop] = rng.choice(bad, drop.sum())
    idx = idx.astype(np.int32)
    shape = m.SortShape(T, E, k, D, TYPES[ty][0], align, first, D + tgap if tgap else 0,
                        D + rgap if rgap else 0)
    return shape, idx, rng, TYPES[ty][1]


def rows(rng, n, D, gap, dtype, scale=1.0):
    t = torch.from_numpy(rng.standard_normal((n, D + gap)).astype(np.float32) * scale).to(dtype)
    return t.cuda()[:, :D]


def f64(t):
    return t.detach().cpu().double().numpy()


def close(name, got, want, mag, terms, dtype):
    """|got - want| within the roundings of `terms` fp32 operations and of the type."""
    fi = torch.finfo(dtype)
    tiny = float(np.nextafter(np.float32(0), np.float32(1))) if dtype is torch.float32 else \
        fi.smallest_normal * fi.eps
    acc = terms * 2.0 ** -24 * mag
    tol = acc + (np.abs(want) + acc) * (fi.eps / 2) + tiny
    err = np.abs(f64(got) - want)
    assert np.all(err <= tol), (name, float((err - tol).max()))


@pytest.mark.parametrize("name", list(CASES))
def test_layout_and_rows(name):
    shape, idx, rng, dtype = make(name)
    note(f"sort {name}: {shape}")
    T, k, D = shape.tokens, shape.top_k, shape.width
    counts, offsets, perm, inv = ro.layout(idx, shape.experts, shape.first_expert, shape.align)
    op = m.TokenSort(shape)
    assert op.max_rows == len(perm)
    x = rows(rng, T, D, (shape.token_stride or D) - D, dtype)
    full = torch.full((op.max_rows, shape.row_stride or D), 7.0, dtype=dtype, device="cuda")
    got = op.sort(x, torch.from_numpy(idx).cuda(), out=full[:, :D])
    torch.cuda.synchronize()
    for what, a, b in (("counts", op.counts, counts), ("offsets", op.offsets, offsets),
                       ("perm", op.perm, perm), ("inv", op.inv_perm, inv)):
        assert np.array_equal(a.cpu().numpy(), b), what
    want = torch.full_like(full, 7.0)
    live = torch.from_numpy(np.flatnonzero(perm >= 0)).cuda()
    want[live, :D] = x[torch.from_numpy(perm[perm >= 0] // k).long().cuda()]
    want[torch.from_numpy(ro.padding_rows(counts, offsets)).cuda(), :D] = 0
    assert torch.equal(full, want)       # rows behind the last segment and the gaps untouched
    # the layout alone
    alone = [torch.full_like(b, -7) for b in (op.counts, op.offsets, op.perm, op.inv_perm)]
    m.moe_sort_layout(shape, torch.from_numpy(idx).cuda(), *alone, op.ws)
    for a, b in zip(alone, (op.counts, op.offsets, op.perm, op.inv_perm)):
        assert torch.equal(a, b)
    # the same layout again, other rows
    x2 = rows(rng, T, D, (shape.token_stride or D) - D, dtype)
    op.sort_again(x2, out=full[:, :D])
    want[live, :D] = x2[torch.from_numpy(perm[perm >= 0] // k).long().cuda()]
    assert torch.equal(full, want)
    assert got.data_ptr() == full.data_ptr()


def planned(name):
    shape, idx, rng, dtype = make(name, 1)
    op = m.TokenSort(shape)
    D = shape.width
    gaps = (shape.token_stride or D) - D, (shape.row_stride or D) - D
    op.sort(rows(rng, shape.tokens, D, gaps[0], dtype), torch.from_numpy(idx).cuda())
    counts, offsets, perm, inv = ro.layout(idx, shape.experts, shape.first_expert, shape.align)
    y = rows(rng, op.max_rows, D, gaps[1], dtype)
    # what no slot owns holds NaN: it must not reach any result
    y[torch.from_numpy(perm < 0).cuda()] = float("nan")
    w = rng.standard_normal((shape.tokens, shape.top_k)).astype(np.float32)
    wn = w.copy()
    wn[inv < 0] = np.nan
    return shape, op, y, torch.from_numpy(wn).cuda(), w, (counts, offsets, perm, inv), rng, dtype, gaps


@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("weight,add", [(True, False), (True, True), (False, False), (False, True)])
def test_unsort_and_sort_backward(name, weight, add):
    shape, op, y, wt, w, (counts, offsets, perm, inv), rng, dtype, gaps = planned(name)
    note(f"unsort {name} weight={weight} add={add}")
    T, D = shape.tokens, shape.width
    a = rows(rng, T, D, gaps[0], dtype) if add else None
    full = torch.full((T, D + gaps[0]), 7.0, dtype=dtype, device="cuda")
    if weight or add:
        op.unsort(y, wt if weight else None, a, out=full[:, :D])
    else:
        op.sort_backward(y, out=full[:, :D])
    want, mag = ro.unsort(np.nan_to_num(f64(y)), w if weight else None, inv,
                          None if a is None else f64(a))
    close(name, full[:, :D], want, mag, shape.top_k + 1, dtype)
    assert torch.all(full[:, D:] == 7.0)


@pytest.mark.parametrize("name", list(CASES))
def test_unsort_backward(name):
    shape, op, y, wt, w, (counts, offsets, perm, inv), rng, dtype, gaps = planned(name)
    note(f"unsort backward {name}")
    T, D = shape.tokens, shape.width
    dout = rows(rng, T, D, gaps[0], dtype)
    full = torch.full((op.max_rows, D + gaps[1]), 7.0, dtype=dtype, device="cuda")
    dy, dw = op.unsort_backward(dout, y, wt, dy=full[:, :D])
    want_dy, want_dw, mag = ro.unsort_bwd(f64(dout), np.nan_to_num(f64(y)), w, inv, op.max_rows)
    live = perm >= 0
    close(name, dy[torch.from_numpy(live).cuda()], want_dy[live], np.abs(want_dy[live]), 1, dtype)
    pad = ro.padding_rows(counts, offsets)
    assert torch.all(dy[torch.from_numpy(pad).cuda()] == 0)
    assert torch.all(full[:, D:] == 7.0) and torch.all(full[int(offsets[-1]):] == 7.0)
    close(name, dw, want_dw, mag, D, torch.float32)
    assert torch.all(dw[torch.from_numpy(inv < 0).cuda()] == 0)
    # only dy: y is not read
    from mixture_experts_layer_offsets_amd import _lib
    full2 = torch.full_like(full, 7.0)
    _lib.moe_unsort_bwd(shape, dout, None, wt, op.counts, op.offsets, op.inv_perm, full2[:, :D],
                        None)
    assert torch.equal(full2, full)


def test_gradients_against_differences():
    """unsort(sort(x)) is linear in x, in y and in w: the gradients' products
    with a direction equal the difference of the outputs along it.  fp32 rows;
    each side's roundings are at most (terms) 2^-24 of the absolute sums."""
    shape, idx, rng, dtype = make("half-masked-f32", 3)
    T, k, D = shape.tokens, shape.top_k, shape.width
    op = m.TokenSort(shape)
    gap = shape.token_stride - D
    x, dx_dir = (rows(rng, T, D, gap, dtype) for _ in range(2))
    dout = rows(rng, T, D, gap, dtype)
    w = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    w_dir = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    xs = op.sort(x, torch.from_numpy(idx).cuda()).clone()
    end = int(op.offsets[-1])
    xs[end:] = 0
    out = op.unsort(xs, w).clone()
    dy, dw = op.unsort_backward(dout, xs, w)
    dy[end:] = 0
    dx = op.sort_backward(dy)
    moved = op.unsort(op.sort_again(dx_dir), w)            # the derivative along dx_dir
    lhs, rhs = (f64(dout) * f64(moved)).sum(), (f64(dx) * f64(dx_dir)).sum()
    mag = (np.abs(f64(dout)) * np.abs(f64(moved))).sum() + (np.abs(f64(dx)) * np.abs(f64(dx_dir))).sum()
    assert abs(lhs - rhs) <= 2 * (k + 2) * 2.0 ** -24 * mag * 4
    eps = 0.5
    plus = op.unsort(xs, w + eps * w_dir)
    diff = (f64(dout) * (f64(plus) - f64(out))).sum()
    grad = eps * (f64(dw) * f64(w_dir)).sum()
    mag = (np.abs(f64(dout)) * (np.abs(f64(plus)) + np.abs(f64(out)))).sum()
    assert abs(diff - grad) <= (D + 2 * k + 4) * 2.0 ** -24 * mag


def test_nonfinite_values_stay_in_their_token():
    """An infinity or NaN in one token's row reaches that token alone."""
    shape, idx, rng, dtype = make("aligned-f16", 5)
    op = m.TokenSort(shape)
    D = shape.width
    x = rows(rng, shape.tokens, D, shape.token_stride - D, dtype)
    x[3, 0], x[5, D - 1] = float("inf"), float("nan")
    xs = op.sort(x, torch.from_numpy(idx).cuda())
    out = op.unsort(xs, torch.ones(shape.tokens, shape.top_k, device="cuda"))
    inv = op.inv_perm.cpu().numpy()
    for t, c in ((3, 0), (5, D - 1)):
        if (inv[t] >= 0).any():
            assert not torch.isfinite(out[t, c])
            out[t, c] = 0
    assert torch.all(torch.isfinite(out))
    # the largest fp16 values overflow to infinity when doubled, as fp16 does
    big = op.sorted_rows().fill_(torch.finfo(torch.float16).max)
    two = op.unsort(big, torch.full((shape.tokens, shape.top_k), 2.0, device="cuda"))
    kept = torch.from_numpy((inv >= 0).any(1)).cuda()
    assert torch.all(torch.isinf(two[kept])) and torch.all(two[~kept] == 0)


def test_no_tokens():
    shape = m.SortShape(0, 5, 3, 64, align=8)
    op = m.TokenSort(shape)
    op.counts.fill_(-7)
    op.offsets.fill_(-7)
    xs = op.sort(op.token_rows(), torch.empty((0, 3), dtype=torch.int32, device="cuda"))
    assert xs.shape == (0, 64)
    assert torch.all(op.counts == 0) and torch.all(op.offsets == 0)
    assert op.unsort(xs, torch.empty((0, 3), device="cuda")).shape == (0, 64)
    dy, dw = op.unsort_backward(op.token_rows(), xs, torch.empty((0, 3), device="cuda"))
    assert dy.shape == (0, 64) and dw.shape == (0, 3)


@pytest.mark.parametrize("name", ["one-token", "aligned-f16", "many-chunks"])
def test_captured_and_replayed_on_another_stream(name):
    """The four calls captured into one graph on a side stream, replayed with
    new inputs and eager work between the replays; bitwise equal to eager
    calls (which also repeat bitwise)."""
    shape, _, rng, dtype = make(name)
    D = shape.width
    tg, rg = (shape.token_stride or D) - D, (shape.row_stride or D) - D
    op, eager = m.TokenSort(shape), m.TokenSort(shape)
    x = rows(rng, shape.tokens, D, tg, dtype)
    dout = rows(rng, shape.tokens, D, tg, dtype)
    w = torch.rand((shape.tokens, shape.top_k), device="cuda")
    idx = torch.from_numpy(make(name)[1]).cuda()
    bufs = dict(xs=op.sorted_rows().zero_(), out=op.token_rows(), dy=op.sorted_rows().zero_(),
                dw=torch.empty_like(w), dx=op.token_rows())

    def step(o, b):
        o.sort(x, idx, out=b["xs"])
        o.unsort(b["xs"], w, out=b["out"])
        o.unsort_backward(dout, b["xs"], w, dy=b["dy"], dtopk_w=b["dw"])
        o.sort_backward(b["dy"], out=b["dx"])

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(op, bufs)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(op, bufs)
    for seed in range(4):
        _, new, r2, _ = make(name, 10 + seed)
        idx.copy_(torch.from_numpy(new))
        x.copy_(rows(r2, shape.tokens, D, 0, dtype))
        dout.copy_(rows(r2, shape.tokens, D, 0, dtype))
        for b in bufs.values():
            b.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for _ in range(2):
            ref = {n: torch.zeros_like(b) for n, b in bufs.items()}
            ref["xs"] = eager.sorted_rows().zero_()
            ref["dy"] = eager.sorted_rows().zero_()
            ref["out"], ref["dx"] = eager.token_rows(), eager.token_rows()
            step(eager, ref)
            torch.cuda.synchronize()
            for n in bufs:
                assert torch.equal(bufs[n], ref[n]), (seed, n)
        assert torch.equal(op.perm, eager.perm) and torch.equal(op.offsets, eager.offsets)


def test_buffers_past_four_gib():
    """Rows whose byte offsets pass 32 bits (sorted rows of 4.6 GB)."""
    T, k, E, D = 40000, 8, 64, 7168
    shape = m.SortShape(T, E, k, D)
    note(f"large {shape}")
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((T, D), generator=g, device="cuda").to(torch.bfloat16)
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand((T, k), generator=g, device="cuda")
    op = m.TokenSort(shape)
    xs = op.sort(x, idx)
    perm = op.perm.long()
    assert torch.equal(perm.sort().values, torch.arange(T * k, device="cuda"))
    for part in torch.arange(T * k, device="cuda").split(1 << 16):
        assert torch.equal(xs[part], x[perm[part] // k])
    out = op.unsort(xs, w)          # the rows are copies: out = x * sum_j w, in fp32 steps
    ref = x.double() * w.double().sum(1, keepdim=True)
    tol = ref.abs() * (2.0 ** -8 + (k + 2) * 2.0 ** -23)
    assert torch.all((out.double() - ref).abs() <= tol)
    del ref, tol
    dy, dw = op.unsort_backward(x, xs, w)
    for part in torch.arange(T * k, device="cuda").split(1 << 16):
        f = perm[part]
        assert torch.equal(dy[part], (x[f // k].float() * w.reshape(-1)[f][:, None]).to(torch.bfloat16))
    norm = (x.double() ** 2).sum(1, keepdim=True)
    assert torch.all((dw.double() - norm).abs() <= D * 2.0 ** -24 * norm)


def test_same_layout_as_the_layer():
    """Without masks and alignment the layout is moe_layout's, and the rows
    returned are moe_dispatch's and moe_combine's, bit for bit."""
    T, k, E, H = 300, 6, 24, 256
    rng = np.random.default_rng(3)
    idx = torch.from_numpy(rng.integers(0, E, (T, k)).astype(np.int32)).cuda()
    x = rows(rng, T, H, 0, torch.bfloat16)
    w = torch.rand((T, k), device="cuda")
    layer = m.Shape(T, H, E, k, 64)
    i32 = dict(dtype=torch.int32, device="cuda")
    lay = [torch.empty(n, **i32) for n in (E, E + 1, T * k, T * k)]
    ws = torch.empty(m.moe_workspace_bytes(layer), dtype=torch.uint8, device="cuda")
    m.moe_layout(layer, idx, *lay, ws)
    xp, out = torch.empty((T * k, H), **i32).to(torch.bfloat16), torch.empty_like(x)
    m.moe_dispatch(layer, x, lay[2], xp)
    m.moe_combine(layer, xp, w, lay[3], None, out)
    op = m.TokenSort(m.SortShape(T, E, k, H))
    xs = op.sort(x, idx)
    for a, b in zip(lay, (op.counts, op.offsets, op.perm, op.inv_perm.reshape(-1))):
        assert torch.equal(a, b)
    assert torch.equal(xs, xp) and torch.equal(op.unsort(xs, w), out)
