"""4-bit expert weights (moe_w4_*) against plain 64-bit forms.

Packing and the values that codes stand for are exact, and so is a product
with rows of the identity (one weight times one, rounded to bf16).  Sums are
held to the bounds derived in w4_oracle.py."""
import os

import numpy as np
import pytest
import torch

import mixture_experts_layer_offsets_amd as m
import w4_oracle as wo
from gpu_util import note
from oracle.mx import mx_dequantize, mx_quantize

pytestmark = pytest.mark.gpu

FORMATS = [("mxfp4", 32, "bf16", False), ("int4", 32, "bf16", False), ("int4", 64, "f16", False),
           ("int4", 128, "bf16", False), ("int4", 32, "f16", True), ("int4", 64, "bf16", True),
           ("int4", 128, "f16", True)]
IDS = ["-".join(str(v) for v in f) for f in FORMATS]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mixture_experts_layer_offsets_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_layer_offsets_amd import build
        build.build(verbose=False)
    m.load()


def shape_of(groups, n, k, f):
    return m.W4Shape(groups, n, k, m.MOE_W4_MXFP4 if f[0] == "mxfp4" else m.MOE_W4_INT4, f[1],
                     m.MOE_SCALE_F16 if f[2] == "f16" else m.MOE_SCALE_BF16, int(f[3]))


def make(rng, groups, n, k, f):
    """(W4Linear, codes, scales, zeros) of random weights."""
    codes, scales, zeros = wo.random_weights(rng, groups, n, k, f[0], f[1], f[3])
    sc = torch.from_numpy(scales).cuda()
    if f[0] != "mxfp4":
        sc = sc.to(torch.float16 if f[2] == "f16" else torch.bfloat16)
    z = None if zeros is None else torch.from_numpy(zeros).cuda()
    lin = m.W4Linear.pack(shape_of(groups, n, k, f), torch.from_numpy(codes).cuda(), sc, z)
    return lin, codes, scales, zeros


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


def within(name, got, want, tol):
    err = np.abs(f64(got) - want)
    assert np.all(err <= tol), (name, float((err - tol).max()), float((err / tol).max()))


@pytest.mark.parametrize("f", FORMATS, ids=IDS)
@pytest.mark.parametrize("groups,n,k", [(1, 1, 128), (2, 17, 384), (3, 16, 256), (1, 33, 1152)])
def test_pack_and_values(f, groups, n, k):
    rng = np.random.default_rng([n, k])
    lin, codes, scales, zeros = make(rng, groups, n, k, f)
    want, _ = wo.values(codes, scales, zeros, f[0], f[1])
    assert np.array_equal(f64(lin.values()), want.transpose(0, 2, 1))


@pytest.mark.parametrize("f", FORMATS, ids=IDS)
@pytest.mark.parametrize("n", [1, 16, 37])
@pytest.mark.parametrize("blocks", [1, 3, 5, 12])
def test_identity_rows_give_the_weights(f, n, blocks):
    """Every weight alone, through the product: bf16 of its value, exactly."""
    k = f[1] * blocks
    rng = np.random.default_rng([n, k])
    lin, codes, scales, zeros = make(rng, 1, n, k, f)
    note(f"w4 identity {f} n={n} k={k}")
    out = lin(torch.eye(k, device="cuda").to(torch.bfloat16))
    want, _ = wo.values(codes, scales, zeros, f[0], f[1])
    assert torch.equal(out.cpu(), bf16(want[0].T))


def test_every_mxfp4_scale():
    """Every scale whose values bf16 holds (0..252: 6 * 2^125 is finite; with
    larger ones an infinite weight times the identity's zeros is NaN), down to
    the subnormal values: exact through values() and through the product."""
    scales = np.arange(0, 253, dtype=np.uint8)[:, None]           # one output per scale
    codes = np.tile((np.arange(0, 16, 2) | (np.arange(1, 16, 2) << 4)).astype(np.uint8), (253, 2))
    lin = m.W4Linear.pack(m.W4Shape(1, 253, 32), torch.from_numpy(codes[None]).cuda(),
                          torch.from_numpy(scales[None]).cuda())
    want, _ = wo.values(codes, scales, None, "mxfp4", 32)
    assert np.array_equal(f64(lin.values())[0], want.T)
    out = f64(lin(torch.eye(32, device="cuda").to(torch.bfloat16)))
    assert np.array_equal(out, want.T)


@pytest.mark.parametrize("f", FORMATS, ids=IDS)
@pytest.mark.parametrize("rows,n,k", [(1, 2048, 2048), (1, 5, 7168), (3, 40, 128), (16, 1001, 640),
                                      (17, 64, 1152), (33, 100, 256), (64, 48, 384), (130, 31, 512)])
def test_dense_product(f, rows, n, k):
    rng = np.random.default_rng([rows, n, k])
    lin, codes, scales, zeros = make(rng, 1, n, k, f)
    x = bf16(rng.standard_normal((rows, k)))
    note(f"w4 dense {f} rows={rows} n={n} k={k}")
    w, sabs = wo.values(codes, scales, zeros, f[0], f[1])
    y, bound = wo.product(f64(x), w[0], sabs[0], f[0], f[1])
    out = lin(x.cuda())
    within("dense", out, y, wo.rounded(y, bound))
    assert torch.equal(out, lin(x.cuda()))


@pytest.mark.parametrize("f", [f for f in FORMATS if f[1] == 32], ids=[i for f, i in zip(FORMATS, IDS) if f[1] == 32])
@pytest.mark.parametrize("k", [32, 96, 160, 416])
@pytest.mark.parametrize("rows,n", [(1, 20), (5, 33), (12, 8200), (20, 130), (40, 130), (70, 30)])
def test_contraction_ends_inside_a_tile(f, k, rows, n):
    """k not a multiple of the 128 of a tile, for every way rows are taken."""
    rng = np.random.default_rng([rows, n, k])
    lin, codes, scales, zeros = make(rng, 1, n, k, f)
    x = bf16(rng.standard_normal((rows, k)))
    note(f"w4 tail {f} rows={rows} n={n} k={k}")
    w, sabs = wo.values(codes, scales, zeros, f[0], f[1])
    y, bound = wo.product(f64(x), w[0], sabs[0], f[0], f[1])
    # the values behind the rows are NaN: they must not be read into a product
    wide = torch.full((rows, k + 8), float("nan"), dtype=torch.bfloat16)
    wide[:, :k] = x
    within("tail", lin(wide.cuda()[:, :k]), y, wo.rounded(y, bound))


@pytest.mark.parametrize("f", [FORMATS[0], FORMATS[4]], ids=[IDS[0], IDS[4]])
@pytest.mark.parametrize("rows", [9, 20, 70, 200])
def test_many_outputs(f, rows):
    """Enough tiles for the workgroups that take two of them a wave."""
    n, k = 33000, 128
    rng = np.random.default_rng(rows)
    lin, codes, scales, zeros = make(rng, 1, n, k, f)
    x = bf16(rng.standard_normal((rows, k)))
    note(f"w4 many outputs {f} rows={rows}")
    w, sabs = wo.values(codes, scales, zeros, f[0], f[1])
    y, bound = wo.product(f64(x), w[0], sabs[0], f[0], f[1])
    within("many outputs", lin(x.cuda()), y, wo.rounded(y, bound))


@pytest.mark.parametrize("f", FORMATS, ids=IDS)
@pytest.mark.parametrize("rows,n", [(7, 6200), (8, 8300), (12, 6200), (12, 33000), (20, 4100),
                                    (20, 12300), (20, 33000), (24, 500), (40, 2000), (40, 2100),
                                    (70, 8200), (70, 33000)])
def test_every_choice_of_rows_and_tiles(f, rows, n):
    """Staged rows of every block count, one and two tiles a wave, and split
    contractions of 4, 8 and 16 waves with passes side by side."""
    k = 256 + f[1]
    rng = np.random.default_rng([rows, n])
    lin, codes, scales, zeros = make(rng, 1, n, k, f)
    x = bf16(rng.standard_normal((rows, k)))
    note(f"w4 choice {f} rows={rows} n={n}")
    w, sabs = wo.values(codes, scales, zeros, f[0], f[1])
    y, bound = wo.product(f64(x), w[0], sabs[0], f[0], f[1])
    within("choice", lin(x.cuda()), y, wo.rounded(y, bound))


@pytest.mark.parametrize("f", [FORMATS[0], FORMATS[5]], ids=[IDS[0], IDS[5]])
@pytest.mark.parametrize("n", [100, 1500, 6200])
def test_groups_longer_than_the_average(f, n):
    """Passes side by side are counted from the average: a longer group's
    workgroups walk on, an empty one's have nothing to do."""
    groups, k, off = 3, 256, [0, 101, 101, 120]
    rng = np.random.default_rng(n)
    lin, codes, scales, zeros = make(rng, groups, n, k, f)
    x = bf16(rng.standard_normal((off[-1], k)))
    note(f"w4 long group {f} n={n}")
    out = lin(x.cuda(), torch.tensor(off, dtype=torch.int32, device="cuda"))
    w, sabs = wo.values(codes, scales, zeros, f[0], f[1])
    for g in range(groups):
        rows = slice(off[g], off[g + 1])
        y, bound = wo.product(f64(x[rows]), w[g], sabs[g], f[0], f[1])
        within(f"group {g}", out[rows], y, wo.rounded(y, bound)) if off[g + 1] > off[g] else None


def test_more_passes_than_a_grid_dimension():
    """More than 65535 passes of 32 rows (groups of 32 of INT4), the same 2048
    rows again and again: every one of their outputs is the same."""
    f, n, k, part = FORMATS[4], 8, 32, 2048
    assert f[0] == "int4" and f[1] == 32
    rng = np.random.default_rng(65)
    lin, codes, scales, zeros = make(rng, 1, n, k, f)
    x = bf16(rng.standard_normal((part, k)))
    times = 65536 * 32 // part + 1
    note(f"w4 {times * part} rows")
    out = lin(x.cuda().repeat(times, 1)).view(times, part, n)
    w, sabs = wo.values(codes, scales, zeros, f[0], f[1])
    y, bound = wo.product(f64(x), w[0], sabs[0], f[0], f[1])
    within("first rows", out[0], y, wo.rounded(y, bound))
    assert torch.equal(out, out[:1].expand_as(out))


def test_strides_past_four_gib():
    """Rows of x and out whose byte offsets pass 32 bits."""
    f = FORMATS[0]
    rng = np.random.default_rng(4)
    lin, codes, scales, zeros = make(rng, 1, 40, 256, f)
    w, sabs = wo.values(codes, scales, zeros, f[0], f[1])
    big = torch.empty((5, 1 << 30), dtype=torch.bfloat16, device="cuda")
    for rows in (3, 5):
        x = bf16(rng.standard_normal((rows, 256)))
        big[:rows, :256] = x.cuda()
        lin(big[:rows, :256], out=big[:rows, 512:552])
        y, bound = wo.product(f64(x), w[0], sabs[0], f[0], f[1])
        within("strides", big[:rows, 512:552], y, wo.rounded(y, bound))


def test_packed_past_four_gib():
    """Codes whose byte offsets pass 32 bits: the last of 40 matrices."""
    groups, n, k = 40, 8192, 32768
    g = torch.Generator(device="cuda").manual_seed(3)
    codes = torch.randint(0, 256, (groups, n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(118, 124, (groups, n, k // 32), generator=g, device="cuda",
                           dtype=torch.uint8)
    lin = m.W4Linear.pack(m.W4Shape(groups, n, k), codes, scales)
    assert lin.packed.numel() > 1 << 32
    off = torch.zeros(groups + 1, dtype=torch.int32, device="cuda")
    off[groups] = 2
    x = torch.randn((2, k), generator=g, device="cuda").to(torch.bfloat16)
    note("w4 packed past 4 GiB")
    out = f64(lin(x, off))
    part = slice(n - 64, n)
    c = codes[-1, part].cpu().numpy()
    w, sabs = wo.values(c, scales[-1, part].cpu().numpy(), None, "mxfp4", 32)
    y, bound = wo.product(f64(x), w, sabs, "mxfp4", 32)
    assert np.all(np.abs(out[:, part] - y) <= wo.rounded(y, bound))


@pytest.mark.parametrize("f", FORMATS, ids=IDS)
def test_grouped_strided_product(f):
    """Ragged groups (empty ones, one longer than a pass, rows before the
    first and behind the last), strided x and out at odd offsets."""
    groups, n, k, rows = 6, 45, 3 * 128, 150
    rng = np.random.default_rng(7)
    lin, codes, scales, zeros = make(rng, groups, n, k, f)
    off = np.array([2, 2, 75, 76, 76, 140, 141], np.int32)
    xs = torch.zeros((rows, k + 5), dtype=torch.bfloat16)
    xs[:, 1:k + 1] = bf16(rng.standard_normal((rows, k)))
    x = xs.cuda()[:, 1:k + 1]
    full = torch.full((rows, n + 4), 7.0, dtype=torch.bfloat16, device="cuda")
    lin(x, torch.from_numpy(off).cuda(), out=full[:, 3:n + 3])
    got = full[:, 3:n + 3]
    w, sabs = wo.values(codes, scales, zeros, f[0], f[1])
    for g in range(groups):
        a, b = off[g], off[g + 1]
        y, bound = wo.product(f64(x[a:b]), w[g], sabs[g], f[0], f[1])
        within(f"group {g}", got[a:b], y, wo.rounded(y, bound))
    assert torch.all(full[:, :3] == 7) and torch.all(full[:, n + 3:] == 7)
    assert torch.all(got[:2] == 7) and torch.all(got[141:] == 7)


def test_no_rows_and_bad_offsets():
    rng = np.random.default_rng(1)
    lin = make(rng, 3, 20, 128, FORMATS[0])[0]
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert lin(torch.empty((0, 128), dtype=torch.bfloat16, device="cuda"), off).shape == (0, 20)
    # offsets outside [0, rows] are kept inside: memory-safe, rows still in range
    off = torch.tensor([-5, 1, 2, 1000], dtype=torch.int32, device="cuda")
    out = lin(torch.ones((4, 128), dtype=torch.bfloat16, device="cuda"), off)
    assert torch.all(torch.isfinite(out.float()))


def test_rows_do_not_mix():
    """A NaN or infinity in one row leaves the other rows' bits alone."""
    for f in (FORMATS[0], FORMATS[4]):
        rng = np.random.default_rng(2)
        lin = make(rng, 1, 50, 256, f)[0]
        x = bf16(rng.standard_normal((20, 256))).cuda()
        clean = lin(x)
        bad = x.clone()
        bad[4, 7], bad[11, 100] = float("nan"), float("inf")
        out = lin(bad)
        keep = torch.tensor([r not in (4, 11) for r in range(20)], device="cuda")
        assert torch.equal(out[keep], clean[keep])
        assert not torch.any(torch.isfinite(out[4].float()))
        assert not torch.any(torch.isfinite(out[11].float()) & (lin.values()[0, 100] != 0))


@pytest.mark.parametrize("f", FORMATS, ids=IDS)
@pytest.mark.parametrize("k,n", [(256, 40), (640, 17)])
def test_quantize(f, k, n):
    """The documented steps in fp32, value by value."""
    rng = np.random.default_rng([k, n])
    w = (rng.standard_normal((2, k, n)) * np.exp(rng.standard_normal((2, 1, n)))).astype(np.float32)
    w[0, :f[1], 0] = 0                       # an all-zero group
    w[1, f[1]:2 * f[1], 1] = np.abs(w[1, f[1]:2 * f[1], 1])    # one sign only
    wb = bf16(w)
    w32 = wb.float().numpy()
    lin = m.W4Linear.quantize(wb.cuda(), *(shape_of(1, n, k, f).__dict__[a] for a in
                                           ("format", "group_size", "scale_type", "zeros")))
    got = lin.values().cpu().numpy()
    if f[0] == "mxfp4":
        codes, scales = mx_quantize(w32.astype(np.float64), axis=1, fmt="e2m1")
        assert np.array_equal(got.astype(np.float64), mx_dequantize(codes, scales, axis=1, fmt="e2m1"))
        return
    sdt = torch.float16 if f[2] == "f16" else torch.bfloat16
    b = w32.reshape(2, k // f[1], f[1], n)
    lo, hi = np.minimum(b.min(2), 0), np.maximum(b.max(2), 0)
    s = ((hi - lo) / np.float32(15)) if f[3] else np.maximum(-lo, hi) / np.float32(7)
    s = torch.from_numpy(s.astype(np.float32)).to(sdt).float().numpy()
    safe = np.where(s > 0, s, 1).astype(np.float32)
    z = np.clip(np.rint(-lo / safe), 0, 15) if f[3] else np.full_like(s, 8)
    z = np.where(s > 0, z, 0 if f[3] else 8)
    q = np.clip(np.rint(b / safe[:, :, None]) + z[:, :, None], 0, 15)
    q = np.where(s[:, :, None] > 0, q, z[:, :, None])
    want = (s[:, :, None] * (q - z[:, :, None])).reshape(2, k, n)
    assert np.array_equal(got, want.astype(np.float32))


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
    # contractions that end inside a tile, with few rows an expert and with many
    "tails": (6, 3, 5, 0, 0, 5, 192, 320, 64),
    "heavy-tails": (40, 4, 2, 0, 0, 2, 192, 320, 0),
    # more slots than a workgroup looks through: planned, at each average
    "planned": (100, 4, 64, 5, 0, 80, 128, 64, 64),
    "planned-more": (80, 4, 16, 0, 0, 16, 128, 192, 0),
    "slots-256": (64, 4, 40, 0, 0, 44, 128, 64, 0),
    "slots-257": (257, 1, 40, 0, 0, 44, 128, 64, 0),
    "shared": (7, 2, 6, 0, 0, 6, 256, 128, 320),
    "shared-heavy": (70, 2, 6, -3, -3, 6, 128, 64, 64),
    "k16-E1024": (6, 16, 1024, 0, 0, 1024, 64, 64, 0),
    "most-slots": (256, 16, 24, 0, 0, 24, 128, 64, 0),
    "long": (3, 3, 5, 0, 0, 5, 7168, 2048, 0),
    "wide-plan-E1024": (20, 16, 1024, 0, 0, 1024, 64, 64, 0),
}


def layer_case(name, f, seed=0):
    T, k, E, first, lo, hi, H, I, Is = LAYERS[name]
    rng = np.random.default_rng([seed, sorted(LAYERS).index(name)])
    lins, vals = [], []
    for groups, n, kk in [(E, I, H), (E, I, H), (E, H, I)] + ([(1, Is, H), (1, Is, H), (1, H, Is)]
                                                             if Is else []):
        codes, scales, zeros = wo.random_weights(rng, groups, n, kk, f[0], f[1], f[3])
        down = int(np.log2(kk) / 2) + (2 if f[0] == "mxfp4" else 3)
        if f[0] == "mxfp4":
            scales = np.clip(scales.astype(int) // 8 + 127 - 15 - down, 1, 254).astype(np.uint8)
        else:
            scales = np.ldexp(scales, -down).astype(np.float32)
        sc = torch.from_numpy(scales).cuda()
        if f[0] != "mxfp4":
            sc = sc.to(torch.float16 if f[2] == "f16" else torch.bfloat16)
            scales = sc.float().cpu().numpy()
        lins.append(m.W4Linear.pack(shape_of(groups, n, kk, f), torch.from_numpy(codes).cuda(), sc,
                                    None if zeros is None else torch.from_numpy(zeros).cuda()))
        vals.append(wo.values(codes, scales, zeros, f[0], f[1]))
    idx = rng.integers(lo, hi, (T, k)).astype(np.int32)
    wt = rng.random((T, k)).astype(np.float32)
    x = bf16(rng.standard_normal((T, H)))
    experts = [tuple((v[0][e], v[1][e]) for v in vals[:3]) for e in range(E)]
    shared = tuple((v[0][0], v[1][0]) for v in vals[3:]) if Is else None
    return m.Shape(T, H, E, k, I, Is), lins, x, idx, wt, experts, shared, first


def fits(name, f):
    T, k, E, first, lo, hi, H, I, Is = LAYERS[name]
    return not (H % f[1] or I % f[1] or Is % f[1])


# every format whose group size divides H, I and the shared I (the long
# contraction in two of them)
@pytest.mark.parametrize("name,f", [
    pytest.param(n, f, id=f"{n}-{i}") for n in LAYERS for f, i in zip(FORMATS, IDS)
    if fits(n, f) and (n != "long" or f in (FORMATS[0], FORMATS[6]))])
def test_decode_layer(name, f):
    shape, lins, x, idx, wt, experts, shared, first = layer_case(name, f)
    note(f"w4 decode {name} {f}")
    dec = m.W4Decoder(shape, m.W4Experts.of(*lins, first_expert=first))
    wn = wt.copy()
    wn[(idx < first) | (idx >= first + shape.experts)] = np.nan   # masked slots: unused weights
    args = dict(topk_idx=torch.from_numpy(idx).cuda(), topk_w=torch.from_numpy(wn).cuda())
    out = dec(x.cuda(), **args)
    want, tol = wo.layer(f64(x), idx, wt, experts, first, f[0], f[1], shared)
    within(name, out, want, tol)
    dec.ws.fill_(255)                                            # nothing is kept in the workspace
    assert torch.equal(out, dec(x.cuda(), **args))


def test_decode_with_a_router():
    """The router path is the layer's routing followed by the supplied path."""
    f = FORMATS[0]
    shape, lins, x, _, _, _, _, _ = layer_case("few", f)
    rng = np.random.default_rng(3)
    wr = bf16(rng.standard_normal((shape.hidden, shape.experts)) * 0.1).cuda()
    bias = torch.from_numpy(rng.standard_normal(shape.experts).astype(np.float32)).cuda()
    dec = m.W4Decoder(shape, m.W4Experts.of(*lins))
    out = dec(x.cuda(), w_router=wr, bias=bias)
    logits = torch.empty((shape.tokens, shape.experts), device="cuda")
    ws = torch.empty(m.moe_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
    m.moe_router_logits(shape, x.cuda(), wr, bias, logits, ws)
    idx = torch.empty((shape.tokens, shape.top_k), dtype=torch.int32, device="cuda")
    w = torch.empty((shape.tokens, shape.top_k), device="cuda")
    m.moe_route(shape, logits, idx, w)
    assert torch.equal(out, dec(x.cuda(), topk_idx=idx, topk_w=w))


@pytest.mark.parametrize("f", [FORMATS[0], FORMATS[4]], ids=[IDS[0], IDS[4]])
def test_sorted_rows_through_the_products(f):
    """The operators together: rows sorted by expert (some slots elsewhere,
    segments aligned), the three products on them, the weighted return --
    against the 64-bit layer and the few-token call on the same inputs."""
    name = "share"
    shape, lins, x, idx, wt, experts, shared, first = layer_case(name, f, 4)
    T, H, E, k = shape.tokens, shape.hidden, shape.experts, shape.top_k
    op = m.TokenSort(m.SortShape(T, E, k, H, align=8, first_expert=first))
    xs = op.sort(x.cuda(), torch.from_numpy(idx).cuda(), out=op.sorted_rows().zero_())
    g, u = (lin(xs, op.offsets).float() for lin in lins[:2])
    a = (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16)
    y = lins[2](a, op.offsets)
    out = op.unsort(y, torch.from_numpy(wt).cuda())
    want, tol = wo.layer(f64(x), idx, wt, experts, first, f[0], f[1])
    # three more roundings to bf16 on the way than the few-token call: g, u, y
    size = np.abs(want).max()
    assert np.all(np.abs(f64(out) - want) <= tol + 4 * 2.0 ** -8 * size)
    dec = m.W4Decoder(shape, m.W4Experts.of(*lins, first_expert=first))
    few = dec(x.cuda(), topk_idx=torch.from_numpy(idx).cuda(), topk_w=torch.from_numpy(wt).cuda())
    assert np.all(np.abs(f64(out) - f64(few)) <= tol * 2 + 4 * 2.0 ** -8 * size)


def test_captured_and_replayed_on_another_stream():
    """Product and layer captured into one graph on a side stream, replayed
    with new inputs and routings, bitwise equal to eager calls."""
    f = FORMATS[5]
    shape, lins, x0, idx0, wt0, *_ , first = layer_case("few", f)
    experts = m.W4Experts.of(*lins, first_expert=first)
    dec, eager = m.W4Decoder(shape, experts), m.W4Decoder(shape, experts)
    x, idx, wt = x0.cuda(), torch.from_numpy(idx0).cuda(), torch.from_numpy(wt0).cuda()
    off = torch.tensor([0] + [2] * (shape.experts - 1) + [5], dtype=torch.int32, device="cuda")
    out, lin_out = torch.empty_like(x), torch.zeros((5, shape.inter), dtype=x.dtype, device="cuda")

    def step(d, o, lo):
        d(x, topk_idx=idx, topk_w=wt, out=o)
        lins[0](x, off, out=lo)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(dec, out, lin_out)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(dec, out, lin_out)
    for seed in range(4):
        rng = np.random.default_rng(seed)
        x.copy_(bf16(rng.standard_normal(x0.shape)))
        idx.copy_(torch.from_numpy(rng.integers(-2, shape.experts + 2, idx0.shape).astype(np.int32)))
        out.zero_()
        lin_out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        ref, lref = torch.empty_like(out), torch.zeros_like(lin_out)
        step(eager, ref, lref)
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(lin_out, lref)


@pytest.mark.parametrize("name", ["one-token", "planned", "heavy-expert", "share"])
def test_each_way_of_the_layer_captured(name):
    """One token, planned, staged and few-row layers in a graph, replayed with
    new inputs, routings and a spoiled workspace between the replays."""
    f = FORMATS[2]
    shape, lins, x0, idx0, wt0, *_, first = layer_case(name, f, 7)
    experts = m.W4Experts.of(*lins, first_expert=first)
    dec, eager = m.W4Decoder(shape, experts), m.W4Decoder(shape, experts)
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


def test_two_layers_and_a_product_at_once():
    """Decoders of the same experts on two streams of their own, and a product
    on a third: the same as one after the other."""
    f = FORMATS[0]
    cases = [layer_case(n, f, 9) for n in ("few", "few")]
    shape, lins = cases[0][0], cases[0][1]
    experts = m.W4Experts.of(*lins)
    decs = [m.W4Decoder(shape, experts) for _ in cases]
    rng = np.random.default_rng(12)
    xs = [bf16(rng.standard_normal((shape.tokens, shape.hidden))).cuda() for _ in cases]
    ids = [torch.from_numpy(rng.integers(0, shape.experts, c[3].shape).astype(np.int32)).cuda()
           for c in cases]
    wts = [torch.from_numpy(c[4]).cuda() for c in cases]
    rows = bf16(rng.standard_normal((7, shape.hidden))).cuda()
    off = torch.arange(shape.experts + 1, dtype=torch.int32, device="cuda").clamp_(max=7)
    want = [d(x, topk_idx=i, topk_w=w) for d, x, i, w in zip(decs, xs, ids, wts)]
    want.append(lins[0](rows, off))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(20):
        got = []
        for s, d, x, i, w in zip(streams, decs, xs, ids, wts):
            with torch.cuda.stream(s):
                got.append(d(x, topk_idx=i, topk_w=w))
        with torch.cuda.stream(streams[2]):
            got.append(lins[0](rows, off))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
