"""8-bit products with a scale per block of 128 (moe_f8_*) against plain 64-bit
forms.

Packing, quantising and the values that codes stand for are exact, and so is a
product with rows of the identity (one weight times one, rounded to the rows' type).
Sums are held to the bounds derived in f8_oracle.py."""
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
BOTH = pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mixture_experts_layer_offsets_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_layer_offsets_amd import build
        build.build(verbose=False)
    m.load()


def make(rng, groups, n, k, dtype=BF):
    """(F8Linear, values [groups][n][k] in 64 bits) of random codes."""
    codes, scales, w = fo.random_codes(rng, groups, n, k)
    shape = m.F8Shape(groups, n, k, ROW[dtype])
    return m.F8Linear.pack(shape, torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()), w


def rows(rng, M, k, dtype=BF):
    """Rows whose columns differ in size."""
    x = rng.standard_normal((M, k)) * np.exp(rng.standard_normal(k))
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def within(name, got, want, tol):
    err = np.abs(f64(got) - want)
    assert np.all(err <= tol), (name, float((err - tol).max()), float((err / np.maximum(tol, 1e-300)).max()))


def check(name, got, x, w, dtype):
    """got [M][n] against the rows x (host tensor) times w [n][k]."""
    y, bound = fo.product(fo.rows_quantised(x.float().numpy())[2], w)
    within(name, got, y, fo.rounded(y, bound, dtype))


def offsets(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ packing

@pytest.mark.parametrize("groups,n,k", [(1, 1, 1), (2, 17, 130), (3, 128, 256), (1, 300, 129), (2, 140, 40)])
def test_pack_and_values(groups, n, k):
    rng = np.random.default_rng([n, k])
    lin, w = make(rng, groups, n, k)
    assert np.array_equal(f64(lin.values()), w.transpose(0, 2, 1).astype(np.float32))


@pytest.mark.parametrize("groups,n,k", [(1, 1, 1), (2, 17, 130), (1, 300, 129), (3, 256, 128)])
def test_transposed(groups, n, k):
    """The same values turned, and turned twice the same packed bytes."""
    rng = np.random.default_rng([n, k, 1])
    lin, w = make(rng, groups, n, k)
    turned = lin.transposed()
    assert turned.shape == m.F8Shape(groups, k, n)
    assert np.array_equal(f64(turned.values()), w.astype(np.float32))
    assert torch.equal(turned.transposed().values(), lin.values())
    size = lin.shape.groups * -(-n // 16) * -(-k // 128) * (2048 + 4)
    assert torch.equal(turned.transposed().packed[:size], lin.packed[:size])


@pytest.mark.parametrize("dtype", [BF, FP, torch.float32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("groups,k,n", [(1, 1, 1), (2, 200, 150), (1, 128, 300)])
def test_quantize(groups, k, n, dtype):
    """The documented steps in fp32, value by value."""
    rng = np.random.default_rng([k, n])
    w = torch.from_numpy((rng.standard_normal((groups, k, n)) * np.exp(rng.standard_normal((1, k, 1))))
                         .astype(np.float32)).to(dtype)
    if k > 128:
        w[0, :128, :128] = 0          # an all-zero block
    got = m.F8Linear.quantize(w.cuda()).values()
    assert np.array_equal(f64(got), fo.weights_quantised(w.float().numpy()).astype(np.float32))


def quantised(x, k, dtype):
    M = x.shape[0]
    ks = -(-k // 128)
    codes = torch.full((ks, M, 128), 255, dtype=torch.uint8, device="cuda")
    scales = torch.full((ks, M), -1.0, device="cuda")
    m.moe_f8_quantize_rows(m.F8Shape(1, 1, k, ROW[dtype]), x, codes, scales)
    return codes, scales


@BOTH
@pytest.mark.parametrize("M,k,pad", [(1, 1, 0), (3, 127, 0), (17, 128, 5), (40, 640, 3), (5, 1030, 1), (33, 8, 0)])
def test_quantize_rows(M, k, pad, dtype):
    """Codes and scales bit for bit; rows at odd strides; zero codes past k."""
    rng = np.random.default_rng([M, k])
    x = rows(rng, M, k + pad, dtype)
    x[0, :min(k, 128)] = 0
    if M > 2:
        x[2, 0] = torch.finfo(dtype).max
        x[1, 0] = torch.finfo(dtype).tiny
    codes, scales = quantised(x.cuda()[:, :k], k, dtype)
    c, s, _ = fo.rows_quantised(x[:, :k].float().numpy())
    assert np.array_equal(scales.cpu().numpy(), s.T)
    assert np.array_equal(codes.cpu().numpy(), c.transpose(1, 0, 2))


def test_every_rounding():
    """Values on and next to every border between two codes, of both signs."""
    grid = np.unique(np.abs(fo.decode(np.arange(127, dtype=np.uint8))))
    mid = (grid[1:] + grid[:-1]) / 2
    v = np.concatenate([grid, mid, mid * (1 - 2.0 ** -9), mid * (1 + 2.0 ** -9)])
    v = np.concatenate([v, -v])
    x = np.zeros((len(v) // 64 + 1, 128), np.float32)
    x[:, 0] = 448                        # a scale of about one
    x.reshape(-1)[np.arange(len(v)) // 64 * 128 + 64 + np.arange(len(v)) % 64] = v
    for dtype in (BF, FP):
        xt = torch.from_numpy(x).to(dtype)
        codes, _ = quantised(xt.cuda(), 128, dtype)
        assert np.array_equal(codes.cpu().numpy()[0], fo.rows_quantised(xt.float().numpy())[0][:, 0])


# ------------------------------------------------------------------ products

@BOTH
@pytest.mark.parametrize("n", [1, 16, 37, 300])
@pytest.mark.parametrize("k", [1, 40, 128, 300])
def test_identity_rows_give_the_weights(n, k, dtype):
    """Every weight alone, through the product.  A row of the identity is 448 / 448:
    its code is the largest, its scale 1 / 448 in fp32, so that a result is off by
    the roundings of 448 (1 / 448) and of two products in fp32 at most."""
    rng = np.random.default_rng([n, k])
    lin, w = make(rng, 1, n, k, dtype)
    note(f"f8 identity n={n} k={k} {dtype}")
    out = lin(torch.eye(k, device="cuda").to(dtype))
    want = w[0].T
    within("identity", out, want, np.abs(want) * (fo.HALF[dtype] + 4 * fo.ULP) + fo.LEAST[dtype])


@BOTH
@pytest.mark.parametrize("M,n,k", [
    (1, 2048, 2048), (1, 5, 7168), (1, 1, 1), (3, 40, 128), (16, 1001, 640), (2, 9000, 70), (7, 5000, 200),
    (17, 64, 1152), (33, 100, 256), (64, 48, 384), (65, 256, 129), (130, 31, 512), (128, 513, 77),
    (300, 300, 1000), (257, 520, 2000), (1000, 17, 130)])
def test_dense_product(M, n, k, dtype):
    rng = np.random.default_rng([M, n, k])
    lin, w = make(rng, 1, n, k, dtype)
    x = rows(rng, M, k, dtype)
    note(f"f8 dense rows={M} n={n} k={k} {dtype}")
    out = lin(x.cuda())
    check("dense", out, x, w[0], dtype)
    # the same from rows that are quantised already
    codes, scales = quantised(x.cuda(), k, dtype)
    again = torch.empty_like(out)
    m.moe_f8_linear_codes(lin.shape, codes, scales, None, lin.packed, again)
    check("codes", again, x, w[0], dtype)


def grouped_case(seed, groups, n, k, off, M, dtype, pads=(5, 4)):
    rng = np.random.default_rng(seed)
    lin, w = make(rng, groups, n, k, dtype)
    xs = rows(rng, M, k + pads[0], dtype)
    x = xs.cuda()[:, 1:k + 1]
    full = torch.full((M, n + pads[1]), 7.0, dtype=dtype, device="cuda")
    return lin, w, xs[:, 1:k + 1], x, full


# ragged groups: empty ones, ones longer than a tile, rows before the first and behind the last
SPANS = {
    "few": (80, [2, 2, 9, 10, 10, 40, 41]),
    "one-long": (700, [3, 3, 640, 641, 641, 690, 691]),
    "tiles": (1400, [0, 256, 512, 513, 1024, 1024, 1300]),
    "middle": (560, [10, 100, 164, 300, 428, 429, 557]),
    "empty": (40, [20] * 7),
}


@BOTH
@pytest.mark.parametrize("n,k", [(45, 3 * 128), (300, 200), (4999, 200)])
@pytest.mark.parametrize("name", list(SPANS))
def test_grouped_strided_product(name, n, k, dtype):
    """x and out at odd offsets and strides; rows in no group are left as they were."""
    M, off = SPANS[name]
    groups = len(off) - 1
    lin, w, xh, x, full = grouped_case([7, n], groups, n, k, off, M, dtype)
    note(f"f8 grouped {name} n={n} k={k} {dtype}")
    got = full[:, 3:n + 3]
    lin(x, offsets(off), out=got)
    for g in range(groups):
        a, b = off[g], off[g + 1]
        if b > a:
            check(f"group {g}", got[a:b], xh[a:b], w[g], dtype)
    assert torch.all(full[:, :3] == 7) and torch.all(full[:, n + 3:] == 7)
    assert torch.all(got[:off[0]] == 7) and torch.all(got[off[-1]:] == 7)


def test_many_groups():
    """1024 groups, most of them empty."""
    groups, n, k, M = 1024, 20, 130, 300
    rng = np.random.default_rng(5)
    lin, w = make(rng, groups, n, k)
    x = rows(rng, M, k)
    ids = np.sort(rng.choice(groups, M) // 7 * 7)
    off = np.searchsorted(ids, np.arange(groups + 1)).astype(np.int32)
    note("f8 1024 groups")
    for size in (M, 20):
        o = np.minimum(off, size)
        out = lin(x[:size].cuda(), torch.from_numpy(o).cuda())
        for g in np.unique(ids[:size]):
            check(f"group {g}", out[o[g]:o[g + 1]], x[o[g]:o[g + 1]], w[g], BF)


def test_no_rows_and_bad_offsets():
    rng = np.random.default_rng(1)
    lin, _ = make(rng, 3, 20, 128)
    assert lin(torch.empty((0, 128), dtype=BF, device="cuda"), offsets([0] * 4)).shape == (0, 20)
    # offsets outside [0, rows] are kept inside: memory-safe, rows still in range
    for M in (4, 400, 40000):
        out = lin(torch.ones((M, 128), dtype=BF, device="cuda"), offsets([-5, 1, 2, 100000]))
        assert torch.all(torch.isfinite(out.float()))
        out = lin(torch.ones((M, 128), dtype=BF, device="cuda"), offsets([M, 1, 5, 0]))
        assert torch.all(torch.isfinite(out.float()))


@pytest.mark.parametrize("M", [12, 300, 20000])
def test_rows_do_not_mix(M):
    """A NaN or infinity in one row leaves the other rows' bits alone."""
    rng = np.random.default_rng(2)
    lin, _ = make(rng, 1, 50, 300)
    x = rows(rng, M, 300).cuda()
    clean = lin(x)
    bad = x.clone()
    bad[4, 7], bad[11, 290] = float("nan"), float("-inf")
    out = lin(bad)
    keep = torch.tensor([r not in (4, 11) for r in range(M)], device="cuda")
    assert torch.equal(out[keep], clean[keep])
    assert not torch.any(torch.isfinite(out[4].float())) and not torch.any(torch.isfinite(out[11].float()))


@pytest.mark.parametrize("M", [5, 200, 20000])
def test_large_and_small_rows(M):
    """Rows next to bf16's largest and smallest values: as the oracle's."""
    rng = np.random.default_rng(9)
    codes, _, _ = fo.random_codes(rng, 1, 40, 256)
    for size, scale in ((1e38, 1e-6), (1e-36, 1.0), (0.0, 1.0)):
        scales = np.full((1, 1, 2), scale, np.float32)
        lin = m.F8Linear.pack(m.F8Shape(1, 40, 256), torch.from_numpy(codes).cuda(),
                              torch.from_numpy(scales).cuda())
        x = (torch.rand(M, 256, generator=torch.Generator().manual_seed(3)) * 2 * size).to(BF)
        x = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
        w = fo.weight_values(codes, scales)[0]
        y, bound = fo.product(fo.rows_quantised(x.float().numpy())[2], w)
        out = f64(lin(x.cuda()))
        tol = fo.rounded(y, bound, BF)
        assert np.all((np.abs(out - y) <= tol) | (np.abs(y) + tol > 3.38e38))


def test_strides_past_four_gib():
    """Rows of x and out whose byte offsets pass 32 bits."""
    rng = np.random.default_rng(4)
    lin, w = make(rng, 1, 40, 256)
    big = torch.empty((40, 1 << 27), dtype=BF, device="cuda")
    for M in (3, 40):
        x = rows(rng, M, 256)
        big[:M, :256] = x.cuda()
        lin(big[:M, :256], out=big[:M, 512:552])
        check("strides", big[:M, 512:552], x, w[0], BF)


def test_strides_past_four_gib_in_tiles():
    """The same in tiles of 128 rows: the rows behind 4 GiB."""
    rng = np.random.default_rng(14)
    M, n = 600, 8192
    lin, w = make(rng, 1, n, 256)
    big = torch.empty((M, 1 << 23), dtype=BF, device="cuda")
    x = rows(rng, M, 256)
    big[:, :256] = x.cuda()
    note("f8 strides past 4 GiB in tiles")
    lin(big[:, :256], out=big[:, 512:512 + n])
    check("strides", big[:, 512:512 + n], x, w[0], BF)


def test_packed_past_four_gib():
    """Codes whose byte offsets pass 32 bits: the last of 20 matrices."""
    groups, n, k = 20, 8192, 32768
    codes = torch.randint(0, 127, (1, n, k), device="cuda", dtype=torch.uint8).expand(groups, n, k).contiguous()
    codes[-1] = codes[-1] ^ 128
    scales = torch.full((groups, n // 128, k // 128), 2.0 ** -9, device="cuda")
    lin = m.F8Linear.pack(m.F8Shape(groups, n, k), codes, scales)
    assert lin.packed.numel() > 1 << 32
    for M in (2, 400):
        x = torch.randn((M, k), generator=torch.Generator().manual_seed(3)).to(BF)
        note(f"f8 packed past 4 GiB, {M} rows")
        out = lin(x.cuda(), offsets([0] * groups + [M]))
        part = slice(n - 64, n)
        w = fo.weight_values(codes[-1:, part].cpu().numpy(), scales[-1:, -1:].cpu().numpy())
        check("last", out[:2, part], x[:2], w[0], BF)


def test_every_group_the_same():
    """Long groups take the same values in every tile: bitwise equal rows."""
    rng = np.random.default_rng(8)
    lin, w = make(rng, 1, 300, 256)
    x = rows(rng, 16, 256)
    out = lin(x.repeat(1500, 1).cuda())
    check("rows", out[:16], x, w[0], BF)
    assert torch.equal(out, out[:16].repeat(1500, 1))


def repeated(rng, groups, reps, k, dtype):
    """F8Linear of 256 random outputs that follow one another `reps` times, and their values."""
    codes, scales, w = fo.random_codes(rng, groups, 256, k)
    lin = m.F8Linear.pack(m.F8Shape(groups, 256 * reps, k, ROW[dtype]),
                          torch.from_numpy(codes).cuda().repeat(1, reps, 1),
                          torch.from_numpy(scales).cuda().repeat(1, reps, 1))
    return lin, w


# each choice of workgroup by the numbers of rows, outputs and groups: (rows, end of every
# group's rows, times 256 outputs, contraction)
CHOICES = {
    "8 rows quantised first, 16 waves": (8, None, 10, 62 * 128),
    "8 waves": (8, None, 20, 40 * 128),
    "4 waves": (8, None, 40, 20 * 128),
    "8 rows on average, some groups longer": (24, [0, 1, 23], 14, 20 * 128),
    "24 rows, few outputs": (24, None, 10, 390),
    "pairs of tiles": (24, None, 40, 390),
    "pairs of tiles, two passes": (50, None, 20, 130),
    "pairs of tiles, 4 waves": (12, None, 80, 130),
    "pairs of tiles, 4 waves, groups": (30, [3, 27, 27], 28, 130),
    "pairs of tiles, 64 rows": (60, None, 40, 390),
    "4 tiles, 64 rows": (60, None, 60, 390),
    "4 tiles, 64 rows, two passes": (100, None, 30, 130),
    "one group long": (96, [2, 3, 95], 4, 390),
    "passes of 8, 16 waves": (200, None, 1, 390),
    "passes of 8, 8 waves": (33, None, 5, 520),
    "passes of 8, 4 waves": (500, [100, 100, 101, 499], 1, 130),
    "tiles of 128 rows": (600, None, 40, 390),
    "tiles of 128 rows, groups": (500, [1, 166, 495], 28, 520),
    "tiles of 256 rows": (500, None, 128, 390),
    "tiles of 256 rows, groups": (2000, [5, 70, 1999], 28, 520),
}


@BOTH
@pytest.mark.parametrize("name", list(CHOICES))
def test_each_choice(name, dtype):
    M, ends, reps, k = CHOICES[name]
    rng = np.random.default_rng([M, reps, k])
    ends = [M] if ends is None else ends
    lin, w = repeated(rng, len(ends), reps, k, dtype)
    x = rows(rng, M, k, dtype)
    note(f"f8 {name} {dtype}")
    off = offsets([0] + ends)
    out = lin(x.cuda(), off)
    codes, scales = quantised(x.cuda(), k, dtype)
    again = torch.zeros_like(out)
    m.moe_f8_linear_codes(lin.shape, codes, scales, off, lin.packed, again)
    for got in (out.view(M, reps, 256), again.view(M, reps, 256)):
        assert torch.equal(got, got[:, :1].expand(M, reps, 256))
        for g, (a, b) in enumerate(zip([0] + ends, ends)):
            if b > a:
                check(f"group {g}", got[a:b, 0], x[a:b], w[g], dtype)
        assert torch.all(got[ends[-1]:] == 0)


@pytest.mark.parametrize("k,reps", [(300, 1), (300, 3), (520, 24), (520, 128)],
                         ids=["64", "64-uneven", "128", "256"])
def test_each_choice_of_the_weight_gradient(k, reps):
    """Tiles of 64, 128 and 256 rows of dw."""
    rng = np.random.default_rng([k, reps])
    M, off = 420, [3, 3, 390] if reps > 1 else [3, 200, 390]
    lin, _ = repeated(rng, 2, reps, k, FP)
    x, dy = rows(rng, M, k, FP), rows(rng, M, 256, FP)
    note(f"f8 weight gradient {k} x {256 * reps}")
    got = lin.weight_gradient(x.cuda(), dy.cuda().repeat(1, reps), offsets(off)).view(2, k, reps, 256)
    assert torch.equal(got, got[:, :, :1].expand(2, k, reps, 256))
    for g in range(2):
        span = slice(off[g], off[g + 1])
        dw, bound = fo.weight_gradient(x[span].float().numpy(), dy[span].float().numpy())
        within(f"group {g}", got[g, :, 0], dw, fo.rounded(dw, bound, FP))


def test_many_groups_of_many_rows():
    """More groups than lanes, in tiles of 128 rows, empty ones among them."""
    groups, n, k = 300, 20, 130
    rng = np.random.default_rng(15)
    lin, w = make(rng, groups, n, k)
    lengths = rng.integers(0, 90, groups)
    lengths[[0, 63, 64, 65, 299]] = 0
    lengths[[5, 128]] = 300
    off = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    x = rows(rng, int(off[-1]), k)
    note("f8 300 groups")
    out = lin(x.cuda(), torch.from_numpy(off).cuda())
    for g in range(groups):
        if lengths[g]:
            check(f"group {g}", out[off[g]:off[g + 1]], x[off[g]:off[g + 1]], w[g], BF)


@pytest.mark.parametrize("M", [3, 40, 300, 20000])
def test_out_beside_x_in_one_buffer(M):
    """Rows of x and out that lie between each other's."""
    rng = np.random.default_rng(M)
    lin, w = make(rng, 1, 50, 200)
    x = rows(rng, M, 200)
    both = torch.zeros((M, 260), dtype=BF, device="cuda")
    both[:, 60:] = x.cuda()
    lin(both[:, 60:], out=both[:, 5:55])
    check("beside", both[:, 5:55], x, w[0], BF)
    assert torch.equal(both[:, 60:].cpu(), x)


# ------------------------------------------------------------------ gradients

@BOTH
@pytest.mark.parametrize("groups,M,n,k", [(1, 5, 40, 130), (3, 90, 150, 64), (2, 700, 260, 300),
                                            (3, 9000, 130, 300)])
def test_data_gradient(groups, M, n, k, dtype):
    """dx of x*W is dy's 8-bit values times W^T."""
    rng = np.random.default_rng([M, n])
    lin, w = make(rng, groups, n, k, dtype)
    dy = rows(rng, M, n, dtype)
    off = np.linspace(0, M, groups + 1).astype(np.int32)
    dx = lin.transposed()(dy.cuda(), torch.from_numpy(off).cuda())
    for g in range(groups):
        check(f"group {g}", dx[off[g]:off[g + 1]], dy[off[g]:off[g + 1]], w[g].T, dtype)


@BOTH
@pytest.mark.parametrize("name,n,k", [
    ("few", 1, 1), ("few", 45, 300), ("one-long", 300, 130), ("tiles", 33, 520), ("middle", 257, 64),
    ("empty", 40, 40), ("few", 1031, 300), ("one-long", 1030, 170), ("middle", 301, 1027), ("tiles", 720, 520),
    ("empty", 700, 700), ("one-long", 1030, 670), ("middle", 301, 2027)])
def test_weight_gradient(name, n, k, dtype):
    M, off = SPANS[name]
    rng = np.random.default_rng([n, k])
    x, dy = rows(rng, M, k + 3, dtype), rows(rng, M, n + 5, dtype)
    x[:, 0] *= 100
    lin, _ = make(rng, len(off) - 1, n, k, dtype)
    note(f"f8 weight gradient {name} n={n} k={k} {dtype}")
    out = torch.full((len(off) - 1, k, n), 7.0, dtype=dtype, device="cuda")
    got = lin.weight_gradient(x.cuda()[:, 1:k + 1], dy.cuda()[:, 2:n + 2], offsets(off), out=out)
    for g in range(len(off) - 1):
        span = slice(off[g], off[g + 1])
        dw, bound = fo.weight_gradient(x[span, 1:k + 1].float().numpy(), dy[span, 2:n + 2].float().numpy())
        within(f"group {g}", got[g], dw, fo.rounded(dw, bound, dtype))


@BOTH
@pytest.mark.parametrize("M,off,n,k", [
    (17000, [0, 17000], 33, 40), (5000, [7, 4000, 4990], 45, 300), (8000, [5, 5, 6, 7999], 300, 130)])
def test_weight_gradient_of_many_rows(M, off, n, k, dtype):
    """Each group's rows in pieces, some of them without a stage."""
    rng = np.random.default_rng([M, n])
    x, dy = rows(rng, M, k, dtype), rows(rng, M, n + 1, dtype)
    groups = len(off) - 1
    lin, _ = make(rng, groups, n, k, dtype)
    note(f"f8 weight gradient of {M} rows n={n} k={k} {dtype}")
    got = lin.weight_gradient(x.cuda(), dy.cuda()[:, 1:], offsets(off))
    for g in range(groups):
        span = slice(off[g], off[g + 1])
        dw, bound = fo.weight_gradient(x[span].float().numpy(), dy[span, 1:].float().numpy())
        within(f"group {g}", got[g], dw, fo.rounded(dw, bound, dtype))


def test_weight_gradient_without_rows():
    lin, _ = make(np.random.default_rng(0), 3, 40, 50)
    got = lin.weight_gradient(torch.empty((0, 50), dtype=BF, device="cuda"),
                              torch.empty((0, 40), dtype=BF, device="cuda"), offsets([0] * 4),
                              out=torch.full((3, 50, 40), 7.0, dtype=BF, device="cuda"))
    assert torch.all(got == 0)


def test_weight_gradient_columns_do_not_mix():
    """A NaN in one column of x reaches that row of dw only."""
    rng = np.random.default_rng(3)
    lin, _ = make(rng, 1, 40, 50)
    x, dy = rows(rng, 200, 50).cuda(), rows(rng, 200, 40).cuda()
    clean = lin.weight_gradient(x, dy)
    x[130, 7], dy[3, 9] = float("nan"), float("inf")
    got = lin.weight_gradient(x, dy)
    keep = torch.ones((50, 40), dtype=torch.bool, device="cuda")
    keep[7], keep[:, 9] = False, False
    assert torch.equal(got[0][keep], clean[0][keep])
    assert not torch.any(torch.isfinite(got[0][~keep].float()))


def test_gradients_against_differences():
    """With values that 8 bits hold exactly (a 448 in every block meets zero weights),
    y = x W is linear in x and in W, so that <dy, y(x + d) - y(x)> = <dx, d> and the
    same in W: all numbers are small integers, which every type here holds."""
    rng = np.random.default_rng(6)
    M, n, k = 40, 128, 128
    ints = lambda *s: rng.integers(-1, 2, s).astype(np.float32)  # noqa: E731
    x, dy, w = ints(M, k), ints(M, n), ints(k, n)
    # anchors: column 0 of x and of dy, row 0 of w's contraction, keep every scale at one
    x[:, 0] = dy[:, 0] = 448
    w[0], w[:, 0] = 0, 0
    one = np.float32(448) * np.float32(1 / 448)
    assert one == 1
    codes = torch.from_numpy(np.ascontiguousarray(w.T)).to(torch.float8_e4m3fn).view(torch.uint8)

    def lin_of(c):
        return m.F8Linear.pack(m.F8Shape(1, n, k), c[None].cuda(), torch.ones((1, 1, 1), device="cuda"))

    def y_of(xv, c):
        return f64(lin_of(c)(torch.from_numpy(xv).to(BF).cuda()))
    y = y_of(x, codes)
    dx = f64(lin_of(codes).transposed()(torch.from_numpy(dy).to(BF).cuda()))
    d = ints(M, k)
    d[:, 0] = 0
    assert np.sum(dy[:, 1:] * (y_of(x + d, codes) - y)[:, 1:]) == np.sum(dx[:, 1:] * d[:, 1:])
    # W: its gradient's blocks run down the 40 rows; a row of 448 keeps their scales at one
    x2, dy2 = ints(M, k), ints(M, n)
    x2[0], dy2[0] = 448, 0
    x2[1], dy2[1] = 0, 448
    dw = f64(lin_of(codes).weight_gradient(torch.from_numpy(x2).to(BF).cuda(),
                                          torch.from_numpy(dy2).to(BF).cuda()))[0]
    assert np.array_equal(dw, x2.astype(np.float64).T @ dy2)
    dwd = ints(k, n)
    dwd[0], dwd[:, 0] = 0, 0
    w2 = w + dwd
    x2[0, 1:], x2[1, 1:] = 0, 0
    x2[:, 0] = 448
    c2 = torch.from_numpy(np.ascontiguousarray(w2.T)).to(torch.float8_e4m3fn).view(torch.uint8)
    diff = y_of(x2, c2) - y_of(x2, codes)
    assert np.sum(dy2 * diff) == np.sum((x2.astype(np.float64).T @ dy2) * dwd)


# ------------------------------------------------------------------ as they are used

@pytest.mark.parametrize("M,n", [(300, 140), (9000, 300)])
def test_captured_and_replayed_on_another_stream(M, n):
    """Forward, data and weight gradient captured into one graph on a side stream,
    replayed with new inputs and offsets, bitwise equal to eager calls."""
    rng = np.random.default_rng(11)
    groups, k = 3, 200
    lin, _ = make(rng, groups, n, k)
    turned = lin.transposed()
    x, dy = rows(rng, M, k).cuda(), rows(rng, M, n).cuda()
    off = offsets([0, 20, 250, M])
    y, dx = torch.zeros_like(dy), torch.zeros_like(x)
    dw = torch.zeros((groups, k, n), dtype=BF, device="cuda")
    few = torch.zeros((groups, n), dtype=BF, device="cuda")
    few_off = offsets([0, 1, 1, 3])

    def step(y, dx, dw, few):
        lin(x, off, out=y)
        turned(dy, off, out=dx)
        lin.weight_gradient(x, dy, off, out=dw)
        lin(x[:groups], few_off, out=few)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(y, dx, dw, few)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(y, dx, dw, few)
    for seed in range(4):
        rng = np.random.default_rng(seed)
        x.copy_(rows(rng, M, k))
        dy.copy_(rows(rng, M, n))
        off.copy_(torch.from_numpy(np.sort(rng.integers(0, M + 1, groups + 1)).astype(np.int32)))
        outs = (y, dx, dw, few)
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = [torch.zeros_like(o) for o in outs]
        step(*want)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_products_at_once_on_three_streams():
    rng = np.random.default_rng(12)
    lin, _ = make(rng, 1, 300, 500)
    xs = [rows(rng, M, 500).cuda() for M in (4, 90, 600, 9000)]
    want = [(lin(x), lin.weight_gradient(x, x[:, :300])) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(10):
        got = []
        for s, x in zip(streams, xs):
            with torch.cuda.stream(s):
                got.append((lin(x), lin.weight_gradient(x, x[:, :300])))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))


def test_sorted_rows_train_step():
    """The operators together: rows sorted by expert, product, weighted return, and
    back: the return's gradient, data and weight gradient, the sort's gradient, and the
    clipped weight gradient -- against the same in 64 bits, to the bounds of each
    rounding."""
    rng = np.random.default_rng(13)
    T, E, k, H, n = 60, 5, 2, 200, 130
    lin, w = make(rng, E, n, H)
    x = rows(rng, T, H)
    idx = rng.integers(0, E + 1, (T, k)).astype(np.int32)         # expert E: elsewhere
    wt = rng.random((T, k)).astype(np.float32)
    op = m.TokenSort(m.SortShape(T, E, k, H, align=16))
    back = m.TokenSort(m.SortShape(T, E, k, n, align=16))
    idx_d, wt_d = torch.from_numpy(idx).cuda(), torch.from_numpy(wt).cuda()
    xs = op.sort(x.cuda(), idx_d, out=op.sorted_rows().zero_())
    back.sort(torch.zeros((T, n), dtype=BF, device="cuda"), idx_d)
    y = lin(xs, op.offsets)
    out = back.unsort(y, wt_d)
    perm = op.perm.cpu().numpy()
    off = op.offsets.cpu().numpy()
    live = np.nonzero(perm[:off[-1]] >= 0)[0]
    for g in range(E):
        at = [r for r in live if off[g] <= r < off[g + 1]]
        if at:
            check(f"expert {g}", y[at], x[perm[at] // k], w[g], BF)
    want = np.zeros((T, n))
    np.add.at(want, perm[live] // k, wt.reshape(-1)[perm[live]][:, None] * f64(y)[live])
    size = np.zeros((T, n))
    np.add.at(size, perm[live] // k, wt.reshape(-1)[perm[live]][:, None] * np.abs(f64(y)[live]))
    within("return", out, want, size * 8 * fo.ULP + np.abs(want) * 2.0 ** -8 + 2.0 ** -133)
    dout = rows(rng, T, n).cuda()
    dy, _ = back.unsort_backward(dout, y, wt_d, dy=back.sorted_rows().zero_())
    dxs = lin.transposed()(dy, op.offsets)
    dx = op.sort_backward(dxs)
    want = np.zeros((T, H))
    np.add.at(want, perm[live] // k, f64(dxs)[live])
    size = np.zeros((T, H))
    np.add.at(size, perm[live] // k, np.abs(f64(dxs)[live]))
    within("dx", dx, want, size * 8 * fo.ULP + np.abs(want) * 2.0 ** -8 + 2.0 ** -133)
    dw = lin.weight_gradient(xs, dy, op.offsets)
    xh, dh = xs.float().cpu().numpy(), dy.float().cpu().numpy()
    for g in range(E):
        span = slice(off[g], off[g + 1])
        d, bound = fo.weight_gradient(xh[span], dh[span])
        within(f"dw {g}", dw[g], d, fo.rounded(d, bound, BF))
    clip = m.GradClip(m.GradSet([dw]))
    before = f64(dw)
    norm = clip(1.0)
    true = np.sqrt((before ** 2).sum())
    assert abs(float(norm) - true) <= true * 2.0 ** -22
    within("clipped", dw, before / (true + 1e-6), np.abs(before) / true * (2.0 ** -8 + 2.0 ** -22) + 2.0 ** -133)
