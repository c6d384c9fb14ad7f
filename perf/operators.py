"""Cases of the expert-sorted rows (sort, unsort and their gradients) and of
the 4-bit few-token products, each in a plain form of elementary torch
operations and as calls of libmoe.

Rows: f = t*k + j is the flat (token, slot) index.  A slot takes a row if its
expert id lies in [first, first + held): the experts of this GPU; the others
(experts elsewhere, padded tokens with id -1) take none.  The rows of one
expert are consecutive, in ascending f, and start at a multiple of `align`.

4-bit weights: codes [groups][n][k/2] (even k in the low nibble).  mxfp4: E2M1
values times 2^(scale - 127), one scale per 32 along k.  int4: scale * (code -
zero), one bf16 or fp16 scale (and zero point) per `group` along k.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ------------------------------------------------------------------ the cases

def _rows(name, op, T, k, E, held, D, type="bf16", align=1, pad=0, blank=0.0, skew=0.0, add=False):
    return dict(name=name, op=op, T=T, k=k, E=E, held=held, D=D, type=type, align=align, pad=pad,
                blank=blank, skew=skew, add=add)


def _linear(name, M, groups, n, k, fmt, group, zeros=False, scale="bf16"):
    return dict(name=name, op="w4_linear", M=M, groups=groups, n=n, k=k, fmt=fmt, group=group,
                zeros=zeros, scale=scale)


def _decode(name, T, k, E, held, H, I, fmt, group, zeros=False, scale="bf16"):
    return dict(name=name, op="w4_decode", T=T, k=k, E=E, held=held, H=H, I=I, fmt=fmt, group=group,
                zeros=zeros, scale=scale)


def listed():
    return [
        # one decoded token's rows gathered for 8 of 256 experts: latency alone
        _rows("sort-one-token", "sort", 1, 8, 256, 256, 7168),
        # one GPU's eighth of the experts, segments padded to 128-row tiles, a padded batch
        _rows("sort-share-aligned", "sort", 8192, 8, 256, 32, 7168, align=128, blank=0.03),
        # a whole training batch over every expert: the largest copy
        _rows("sort-all-experts", "sort", 8192, 8, 256, 256, 7168, skew=0.5),
        # the gradient of the sort at a small layer's size
        _rows("sort-grad-mid", "sort_bwd", 4096, 6, 64, 64, 2048),
        # weighted return with a shared expert's rows added, routed rows skewed over few experts
        _rows("unsort-few-experts", "unsort", 2048, 8, 6, 6, 7168, skew=1.0, add=True),
        # a ragged width in fp32, strided token rows, half of the slots elsewhere
        _rows("unsort-f32-ragged", "unsort", 1531, 7, 60, 30, 1111, type="f32", pad=5, blank=0.1),
        # the gradient of the weighted return, rows and weights
        _rows("unsort-grad", "unsort_bwd", 2048, 8, 6, 6, 7168, skew=1.0),
        # the same in fp16 at an odd batch with padded segments and strided token rows
        _rows("unsort-grad-f16", "unsort_bwd", 777, 3, 48, 16, 1000, type="f16", align=16, pad=24),
        # one token through one projection: the smallest product
        _linear("w4-one-row", 1, 1, 2048, 7168, "mxfp4", 32),
        # a few sorted rows over ragged groups, odd output width, zero points
        _linear("w4-grouped-int4", 45, 16, 1001, 2048, "int4", 128, zeros=True),
        # one decoded token through the experts of a layer
        _decode("w4-decode-token", 1, 8, 48, 48, 7168, 2048, "mxfp4", 32),
        # a decode batch on one GPU's half of the experts
        _decode("w4-decode-batch", 32, 6, 64, 32, 2048, 1408, "int4", 64, scale="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sort", "sort_bwd", "unsort", "unsort_bwd", "w4_linear", "w4_decode"])
    fmt = rng.choice(["mxfp4", "int4"])
    group = 32 if fmt == "mxfp4" else rng.choice([32, 64, 128])
    zeros = fmt == "int4" and rng.random() < 0.5
    scale = rng.choice(["bf16", "f16"]) if fmt == "int4" else "bf16"
    if op == "w4_linear":
        groups = rng.choice([1, 1, _log(rng, 2, 32)])
        k = group * max(1, _log(rng, 64, 8192) // group)
        n = _log(rng, 16, 8192)
        while groups * n * k > 1 << 28:
            n = max(16, n // 2)
        return _linear(None, _log(rng, 1, 96), groups, n, k, fmt, group, zeros, scale)
    if op == "w4_decode":
        E = _log(rng, 2, 64)
        H, I = 128 * _log(rng, 2, 56), 128 * _log(rng, 1, 16)
        k = rng.randint(1, min(8, E))
        while E * H * I > 1 << 29:
            H, I = max(256, H // 256 * 128), max(128, I // 256 * 128)
        return _decode(None, _log(rng, 1, 48), k, E, rng.choice([E, E, max(1, E // 2)]), H, I, fmt,
                       group, zeros, scale)
    E, D = _log(rng, 2, 512), _log(rng, 64, 8192)
    k = rng.randint(1, min(8, E))
    T = _log(rng, 1, 8192)
    while T * k * D > 1 << 28:
        T //= 2
    D = D if rng.random() < 0.3 else max(8, D // 8 * 8)
    return _rows(None, op, T, k, E, rng.choice([E, E, max(1, E // 4)]), D,
                 rng.choice(["bf16", "bf16", "f16", "f32"]), rng.choice([1, 1, 16, 128]),
                 rng.choice([0, 0, 8, 3]), rng.choice([0.0, 0.0, 0.1]), rng.choice([0.0, 0.0, 0.7]),
                 op == "unsort" and rng.random() < 0.5)


# ------------------------------------------------------------------ inputs

def _routing(g, T, k, E, skew, blank):
    """idx [T][k] int32 and its softmax weights: k distinct experts (k > E: independent draws), the
    first ones favoured by `skew`; the last `blank` share of the tokens is padding (-1)."""
    logp = -skew * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
    if k <= E:
        u = torch.rand((T, E), generator=g, device=DEV).clamp_(1e-9, 1 - 1e-7)
        idx = torch.topk(logp - torch.log(-torch.log(u)), k, dim=1).indices
    else:
        idx = torch.multinomial(logp.exp().expand(T, E), k, replacement=True, generator=g)
    idx = idx.to(torch.int32)
    if int(T * blank):
        idx[T - int(T * blank):] = -1
    w = torch.softmax(torch.randn((T, k), generator=g, device=DEV), dim=1)
    return idx.contiguous(), w.contiguous()


def _first(c):
    return (c["E"] - c["held"]) // 2


def _capacity(c):
    R = c["T"] * c["k"]
    return R + (min(c["held"], R) * (c["align"] - 1) if c["align"] > 1 else 0)


def _plan(idx, first, held, align, capacity):
    """counts, offsets, perm, inv of a routing (plain form, no host synchronisation)."""
    R = idx.numel()
    e = idx.reshape(-1).long() - first
    e = torch.where((e >= 0) & (e < held), e, held)
    key, order = e.sort(stable=True)
    bounds = torch.searchsorted(key, torch.arange(held + 1, device=DEV))  # first place of each expert's slots
    counts = bounds[1:] - bounds[:-1]
    padded = (counts + align - 1) // align * align
    offsets = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    f = torch.arange(R, device=DEV)
    place = torch.where(key < held, offsets[key] + f - bounds[key], -1)
    inv = torch.empty_like(place)
    inv[order] = place
    perm = torch.full((capacity + 1,), -1, dtype=torch.int32, device=DEV)
    perm[torch.where(place >= 0, place, capacity)] = order.to(torch.int32)
    return (counts.to(torch.int32), offsets.to(torch.int32), perm[:capacity],
            inv.to(torch.int32).reshape(idx.shape))


def _randn(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _strided(g, T, D, pad, dtype):
    return _randn(g, (T, D + pad), dtype)[:, :D]


def _quantised(g, groups, n, k, fmt, group, zeros, scale):
    """4-bit weights of random matrices [groups][n][k] of standard deviation 1/sqrt(k)."""
    codes = torch.empty((groups, n, k // 2), dtype=torch.uint8, device=DEV)
    sdt = torch.uint8 if fmt == "mxfp4" else TYPES[scale]
    scales = torch.empty((groups, n, k // group), dtype=sdt, device=DEV)
    zp = torch.empty((groups, n, k // group), dtype=torch.uint8, device=DEV) if zeros else None
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    for e in range(groups):
        w = (torch.randn((n, k // group, group), generator=g, device=DEV) / math.sqrt(k))
        if fmt == "mxfp4":
            s = torch.floor(torch.log2(w.abs().amax(-1).clamp(min=1e-30))) - 2
            q = torch.bucketize(w.abs() * torch.exp2(-s)[..., None], edges) + 8 * (w < 0)
            scales[e] = (s + 127).to(torch.uint8)
        elif zeros:
            lo, hi = w.amin(-1).clamp(max=0), w.amax(-1).clamp(min=0)
            s = ((hi - lo) / 15).clamp(min=1e-6).to(sdt)
            z = torch.round(-lo / s.float()).clamp(0, 15)
            q = (torch.round(w / s.float()[..., None]) + z[..., None]).clamp(0, 15)
            scales[e], zp[e] = s, z.to(torch.uint8)
        else:
            s = (w.abs().amax(-1) / 7).clamp(min=1e-6).to(sdt)
            q = (torch.round(w / s.float()[..., None]) + 8).clamp(0, 15)
            scales[e] = s
        q = q.to(torch.uint8).reshape(n, k)
        codes[e] = q[:, 0::2] | (q[:, 1::2] << 4)
    return {"codes": codes, "scales": scales, "zeros": zp, "fmt": fmt, "group": group, "n": n, "k": k,
            "groups": groups, "scale": scale}


def _inputs(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {}
    if c["op"] == "w4_linear":
        s["x"] = _randn(g, (c["M"], c["k"]), torch.bfloat16)
        s["w"] = _quantised(g, c["groups"], c["n"], c["k"], c["fmt"], c["group"], c["zeros"], c["scale"])
        cut = torch.rand(c["groups"] - 1, generator=g, device=DEV)
        cut = (cut * (c["M"] + 1)).long().clamp(max=c["M"]).sort().values
        s["offsets"] = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), c["M"])]).to(torch.int32)
        return s
    dtype = TYPES[c.get("type", "bf16")]
    s["idx"], s["wt"] = _routing(g, c["T"], c["k"], c["E"], c.get("skew", 0.0), c.get("blank", 0.0))
    if c["op"] == "w4_decode":
        s["x"] = _randn(g, (c["T"], c["H"]), dtype)
        q = (c["fmt"], c["group"], c["zeros"], c["scale"])
        s["gate"] = _quantised(g, c["held"], c["I"], c["H"], *q)
        s["up"] = _quantised(g, c["held"], c["I"], c["H"], *q)
        s["down"] = _quantised(g, c["held"], c["H"], c["I"], *q)
        return s
    T, D, cap = c["T"], c["D"], _capacity(c)
    if c["op"] == "sort":
        s["x"] = _strided(g, T, D, c["pad"], dtype)
        return s
    s["counts"], s["offsets"], s["perm"], s["inv"] = _plan(s["idx"], _first(c), c["held"], c["align"], cap)
    # the experts' rows: values in every row that holds a token, zeros in the rest
    rows = _randn(g, (cap, D), dtype)
    rows[s["perm"] < 0] = 0
    s["rows"] = rows
    if c["op"] == "unsort":
        s["add"] = _strided(g, T, D, c["pad"], dtype) if c["add"] else None
    if c["op"] == "unsort_bwd":
        s["dout"] = _strided(g, T, D, c["pad"], dtype)
    return s


def prepare(case, seed):
    c, s = case, _inputs(case, seed)
    s["case"] = c
    if not own:
        return s
    import mixture_experts_layer_offsets_amd as m
    i32 = dict(dtype=torch.int32, device=DEV)

    def packed(q):
        shape = m.W4Shape(q["groups"], q["n"], q["k"],
                          m.MOE_W4_MXFP4 if q["fmt"] == "mxfp4" else m.MOE_W4_INT4, q["group"],
                          m.MOE_SCALE_F16 if q["scale"] == "f16" else m.MOE_SCALE_BF16,
                          int(q["zeros"] is not None))
        buf = torch.empty(m.moe_w4_bytes(shape), dtype=torch.uint8, device=DEV)
        m.moe_w4_pack(shape, q["codes"], q["scales"], q["zeros"], buf)
        return shape, buf

    if c["op"] == "w4_linear":
        s["shape"], s["packed"] = packed(s.pop("w"))
        s["out"] = torch.empty((c["M"], c["n"]), dtype=torch.bfloat16, device=DEV)
        return s
    if c["op"] == "w4_decode":
        s["shape"] = m.Shape(c["T"], c["H"], c["held"], c["k"], c["I"])
        (w4, gate), (_, up), (_, down) = packed(s.pop("gate")), packed(s.pop("up")), packed(s.pop("down"))
        s["experts"] = m.W4Experts(gate, up, down, format=w4.format, group_size=w4.group_size,
                                   scale_type=w4.scale_type, zeros=w4.zeros, first_expert=_first(c))
        s["ws"] = torch.empty(m.moe_w4_decode_workspace_bytes(s["shape"]), dtype=torch.uint8, device=DEV)
        s["out"] = torch.empty((c["T"], c["H"]), dtype=torch.bfloat16, device=DEV)
        return s
    T, D, cap, dtype = c["T"], c["D"], _capacity(c), TYPES[c["type"]]
    s["shape"] = m.SortShape(T, c["held"], c["k"], D,
                             {"bf16": m.MOE_ROW_BF16, "f16": m.MOE_ROW_F16, "f32": m.MOE_ROW_F32}[c["type"]],
                             align=c["align"], first_expert=_first(c), token_stride=D + c["pad"])
    if c["op"] == "sort":
        s["plan"] = (torch.empty(c["held"], **i32), torch.empty(c["held"] + 1, **i32), torch.empty(cap, **i32),
                     torch.empty((T, c["k"]), **i32))
        s["sorted"] = torch.zeros((cap, D), dtype=dtype, device=DEV)
        s["ws"] = torch.empty(m.moe_sort_workspace_bytes(s["shape"]), dtype=torch.uint8, device=DEV)
    if c["op"] in ("sort_bwd", "unsort"):
        s["out"] = torch.empty((T, D + c["pad"]), dtype=dtype, device=DEV)[:, :D]
    if c["op"] == "unsort_bwd":
        s["dy"] = torch.zeros((cap, D), dtype=dtype, device=DEV)
        s["dw"] = torch.empty((T, c["k"]), dtype=torch.float32, device=DEV)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return (_own if own else _plain)(s)


def _own(s):
    import mixture_experts_layer_offsets_amd as m
    op, shape = s["case"]["op"], s["shape"]
    if op == "sort":
        m.moe_sort_fwd(shape, s["x"], s["idx"], *s["plan"], s["sorted"], s["ws"])
        return (*s["plan"], s["sorted"])
    if op == "sort_bwd":
        m.moe_sort_bwd(shape, s["rows"], s["inv"], s["out"])
        return s["out"]
    if op == "unsort":
        m.moe_unsort_fwd(shape, s["rows"], s["wt"], s["inv"], s["add"], s["out"])
        return s["out"]
    if op == "unsort_bwd":
        m.moe_unsort_bwd(shape, s["dout"], s["rows"], s["wt"], s["counts"], s["offsets"], s["inv"],
                         s["dy"], s["dw"])
        return s["dy"], s["dw"]
    if op == "w4_linear":
        m.moe_w4_linear(shape, s["x"], s["offsets"], s["packed"], s["out"])
        return s["out"]
    m.moe_w4_decode_fwd(shape, s["experts"], s["x"], None, None, s["idx"], s["wt"], s["out"], s["ws"])
    return s["out"]


def _values(q, sel=None):
    """fp32 values [.., n, k] of 4-bit weights, all groups or the selected ones."""
    codes, scales, zeros = q["codes"], q["scales"], q["zeros"]
    if sel is not None:
        codes, scales, zeros = codes[sel], scales[sel], None if zeros is None else zeros[sel]
    nib = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1, q["group"])
    if q["fmt"] == "mxfp4":
        v = torch.tensor(E2M1, device=DEV)[nib.int()] * torch.exp2(scales.float() - 127)[..., None]
    else:
        v = nib.float() - (8.0 if zeros is None else zeros.float()[..., None])
        v = v * scales.float()[..., None]
    return v.flatten(-2)


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "sort":
        counts, offsets, perm, inv = _plan(s["idx"], _first(c), c["held"], c["align"], _capacity(c))
        rows = s["x"][perm.clamp(min=0).long() // c["k"]]
        return counts, offsets, perm, inv, torch.where(perm[:, None] >= 0, rows, 0)
    if op in ("sort_bwd", "unsort"):
        kept = s["inv"] >= 0
        rows = s["rows"][s["inv"].clamp(min=0).long()].float()
        rows = torch.where(kept[..., None], rows, 0.0)
        if op == "unsort":
            rows = rows * s["wt"][..., None]
        out = rows.sum(1)
        if op == "unsort" and s["add"] is not None:
            out = out + s["add"].float()
        return out.to(s["rows"].dtype)
    if op == "unsort_bwd":
        f = s["perm"].clamp(min=0).long()
        d = s["dout"][f // c["k"]].float()
        held = s["perm"] >= 0
        dy = torch.where(held[:, None], d * s["wt"].reshape(-1)[f][:, None], 0.0)
        dot = (d * s["rows"].float()).sum(1)
        dw = torch.where(s["inv"] >= 0, dot[s["inv"].clamp(min=0).long()], 0.0)
        return dy.to(s["rows"].dtype), dw
    if op == "w4_linear":
        r = torch.arange(c["M"], device=DEV)
        grp = (r[:, None] >= s["offsets"][None, 1:]).sum(1)
        y = torch.matmul(_values(s["w"]), s["x"].float().t())  # [groups][n][M]
        return y[grp, :, r].to(torch.bfloat16)
    # w4_decode: with fewer slots than experts the slots' own matrices, else every expert on every token
    e = s["idx"].reshape(-1).long() - _first(c)
    kept = (e >= 0) & (e < c["held"])
    e = e.clamp(0, c["held"] - 1)
    x = s["x"].float()
    t = torch.arange(e.numel(), device=DEV) // c["k"]
    if e.numel() < c["held"]:
        xs = x[t][..., None]
        g, u = torch.matmul(_values(s["gate"], e), xs), torch.matmul(_values(s["up"], e), xs)
        y = torch.matmul(_values(s["down"], e), g / (1 + torch.exp(-g)) * u)[..., 0]
    else:
        g, u = torch.matmul(_values(s["gate"]), x.t()), torch.matmul(_values(s["up"]), x.t())
        y = torch.matmul(_values(s["down"]), g / (1 + torch.exp(-g)) * u)[e, :, t]
    w = torch.where(kept, s["wt"].reshape(-1), 0.0)
    return (y * w[:, None]).reshape(c["T"], c["k"], -1).sum(1).to(torch.bfloat16)


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    c, s = case, _inputs(case, seed)
    op = c["op"]

    def dense(q, e):
        """Matrix e of a 4-bit weight as doubles [n][k], code by code."""
        code = q["codes"][e].to(torch.int64)
        out = torch.empty((q["n"], q["k"]), dtype=torch.float64, device=DEV)
        sc = q["scales"][e].double().repeat_interleave(q["group"], dim=1)
        if q["fmt"] == "mxfp4":
            table = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
            out[:, 0::2], out[:, 1::2] = table[code % 16], table[code // 16]
            return out * torch.pow(torch.tensor(2.0, dtype=torch.float64, device=DEV), sc - 127)
        out[:, 0::2], out[:, 1::2] = (code % 16).double(), (code // 16).double()
        z = 8.0 if q["zeros"] is None else q["zeros"][e].double().repeat_interleave(q["group"], dim=1)
        return (out - z) * sc

    if op == "w4_linear":
        at = s["offsets"].tolist()
        x = s["x"].double()
        parts = [x[at[e]:at[e + 1]] @ dense(s["w"], e).T for e in range(c["groups"])]
        return torch.cat(parts)
    ids = s["idx"].tolist()
    T, k, lo = c["T"], c["k"], _first(c)
    if op == "w4_decode":
        out = torch.zeros((T, c["H"]), dtype=torch.float64, device=DEV)
        for e in range(c["held"]):
            at = [(t, j) for t in range(T) for j in range(k) if ids[t][j] == lo + e]
            if not at:
                continue
            t = torch.tensor([a[0] for a in at], device=DEV)
            w = torch.stack([s["wt"][a] for a in at]).double()
            x = s["x"][t].double()
            g, u = x @ dense(s["gate"], e).T, x @ dense(s["up"], e).T
            out.index_add_(0, t, w[:, None] * ((g * torch.sigmoid(g) * u) @ dense(s["down"], e).T))
        return out
    # the layout by its definition: experts in turn, their slots in ascending order
    slots = [[] for _ in range(c["held"])]
    for f, e in enumerate(x for row in ids for x in row):
        if lo <= e < lo + c["held"]:
            slots[e - lo].append(f)
    perm, inv, offsets = [], [-1] * (T * k), [0]
    for rows in slots:
        for f in rows:
            inv[f] = len(perm)
            perm.append(f)
        perm += [-1] * (-len(rows) % c["align"])
        offsets.append(len(perm))
    perm += [-1] * (_capacity(c) - len(perm))
    perm_t, inv_t = torch.tensor(perm, device=DEV), torch.tensor(inv, device=DEV)
    live = (perm_t >= 0).nonzero()[:, 0]
    token = perm_t[live] // k
    if op == "sort":
        rows = torch.zeros((_capacity(c), c["D"]), dtype=torch.float64, device=DEV)
        rows[live] = s["x"].double()[token]
        ints = [torch.tensor([len(r) for r in slots], device=DEV), torch.tensor(offsets, device=DEV), perm_t,
                inv_t.reshape(T, k)]
        return (*[v.to(torch.int32) for v in ints], rows)
    rows = s["rows"].double()
    if op in ("sort_bwd", "unsort"):
        w = s["wt"].double() if op == "unsort" else torch.ones((T, k), dtype=torch.float64, device=DEV)
        out = torch.zeros((T, c["D"]), dtype=torch.float64, device=DEV)
        out.index_add_(0, token, rows[live] * w.reshape(-1)[perm_t[live]][:, None])
        return out if op == "sort_bwd" or s["add"] is None else out + s["add"].double()
    d = s["dout"].double()[token]
    dy = torch.zeros_like(rows)
    dy[live] = d * s["wt"].double().reshape(-1)[perm_t[live]][:, None]
    dw = torch.zeros(T * k, dtype=torch.float64, device=DEV)
    dw[perm_t[live]] = (d * rows[live]).sum(1)
    return dy, dw.reshape(T, k)


# ------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"].startswith("w4"):
        per = 4 + (8 if c["fmt"] == "mxfp4" else 16 + (4 if c["zeros"] else 0)) / c["group"]  # bits a weight
        if c["op"] == "w4_linear":
            # the groups that hold a row, at random cuts
            used = c["groups"] * (1 - (1 - 1 / c["groups"]) ** c["M"]) if c["groups"] > 1 else 1
            return {"bytes": used * c["n"] * c["k"] * per / 8 + 2 * c["M"] * (c["n"] + c["k"]),
                    "flops": 2 * c["M"] * c["n"] * c["k"]}
        used = c["held"] * (1 - (1 - c["k"] / c["E"]) ** c["T"])
        rows = c["T"] * c["k"] * c["held"] / c["E"]
        return {"bytes": used * 3 * c["H"] * c["I"] * per / 8 + 4 * c["T"] * c["H"] + 8 * c["T"] * c["k"],
                "flops": 6 * rows * c["H"] * c["I"]}
    size = TYPES[c["type"]].itemsize
    T, k, D = c["T"], c["k"], c["D"]
    share = c["held"] / c["E"] * (1 - c["blank"])
    kept = T * k * share
    hit = T * (1 - c["blank"]) * (1 - (1 - c["held"] / c["E"]) ** k) if c["held"] < c["E"] else T * (1 - c["blank"])
    pads = c["held"] * (c["align"] - 1) / 2 if kept > c["held"] else 0
    idx = 4 * T * k
    if c["op"] == "sort":
        return {"bytes": (hit + kept + pads) * D * size + 2 * idx + 4 * _capacity(c) + 8 * c["held"], "flops": 0}
    if c["op"] == "sort_bwd":
        return {"bytes": (kept + T) * D * size + idx, "flops": kept * D}
    if c["op"] == "unsort":
        return {"bytes": (kept + T * (2 if c["add"] else 1)) * D * size + 2 * idx, "flops": 2 * kept * D}
    return {"bytes": (hit + 2 * kept + pads) * D * size + 3 * idx, "flops": 3 * kept * D}
