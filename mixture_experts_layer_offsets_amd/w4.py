"""4-bit expert weights: packed matrices, their products, the few-token layer."""
from __future__ import annotations

import torch

from . import _lib
from ._lib import Shape, W4Shape

_SCALE_DTYPE = {_lib.MOE_SCALE_BF16: torch.bfloat16, _lib.MOE_SCALE_F16: torch.float16}
_BF16 = (torch.bfloat16, torch.int16)


def _check(name, t, shape, dtypes, device=None, rows=False):
    """ValueError unless t has this shape and type on the device, contiguous
    (or, with `rows`, rows of contiguous values at least their length apart)."""
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: {t.dtype}, expected {dtypes[0]}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if rows:
        ok = t.numel() == 0 or ((t.shape[1] == 1 or t.stride(1) == 1) and
                                (t.shape[0] == 1 or t.stride(0) >= t.shape[1]))
    else:
        ok = t.is_contiguous()
    if not ok:
        raise ValueError(f"{name}: strides {t.stride()} are not those of plain rows")


def places(tensors):
    """Where each tensor (or None) lies, and how many values are there."""
    return [None if t is None else (t.data_ptr(), t.numel()) for t in tensors]


def check_places(tensors, at):
    if places(tensors) != at:
        raise ValueError("experts: a matrix was given other memory since")


def decode_args(s, dev, x, w_router, bias, topk_idx, topk_w, out):
    """The checked arguments of a few-token layer's call; its ``out``."""
    slots, tokens = (s.tokens, s.top_k), (s.tokens, s.hidden)
    _check("x", x, tokens, _BF16, dev)
    for name, t, shape, dtypes in (("w_router", w_router, (s.hidden, s.experts), _BF16),
                                   ("bias", bias, (s.experts,), (torch.float32,)),
                                   ("topk_idx", topk_idx, slots, (torch.int32,)),
                                   ("topk_w", topk_w, slots, (torch.float32,))):
        if t is not None:
            _check(name, t, shape, dtypes, dev)
    if out is None:
        out = torch.empty(tokens, dtype=x.dtype, device=dev)
    _check("out", out, tokens, _BF16, dev)
    return out


class W4Linear:
    """Packed 4-bit matrices [groups][k][n] and their products with few rows.

    ``W4Linear.quantize`` takes bf16 weights [groups][k][n] (products x*W),
    ``W4Linear.pack`` ready-made codes, scales and zero points; weights that are
    packed already come as a uint8 tensor of moe_w4_bytes (checked in every call).
    Calls enqueue on the current stream.
    """

    def __init__(self, shape: W4Shape, packed: torch.Tensor):
        self.shape, self.packed = shape, packed
        self._need = None, 0  # a shape and its bytes

    def _weights(self):
        """The packed tensor: the kernels read all that the shape says of it.  Looked at in
        every call: it, its memory or the shape may have been exchanged."""
        if self._need[0] is not self.shape:
            self._need = self.shape, self._bytes(self.shape)
        _check("packed", self.packed, (self._need[1],), (torch.uint8,))
        return self.packed

    @staticmethod
    def _bytes(shape):
        n = _lib.moe_w4_bytes(shape)
        if n == 0:
            raise ValueError(f"shape outside the limits of moe_w4_shape: {shape}")
        return n

    @classmethod
    def _buffer(cls, shape, device):
        return torch.empty(cls._bytes(shape), dtype=torch.uint8, device=device)

    @classmethod
    def quantize(cls, w, format=_lib.MOE_W4_MXFP4, group_size=32, scale_type=_lib.MOE_SCALE_BF16,
                 zeros=0):
        if w.dim() != 3:
            raise ValueError(f"w: {w.dim()} dimensions, expected [groups][k][n]")
        shape = W4Shape(w.shape[0], w.shape[2], w.shape[1], format, group_size, scale_type, zeros)
        packed = cls._buffer(shape, w.device)
        _check("w", w, w.shape, _BF16)
        with torch.cuda.device(w.device):
            _lib.moe_w4_quantize(shape, w, packed)
        return cls(shape, packed)

    @classmethod
    def pack(cls, shape: W4Shape, codes, scales, zeros=None):
        packed = cls._buffer(shape, codes.device)
        per = (shape.groups, shape.n, shape.k // shape.group_size)
        _check("codes", codes, (shape.groups, shape.n, shape.k // 2), (torch.uint8,))
        sdt = torch.uint8 if shape.format == _lib.MOE_W4_MXFP4 else _SCALE_DTYPE[shape.scale_type]
        _check("scales", scales, per, (sdt,), codes.device)
        if (zeros is not None) != bool(shape.zeros):
            raise ValueError("zeros: given exactly when the shape has zero points")
        if zeros is not None:
            _check("zeros", zeros, per, (torch.uint8,), codes.device)
        with torch.cuda.device(codes.device):
            _lib.moe_w4_pack(shape, codes, scales, zeros, packed)
        return cls(shape, packed)

    def values(self):
        """The weights [groups][k][n] that the codes stand for, in fp32."""
        s, packed = self.shape, self._weights()
        w = torch.empty((s.groups, s.k, s.n), dtype=torch.float32, device=packed.device)
        with torch.cuda.device(packed.device):
            _lib.moe_w4_unpack(s, packed, w)
        return w

    def __call__(self, x, offsets=None, out=None):
        """x [rows][k] bf16 -> [rows][n] bf16; with ``offsets`` [groups + 1]
        int32 the rows of group g are [offsets[g], offsets[g + 1]), and rows
        in no group are left as they are (zeros in a new ``out``)."""
        s, packed = self.shape, self._weights()
        dev = packed.device
        if x.dim() != 2:
            raise ValueError(f"x: {x.dim()} dimensions, expected [rows][k]")
        _check("x", x, (x.shape[0], s.k), _BF16, dev, rows=True)
        if offsets is None and s.groups != 1:
            raise ValueError("offsets: needed with more than one group")
        if offsets is not None:
            _check("offsets", offsets, (s.groups + 1,), (torch.int32,), dev)
        if out is None:
            make = torch.empty if offsets is None else torch.zeros
            out = make((x.shape[0], s.n), dtype=x.dtype, device=dev)
        _check("out", out, (x.shape[0], s.n), _BF16, dev, rows=True)
        with torch.cuda.device(dev):
            _lib.moe_w4_linear(s, x, offsets, packed, out)
        return out


class W4Experts:
    """moe_w4_experts: the packed matrices of a layer's experts (gate, up
    [E][H][I], down [E][I][H]; the shared expert's with one group), uint8
    tensors as moe_w4_pack and moe_w4_quantize leave them, kept alive here.  A tensor that
    is given other memory afterwards (``t.data = ...``) ends them: calls raise ValueError."""

    def __init__(self, gate, up, down, shared_gate=None, shared_up=None, shared_down=None, *,
                 format=_lib.MOE_W4_MXFP4, group_size=32, scale_type=_lib.MOE_SCALE_BF16, zeros=0,
                 first_expert=0):
        self.tensors = (gate, up, down, shared_gate, shared_up, shared_down)
        self.shapes = None  # of the matrices, where they are known
        self._at = places(self.tensors)
        self._c = _lib.MoeW4Experts(format, group_size, scale_type, zeros, first_expert,
                                    *(a and a[0] for a in self._at))

    @classmethod
    def of(cls, gate: W4Linear, up: W4Linear, down: W4Linear, shared_gate=None, shared_up=None,
           shared_down=None, first_expert=0):
        """From W4Linear matrices of one format."""
        all_ = [m for m in (gate, up, down, shared_gate, shared_up, shared_down) if m is not None]
        kinds = {(m.shape.format, m.shape.group_size, m.shape.scale_type, m.shape.zeros)
                 for m in all_}
        if len(kinds) != 1:
            raise ValueError(f"matrices of different formats: {sorted(kinds)}")
        fmt, group, scale, zeros = kinds.pop()
        mats = (gate, up, down, shared_gate, shared_up, shared_down)
        experts = cls(*(None if m is None else m.packed for m in mats), format=fmt,
                      group_size=group, scale_type=scale, zeros=zeros, first_expert=first_expert)
        experts.shapes = tuple(None if m is None else m.shape for m in mats)
        return experts

    def c(self):
        check_places(self.tensors, self._at)
        return self._c


class W4Decoder:
    """Few-token forward of a layer whose experts are 4-bit (workspace owner)."""

    def __init__(self, shape: Shape, experts: W4Experts):
        self.shape, self.experts = shape, experts
        self.device = experts.tensors[0].device
        n = _lib.moe_w4_decode_workspace_bytes(shape)
        if n == 0:
            raise ValueError(f"shape outside the limits of moe_w4_decode_fwd: {shape}")
        s, e = shape, experts.c()

        def need(groups, nn, kk):
            return W4Shape(groups, nn, kk, e.format, e.group_size, e.scale_type, e.zeros)
        wants = [need(s.experts, s.inter, s.hidden)] * 2 + [need(s.experts, s.hidden, s.inter)]
        if s.shared_inter:
            wants += [need(1, s.shared_inter, s.hidden)] * 2 + [need(1, s.hidden, s.shared_inter)]
        else:
            wants += [None] * 3
        for t, has, want in zip(experts.tensors, experts.shapes or wants, wants):
            if (t is None) != (want is None):
                raise ValueError("experts: shared matrices given exactly when the shape has them")
            if t is None:
                continue
            size = _lib.moe_w4_bytes(want)
            if size == 0:
                raise ValueError("experts: format or group size does not fit the shape")
            if has != want:
                raise ValueError(f"experts: {has}, expected {want}")
            _check("experts", t, (size,), (torch.uint8,), self.device)
        self.ws = torch.empty(n, dtype=torch.uint8, device=self.device)

    def __call__(self, x, w_router=None, bias=None, topk_idx=None, topk_w=None, out=None):
        """[tokens][hidden] bf16 -> the same; routing as MoeLayer.decode."""
        out = decode_args(self.shape, self.device, x, w_router, bias, topk_idx, topk_w, out)
        with torch.cuda.device(self.device):
            _lib.moe_w4_decode_fwd(self.shape, self.experts, x, w_router, bias, topk_idx, topk_w,
                                   out, self.ws)
        return out
