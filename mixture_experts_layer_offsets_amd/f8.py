"""8-bit weights with a scale per 128 x 128 block: packed matrices, their products
and gradients, the few-token layer."""
from __future__ import annotations

import torch

from . import _lib
from ._lib import F8Shape, Shape
from .w4 import _check, check_places, decode_args, places

_ROWS = {_lib.MOE_ROW_BF16: (torch.bfloat16, torch.int16), _lib.MOE_ROW_F16: (torch.float16,)}
_TYPES = {torch.bfloat16: _lib.MOE_ROW_BF16, torch.int16: _lib.MOE_ROW_BF16,
          torch.float16: _lib.MOE_ROW_F16, torch.float32: _lib.MOE_ROW_F32}


class F8Linear:
    """Packed 8-bit matrices [groups][k][n], their products and the gradients.

    ``F8Linear.quantize`` takes weights [groups][k][n] (products x*W), ``F8Linear.pack``
    ready-made E4M3 codes [groups][n][k] and scales; weights that are packed already
    come as a uint8 tensor of moe_f8_bytes (checked in every call).  Calls
    enqueue on the current stream and allocate what they need on it.
    """

    def __init__(self, shape: F8Shape, packed: torch.Tensor):
        self.shape, self.packed = shape, packed
        self._need = None, 0  # a shape and its bytes

    def _size(self):
        """Bytes of the packed tensor; ValueError for a shape outside the limits."""
        if self._need[0] is not self.shape:
            self._need = self.shape, self._bytes(self.shape)
        return self._need[1]

    def _weights(self):
        """The packed tensor: the kernels read all that the shape says of it.  Looked at in
        every call: it, its memory or the shape may have been exchanged."""
        _check("packed", self.packed, (self._size(),), (torch.uint8,))
        return self.packed

    @staticmethod
    def _bytes(shape):
        n = _lib.moe_f8_bytes(shape)
        if n == 0:
            raise ValueError(f"shape outside the limits of moe_f8_shape: {shape}")
        return n

    @classmethod
    def _buffer(cls, shape, device):
        return torch.empty(cls._bytes(shape), dtype=torch.uint8, device=device)

    @classmethod
    def quantize(cls, w, row_type=_lib.MOE_ROW_BF16):
        if w.dim() != 3:
            raise ValueError(f"w: {w.dim()} dimensions, expected [groups][k][n]")
        shape = F8Shape(w.shape[0], w.shape[2], w.shape[1], row_type)
        packed = cls._buffer(shape, w.device)
        _check("w", w, w.shape, tuple(_TYPES))
        with torch.cuda.device(w.device):
            _lib.moe_f8_quantize(shape, w, _TYPES[w.dtype], packed)
        return cls(shape, packed)

    @classmethod
    def pack(cls, shape: F8Shape, codes, scales):
        packed = cls._buffer(shape, codes.device)
        _check("codes", codes, (shape.groups, shape.n, shape.k), (torch.uint8, torch.float8_e4m3fn))
        _check("scales", scales, (shape.groups, -(-shape.n // 128), -(-shape.k // 128)),
               (torch.float32,), codes.device)
        with torch.cuda.device(codes.device):
            _lib.moe_f8_pack(shape, codes, scales, packed)
        return cls(shape, packed)

    def transposed(self):
        """The matrices of x*W^T: the same values, laid out for the data gradient."""
        s, packed = self.shape, self._weights()
        turned = F8Shape(s.groups, s.k, s.n, s.row_type)
        buf = self._buffer(turned, packed.device)
        with torch.cuda.device(packed.device):
            _lib.moe_f8_transpose(s, packed, buf)
        return F8Linear(turned, buf)

    def values(self):
        """The weights [groups][k][n] that the codes stand for, in fp32."""
        s, packed = self.shape, self._weights()
        w = torch.empty((s.groups, s.k, s.n), dtype=torch.float32, device=packed.device)
        with torch.cuda.device(packed.device):
            _lib.moe_f8_unpack(s, packed, w)
        return w

    def _offsets(self, offsets, device):
        s = self.shape
        if offsets is None and s.groups != 1:
            raise ValueError("offsets: needed with more than one group")
        if offsets is not None:
            _check("offsets", offsets, (s.groups + 1,), (torch.int32,), device)

    def _rows(self, name, t, width, device, rows=None):
        if t.dim() != 2:
            raise ValueError(f"{name}: {t.dim()} dimensions, expected [rows][{width}]")
        _check(name, t, (t.shape[0] if rows is None else rows, width), _ROWS[self.shape.row_type],
               device, rows=True)

    def __call__(self, x, offsets=None, out=None):
        """x [rows][k] -> [rows][n] of the shape's row type; with ``offsets``
        [groups + 1] int32 the rows of group g are [offsets[g], offsets[g + 1]), and
        rows in no group are left as they are (zeros in a new ``out``).  Of
        ``transposed()`` matrices and dy: the data gradient."""
        s, packed = self.shape, self._weights()
        dev = packed.device
        self._rows("x", x, s.k, dev)
        self._offsets(offsets, dev)
        rows = x.shape[0]
        if out is None:
            make = torch.empty if offsets is None else torch.zeros
            out = make((rows, s.n), dtype=x.dtype, device=dev)
        self._rows("out", out, s.n, dev, rows)
        n = _lib.moe_f8_linear_workspace_bytes(s, rows)
        if n == 0:
            raise ValueError(f"{rows} rows are outside the limits of moe_f8_linear")
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        with torch.cuda.device(dev):
            _lib.moe_f8_linear(s, x, offsets, packed, out, ws)
        return out

    def weight_gradient(self, x, dy, offsets=None, out=None):
        """dw [groups][k][n] of the shape's row type: per group x^T dy, both in 8 bits
        with a scale per 128 rows of a column."""
        s, dev = self.shape, self.packed.device
        self._size()
        self._rows("x", x, s.k, dev)
        rows = x.shape[0]
        self._rows("dy", dy, s.n, dev, rows)
        self._offsets(offsets, dev)
        if out is None:
            out = torch.empty((s.groups, s.k, s.n), dtype=_ROWS[s.row_type][0], device=dev)
        _check("out", out, (s.groups, s.k, s.n), _ROWS[s.row_type], dev)
        n = _lib.moe_f8_wgrad_workspace_bytes(s, rows)
        if n == 0:
            raise ValueError(f"{rows} rows are outside the limits of moe_f8_wgrad")
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        with torch.cuda.device(dev):
            _lib.moe_f8_wgrad(s, x, dy, offsets, out, ws)
        return out


class F8Experts:
    """moe_f8_experts: the packed matrices of a layer's experts (gate, up [E][H][I],
    down [E][I][H]; the shared expert's with one group), uint8 tensors as moe_f8_pack
    and moe_f8_quantize leave them, kept alive here.  A tensor that is given other memory
    afterwards (``t.data = ...``) ends them: calls raise ValueError."""

    def __init__(self, gate, up, down, shared_gate=None, shared_up=None, shared_down=None, *,
                 first_expert=0):
        self.tensors = (gate, up, down, shared_gate, shared_up, shared_down)
        self.shapes = None  # (groups, n, k) of the matrices, where they are known
        self._at = places(self.tensors)
        self._c = _lib.MoeF8Experts(_lib._i32(first_expert), *(a and a[0] for a in self._at))

    @classmethod
    def of(cls, gate: F8Linear, up: F8Linear, down: F8Linear, shared_gate=None, shared_up=None,
           shared_down=None, first_expert=0):
        """From F8Linear matrices."""
        mats = (gate, up, down, shared_gate, shared_up, shared_down)
        experts = cls(*(None if m is None else m.packed for m in mats), first_expert=first_expert)
        experts.shapes = tuple(None if m is None else (m.shape.groups, m.shape.n, m.shape.k)
                               for m in mats)
        return experts

    def c(self):
        check_places(self.tensors, self._at)
        return self._c


class F8Decoder:
    """Few-token forward of a layer whose experts are 8-bit (workspace owner).

    The workspace is the next call's too, so calls on several streams need one object
    each, and so do graphs that may run at the same time."""

    def __init__(self, shape: Shape, experts: F8Experts):
        self.shape, self.experts = shape, experts
        self.device = experts.tensors[0].device
        n = _lib.moe_f8_decode_workspace_bytes(shape)
        if n == 0:
            raise ValueError(f"shape outside the limits of moe_f8_decode_fwd: {shape}")
        s = shape
        wants = [(s.experts, s.inter, s.hidden)] * 2 + [(s.experts, s.hidden, s.inter)]
        if s.shared_inter:
            wants += [(1, s.shared_inter, s.hidden)] * 2 + [(1, s.hidden, s.shared_inter)]
        else:
            wants += [None] * 3
        for t, has, want in zip(experts.tensors, experts.shapes or wants, wants):
            if (t is None) != (want is None):
                raise ValueError("experts: shared matrices given exactly when the shape has them")
            if t is None:
                continue
            if has != want:
                raise ValueError(f"experts: (groups, n, k) {has}, expected {want}")
            _check("experts", t, (_lib.moe_f8_bytes(F8Shape(*want)),), (torch.uint8,), self.device)
        self.ws = torch.empty(n, dtype=torch.uint8, device=self.device)

    def __call__(self, x, w_router=None, bias=None, topk_idx=None, topk_w=None, out=None):
        """[tokens][hidden] bf16 -> the same; routing as MoeLayer.decode."""
        out = decode_args(self.shape, self.device, x, w_router, bias, topk_idx, topk_w, out)
        with torch.cuda.device(self.device):
            _lib.moe_f8_decode_fwd(self.shape, self.experts, x, w_router, bias, topk_idx, topk_w,
                                   out, self.ws)
        return out
