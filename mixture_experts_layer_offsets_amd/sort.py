"""Tokens sorted by expert and back: caller-side buffers and argument checks."""
from __future__ import annotations

import torch

from . import _lib
from ._lib import SortShape

_ROW_DTYPES = {_lib.MOE_ROW_BF16: (torch.bfloat16, torch.int16), _lib.MOE_ROW_F16: (torch.float16,),
               _lib.MOE_ROW_F32: (torch.float32,)}


class TokenSort:
    """The expert-sorted layout of one routing, and the rows that move by it.

    ``sort`` writes the layout (``counts``, ``offsets``, ``perm``,
    ``inv_perm``) into buffers of this object and returns the sorted rows;
    ``sort_again``, ``sort_backward``, ``unsort`` and ``unsort_backward`` use
    that layout, and raise ValueError on an object that has not sorted yet (a
    captured ``sort`` writes its layout when the graph is replayed).  Every
    call enqueues on the current stream; the buffers are reused by the
    next ``sort``, so calls on several streams need one object each, and so
    do graphs that may run at the same time.  Row tensors take the shape's
    type (bf16 also as int16 bit patterns) and its strides; a tensor that
    does not fit raises ValueError before anything is enqueued.
    """

    def __init__(self, shape: SortShape, device="cuda"):
        self.shape = shape
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.max_rows = _lib.moe_sort_max_rows(shape)
        if self.max_rows < 0:
            raise ValueError(f"shape outside the limits of moe_sort_shape: {shape}")
        i32 = dict(dtype=torch.int32, device=self.device)
        self.counts = torch.empty(shape.experts, **i32)
        self.offsets = torch.empty(shape.experts + 1, **i32)
        self.perm = torch.empty(self.max_rows, **i32)
        self.inv_perm = torch.empty((shape.tokens, shape.top_k), **i32)
        self.ws = torch.empty(_lib.moe_sort_workspace_bytes(shape), dtype=torch.uint8,
                              device=self.device)
        self._has_layout = False  # until the first sort the layout is whatever lay in memory

    # -- buffers
    def token_rows(self) -> torch.Tensor:
        """An uninitialised [tokens][width] tensor with the shape's stride."""
        return self._rows(self.shape.tokens, self.shape.token_stride)

    def sorted_rows(self) -> torch.Tensor:
        """An uninitialised [max_rows][width] tensor with the shape's stride."""
        return self._rows(self.max_rows, self.shape.row_stride)

    def _rows(self, n, stride):
        s = self.shape
        buf = torch.empty((n, stride or s.width), dtype=_ROW_DTYPES[s.row_type][0],
                          device=self.device)
        return buf[:, :s.width]

    def _check(self, name, t, shape, dtypes, stride=None):
        if t.device != self.device:
            raise ValueError(f"{name}: on {t.device}, expected {self.device}")
        if t.dtype not in dtypes:
            raise ValueError(f"{name}: {t.dtype}, expected {dtypes[0]}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
        if t.numel() == 0:
            return
        want = (stride, 1) if stride is not None else torch.empty(shape, device="meta").stride()
        for size, got, exp in zip(t.shape, t.stride(), want):
            if size > 1 and got != exp:
                raise ValueError(f"{name}: strides {t.stride()}, expected {tuple(want)}")

    def _tokens(self, name, t):
        s = self.shape
        self._check(name, t, (s.tokens, s.width), _ROW_DTYPES[s.row_type],
                    s.token_stride or s.width)

    def _sorted(self, name, t):
        s = self.shape
        self._check(name, t, (self.max_rows, s.width), _ROW_DTYPES[s.row_type],
                    s.row_stride or s.width)

    def _layout(self):
        if not self._has_layout:
            raise ValueError("no layout yet: sort first")

    def _slots(self, name, t, dtype):
        self._check(name, t, (self.shape.tokens, self.shape.top_k), (dtype,))

    # -- calls
    def sort(self, x, topk_idx, out=None):
        """The layout of ``topk_idx`` and the tokens' rows sorted by it."""
        out = self.sorted_rows() if out is None else out
        self._tokens("x", x)
        self._slots("topk_idx", topk_idx, torch.int32)
        self._sorted("out", out)
        with torch.cuda.device(self.device):
            _lib.moe_sort_fwd(self.shape, x, topk_idx, self.counts, self.offsets, self.perm,
                              self.inv_perm, out, self.ws)
        self._has_layout = True
        return out

    def sort_again(self, x, out=None):
        """Other rows of the same tokens, sorted by the layout already there."""
        out = self.sorted_rows() if out is None else out
        self._tokens("x", x)
        self._sorted("out", out)
        self._layout()
        with torch.cuda.device(self.device):
            _lib.moe_sort_rows(self.shape, x, self.counts, self.offsets, self.inv_perm, out)
        return out

    def sort_backward(self, dx_sorted, out=None):
        """The tokens' gradient from the sorted rows' gradient."""
        out = self.token_rows() if out is None else out
        self._sorted("dx_sorted", dx_sorted)
        self._tokens("out", out)
        self._layout()
        with torch.cuda.device(self.device):
            _lib.moe_sort_bwd(self.shape, dx_sorted, self.inv_perm, out)
        return out

    def unsort(self, y, topk_w=None, add=None, out=None):
        """The tokens' weighted sums of their rows (plus ``add``)."""
        out = self.token_rows() if out is None else out
        self._sorted("y", y)
        if topk_w is not None:
            self._slots("topk_w", topk_w, torch.float32)
        if add is not None:
            self._tokens("add", add)
        self._tokens("out", out)
        self._layout()
        with torch.cuda.device(self.device):
            _lib.moe_unsort_fwd(self.shape, y, topk_w, self.inv_perm, add, out)
        return out

    def unsort_backward(self, dout, y, topk_w, dy=None, dtopk_w=None):
        """(dy, dtopk_w): the gradients of ``unsort``'s rows and weights.
        Without weights (``topk_w`` None) there is no gradient of them, and y
        is not read: dtopk_w is None."""
        dy = self.sorted_rows() if dy is None else dy
        if topk_w is None and dtopk_w is not None:
            raise ValueError("dtopk_w: given without topk_w")
        self._tokens("dout", dout)
        self._sorted("y", y)
        if topk_w is not None:
            self._slots("topk_w", topk_w, torch.float32)
            if dtopk_w is None:
                dtopk_w = torch.empty((self.shape.tokens, self.shape.top_k), dtype=torch.float32,
                                      device=self.device)
            self._slots("dtopk_w", dtopk_w, torch.float32)
        self._sorted("dy", dy)
        self._layout()
        with torch.cuda.device(self.device):
            if topk_w is None:  # weights of one: the rows' gradients are the tokens'
                _lib.moe_sort_rows(self.shape, dout, self.counts, self.offsets, self.inv_perm, dy)
            else:
                _lib.moe_unsort_bwd(self.shape, dout, y, topk_w, self.counts, self.offsets,
                                    self.inv_perm, dy, dtopk_w)
        return dy, dtopk_w
