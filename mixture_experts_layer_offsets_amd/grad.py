"""The global norm of a training step's gradients, and clipping by it."""
from __future__ import annotations

import torch

from . import _lib

_TYPES = {torch.bfloat16: _lib.MOE_ROW_BF16, torch.float16: _lib.MOE_ROW_F16,
          torch.float32: _lib.MOE_ROW_F32}
_data_ptr = torch.Tensor.data_ptr


def _dense(t):
    """Whether t's values fill one run of memory (in any order of its axes)."""
    want = 1
    for size, stride in sorted(zip(t.shape, t.stride()), key=lambda d: (d[1], d[0])):
        if size == 1:
            continue
        if stride != want:
            return False
        want *= size
    return True


class GradSet:
    """Tensors of moe_grad_tensor: the gradients, and where their scaled values go
    (``outs``; without, in place).

    bf16, fp16 and fp32 tensors of one device, each a dense run of memory (a
    transposed view is one; an out has its gradient's type, shape and strides).
    A value that two tensors hold, and an out that overlaps a gradient other than
    by being the same tensor, raise ValueError.  The tensors and their memory are kept
    alive here; where gradients are new tensors every step, so is their set.  A tensor
    that is given other memory afterwards (``t.data = ...``) ends the set: the calls of
    GradClip, and ``check``, raise ValueError then.  ``c`` itself does not look (40 ns a
    tensor): it names the memory that the tensors had.
    """

    def __init__(self, grads, outs=None):
        self.grads = list(grads)
        self.outs = self.grads if outs is None else list(outs)
        if len(self.grads) != len(self.outs):
            raise ValueError(f"outs: {len(self.outs)} for {len(self.grads)} gradients")
        self.device = self.grads[0].device if self.grads else None
        self._c = (_lib.MoeGradTensor * len(self.grads))()
        self._tensors = self.grads if outs is None else self.grads + self.outs
        # kept, so that an address stands for one piece of memory as long as the set lives
        self._memory = [t.untyped_storage() for t in self._tensors]
        self._at = list(map(_data_ptr, self._tensors))
        spans = []
        for i, (x, o) in enumerate(zip(self.grads, self.outs)):
            for name, t in (("gradient", x), ("out", o)):
                if t.device != self.device:
                    raise ValueError(f"{name} {i}: on {t.device}, expected {self.device}")
                if t.dtype not in _TYPES:
                    raise ValueError(f"{name} {i}: {t.dtype}, expected bf16, fp16 or fp32")
                if t.numel() and not t.is_contiguous() and not _dense(t):
                    raise ValueError(f"{name} {i}: strides {t.stride()} of shape {tuple(t.shape)} "
                                     "are not dense")
            if o is not x and (o.dtype != x.dtype or o.shape != x.shape or
                               (x.numel() > 1 and o.stride() != x.stride())):
                raise ValueError(f"out {i}: not of its gradient's type, shape and strides")
            n = x.numel()
            if n:
                size = n * x.element_size()
                spans.append((x.data_ptr(), x.data_ptr() + size))
                if o.data_ptr() != x.data_ptr():
                    spans.append((o.data_ptr(), o.data_ptr() + size))
            self._c[i] = _lib.MoeGradTensor(x.data_ptr(), o.data_ptr(), n, _TYPES[x.dtype])
        spans.sort()
        for (_, end), (begin, _) in zip(spans, spans[1:]):
            if begin < end:
                raise ValueError("two of the tensors overlap")

    def __len__(self):
        return len(self.grads)

    def check(self):
        """ValueError if a tensor was given other memory since."""
        if list(map(_data_ptr, self._tensors)) != self._at:
            raise ValueError("a tensor of the set was given other memory since")

    def c(self):
        return self._c


class GradClip:
    """Clipping of a GradSet by its global norm (workspace owner).

    The call scales the gradients so that their norm is at most ``max_norm`` and
    returns the norm that they had (fp32, one value on the device: no call waits
    for it).  A norm that is not finite is not caught: look at the returned one.
    Calls enqueue on the current stream; the workspace and the returned tensor are
    reused by the next call, so calls on several streams need one object each, and
    so do graphs that may run at the same time.  ``total`` and ``scale`` are the
    two halves, for ranks that hold parts of the gradients.
    """

    def __init__(self, grads: GradSet, norm_type=_lib.MOE_NORM_2):
        if norm_type not in (_lib.MOE_NORM_2, _lib.MOE_NORM_INF):
            raise ValueError(f"norm_type: {norm_type}")
        self.set, self.norm_type = grads, norm_type
        n = _lib.moe_grad_workspace_bytes(grads)
        if n == 0:
            raise ValueError("more or larger tensors than moe_grad_clip takes")
        if grads.device is None:
            raise ValueError("no gradients")
        self.ws = torch.empty(n, dtype=torch.uint8, device=grads.device)
        self.norm = torch.empty(1, dtype=torch.float32, device=grads.device)
        self._total = torch.empty(1, dtype=torch.float64, device=grads.device)

    @staticmethod
    def _max_norm(max_norm):
        if not max_norm >= 0:
            raise ValueError(f"max_norm: {max_norm}")
        return max_norm

    def __call__(self, max_norm):
        max_norm = self._max_norm(max_norm)
        self.set.check()
        with torch.cuda.device(self.set.device):
            _lib.moe_grad_clip(self.set, self.norm_type, max_norm, self.norm, self.ws)
        return self.norm

    def total(self):
        """The sum of squares, or the largest magnitude (fp64, one value)."""
        self.set.check()
        with torch.cuda.device(self.set.device):
            _lib.moe_grad_norm(self.set, self.norm_type, self._total, self.norm, self.ws)
        return self._total

    def scale(self, total, max_norm):
        """Scale by a total (fp64, one value on the device) of all ranks' parts."""
        max_norm = self._max_norm(max_norm)
        if total.dtype != torch.float64 or total.numel() != 1 or total.device != self.set.device:
            raise ValueError("total: expected one fp64 value on the gradients' device")
        self.set.check()
        with torch.cuda.device(self.set.device):
            _lib.moe_grad_scale(self.set, self.norm_type, total, max_norm, self.norm)
        return self.norm
