"""Objects that hold tensors by address, when the tensors are given other memory: checked
again, or refused (no GPU: the entry points are replaced)."""
import contextlib
import os

import pytest
import torch

import mixture_experts_layer_offsets_amd as m
from mixture_experts_layer_offsets_amd import _lib

ENTRIES = ("moe_f8_linear", "moe_f8_unpack", "moe_f8_transpose", "moe_w4_linear", "moe_w4_unpack",
           "moe_f8_decode_fwd", "moe_w4_decode_fwd", "moe_grad_clip", "moe_grad_norm", "moe_grad_scale")


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_layer_offsets_amd import build
        build.build(verbose=False)
    return _lib.load()


@pytest.fixture
def calls(monkeypatch):
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    made = []
    for name in ENTRIES:
        monkeypatch.setattr(_lib, name, lambda *a, name=name: made.append((name, a)))
    return made


def linears():
    f8, w4 = m.F8Shape(1, 48, 256), m.W4Shape(1, 48, 256)
    return [(m.F8Linear, f8, m.moe_f8_bytes(f8)), (m.W4Linear, w4, m.moe_w4_bytes(w4))]


@pytest.mark.parametrize("which", [0, 1], ids=["f8", "w4"])
def test_weights_of_a_product(which, calls):
    """Another packed tensor, the same one with other memory, and another shape."""
    cls, shape, size = linears()[which]
    x = torch.zeros((3, 256), dtype=torch.bfloat16)
    for exchange in (lambda lin: setattr(lin, "packed", torch.empty(size - 256, dtype=torch.uint8)),
                     lambda lin: setattr(lin, "packed", lin.packed[::2]),
                     lambda lin: setattr(lin.packed, "data", torch.empty(8, dtype=torch.uint8)),
                     lambda lin: setattr(lin, "shape", type(shape)(1, 64, 256))):
        lin = cls(shape, torch.empty(size, dtype=torch.uint8))
        lin(x)
        made = len(calls)
        exchange(lin)
        for call in (lambda: lin(x), lin.values):
            with pytest.raises(ValueError, match="packed"):
                call()
        assert len(calls) == made
    # weights of the same size are taken, wherever they lie
    lin = cls(shape, torch.empty(size, dtype=torch.uint8))
    lin(x)
    lin.packed.data = torch.empty(size, dtype=torch.uint8)
    lin(x)
    lin.packed = torch.empty(size, dtype=torch.uint8)
    lin(x)
    assert len(calls) == made + 3 and calls[-1][1][3] is lin.packed


def experts(cls, shape_of, size_of):
    """A layer's experts of 4- or 8-bit matrices, and the layer."""
    layer = m.Shape(4, 256, 8, 2, 128, 128)
    mats = [shape_of(8, 128, 256)] * 2 + [shape_of(8, 256, 128)] + \
        [shape_of(1, 128, 256)] * 2 + [shape_of(1, 256, 128)]
    return layer, cls(*[torch.zeros(size_of(s), dtype=torch.uint8) for s in mats])


@pytest.mark.parametrize("kind", ["f8", "w4"])
@pytest.mark.parametrize("which", [0, 2, 5])
def test_experts_of_a_layer(kind, which, calls):
    """A matrix given other memory, of the same size or not."""
    cls, shape_of, size_of, dec_of = {
        "f8": (m.F8Experts, m.F8Shape, m.moe_f8_bytes, m.F8Decoder),
        "w4": (m.W4Experts, m.W4Shape, m.moe_w4_bytes, m.W4Decoder)}[kind]
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    idx, w = torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2))
    for size in (0, 5, None):
        layer, e = experts(cls, shape_of, size_of)
        dec = dec_of(layer, e)
        dec(x, topk_idx=idx, topk_w=w)
        assert calls[-1][1][1] is e and e.c().gate == e.tensors[0].data_ptr()
        t = e.tensors[which]
        t.data = torch.zeros(t.numel() if size is None else size, dtype=torch.uint8)
        with pytest.raises(ValueError, match="memory"):
            _lib._shape(e)
        with pytest.raises(ValueError, match="memory"):
            e.c()


@pytest.mark.parametrize("with_outs", [False, True])
def test_gradients_of_a_set(with_outs, calls):
    """A gradient or out with other memory: refused by every call of GradClip, and the old
    memory is not given away while the set has its address."""
    for which in range(3 if with_outs else 2):
        grads = [torch.zeros((4, 6)), torch.zeros(5, dtype=torch.half)]
        outs = [torch.zeros((4, 6)), torch.zeros(5, dtype=torch.half)] if with_outs else None
        clip = m.GradClip(m.GradSet(grads, outs))
        clip(1.0)
        clip.scale(clip.total(), 1.0)
        made = len(calls)
        t = (grads + (outs or []))[which]
        old = t.data_ptr()
        t.data = torch.zeros_like(t)
        assert t.data_ptr() != old
        assert all(torch.zeros_like(t).data_ptr() != old for _ in range(8))
        for call in (clip.set.check, lambda: clip(1.0), clip.total, lambda: clip.scale(clip._total, 1.0)):
            with pytest.raises(ValueError, match="memory"):
                call()
        assert len(calls) == made
