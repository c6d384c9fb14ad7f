"""What W4Linear and W4Decoder are built from, on the host."""
import contextlib
import dataclasses
import os

import pytest
import torch

import mixture_experts_layer_offsets_amd as m
from mixture_experts_layer_offsets_amd import _lib


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_layer_offsets_amd import build
        build.build(verbose=False)
    m.load()


SHAPE = m.W4Shape(2, 48, 256)


def packed(shape, extra=0):
    return torch.zeros(m.moe_w4_bytes(shape) + extra, dtype=torch.uint8)


def test_packed_weights_have_the_size_that_their_shape_says():
    """The kernels read moe_w4_bytes of them: a product or an unpacking of
    anything else is refused before it can read behind it."""
    n = m.moe_w4_bytes(SHAPE)
    bad = [packed(SHAPE)[:-1], packed(SHAPE)[:0], packed(SHAPE, 256), packed(SHAPE, n)[::2],
           packed(SHAPE).view(2, -1), packed(SHAPE).view(torch.int8), packed(SHAPE).float(),
           packed(m.W4Shape(1, 48, 256))]
    x, off = torch.zeros((3, 256), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    for t in bad:
        lin = m.W4Linear(SHAPE, t)
        for call in (lambda: lin(x, off), lin.values):
            with pytest.raises(ValueError, match="packed"):
                call()
    lin = m.W4Linear(dataclasses.replace(SHAPE, k=200), packed(SHAPE))
    with pytest.raises(ValueError, match="limits"):
        lin.values()


def test_packed_weights_that_fit_are_taken(monkeypatch):
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    calls = []
    for name in ("moe_w4_linear", "moe_w4_unpack"):
        monkeypatch.setattr(_lib, name, lambda *a, name=name: calls.append(name))
    lin = m.W4Linear(SHAPE, packed(SHAPE))
    x, off = torch.zeros((3, 256), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    assert lin(x, off).shape == (3, 48) and lin.values().shape == (2, 256, 48)
    assert calls == ["moe_w4_linear", "moe_w4_unpack"]


def test_experts_of_the_wrong_orientation_or_number_are_refused():
    """Matrices [k][n] and [n][k], and 2 groups of n or one of 2n, take the same
    bytes: the layer compares the shapes that they were packed with."""
    layer = m.Shape(4, 256, 8, 2, 128, 128)
    mats = {s: m.W4Linear(s, packed(s)) for s in (
        m.W4Shape(8, 128, 256), m.W4Shape(8, 256, 128), m.W4Shape(4, 256, 256), m.W4Shape(4, 512, 128),
        m.W4Shape(1, 128, 256), m.W4Shape(1, 256, 128))}
    up, down, up4, down4, up1, down1 = mats.values()
    m.W4Decoder(layer, m.W4Experts.of(up, up, down, up1, up1, down1))
    for wrong in ((down, up, down, up1, up1, down1), (up, down, down, up1, up1, down1),
                  (up, up, up, up1, up1, down1), (up4, up4, down, up1, up1, down1),
                  (up, up, down4, up1, up1, down1), (up, up, down, down1, up1, down1),
                  (up, up, down, up1, up1, up1)):
        with pytest.raises(ValueError, match="experts"):
            m.W4Decoder(layer, m.W4Experts.of(*wrong))
    # packed tensors by themselves say nothing but their size
    m.W4Decoder(layer, m.W4Experts(up.packed, up.packed, down.packed, up1.packed, up1.packed,
                                   down1.packed))
