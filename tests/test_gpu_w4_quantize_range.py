"""Quantising weights of the whole bf16 range to 4 bits (moe_w4_quantize): any
finite group stands for finite values.  Steps past the scale type's largest
value are held at it, and the codes saturate; everything else follows the
documented steps exactly."""
import os

import numpy as np
import pytest
import torch

import mixture_experts_layer_offsets_amd as m
from gpu_util import note

pytestmark = pytest.mark.gpu

K, GROUP = 128, 32
BF16_MAX = float(torch.finfo(torch.bfloat16).max)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mixture_experts_layer_offsets_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_layer_offsets_amd import build
        build.build(verbose=False)
    m.load()


def documented(w, sdt, zeros):
    """The values [K][n] that the documented steps give, in fp32 (w holds bf16 values)."""
    b = w.astype(np.float32).reshape(K // GROUP, GROUP, -1)
    lo, hi = np.minimum(b.min(1), 0), np.maximum(b.max(1), 0)
    f32 = np.float32
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        span = hi - lo
        if zeros:
            step = np.where(np.isinf(span), hi / f32(15) - lo / f32(15), span / f32(15))
        else:
            step = np.maximum(-lo, hi) / f32(7)
        s = torch.from_numpy(step).to(sdt).float().numpy()
        limited = np.isinf(s)
        s = np.where(limited, f32(torch.finfo(sdt).max), s)
        safe = np.where(s > 0, s, f32(1))
        z = np.full_like(s, 8)
        if zeros:
            z = np.clip(np.rint(-lo / np.where(limited, step, safe)), 0, 15)
            z = np.where(s > 0, z, 0)
        q = np.clip(np.rint(b / safe[:, None]) + z[:, None], 0, 15)
        q = np.where(s[:, None] > 0, q, z[:, None])
        v = s[:, None] * (q - z[:, None])
        q = np.where(np.isinf(v), q + np.where(q < z[:, None], 1, -1), q)
        return (s[:, None] * (q - z[:, None])).reshape(K, -1)


def weights(seed):
    """One column per kind of group: ordinary, past fp16's scales (one sign, both), bf16's largest."""
    rng = np.random.default_rng(seed)
    u = rng.uniform(-1, 1, (K, 9)).astype(np.float32)
    top = np.array([1, 6.9 * 65504, 7.2 * 65504, 16 * 65504, 1e7, 1e30, BF16_MAX, BF16_MAX, BF16_MAX])
    w = (u * top).astype(np.float32)
    w[:, 4] = np.abs(w[:, 4])
    w[::GROUP, 7], w[1::GROUP, 7] = BF16_MAX, -BF16_MAX
    w[:, 8] = -np.abs(w[:, 8])
    w[::GROUP, 8] = -BF16_MAX
    return torch.from_numpy(w).to(torch.bfloat16)


@pytest.mark.parametrize("zeros", [0, 1])
@pytest.mark.parametrize("scale", ["bf16", "f16"])
def test_finite_weights_quantise_to_finite_values(scale, zeros):
    w = weights(17)
    assert torch.all(torch.isfinite(w.float()))
    note(f"w4 quantise over the whole range: {scale} scales, zeros={zeros}")
    st, sdt = {"bf16": (m.MOE_SCALE_BF16, torch.bfloat16), "f16": (m.MOE_SCALE_F16, torch.float16)}[scale]
    lin = m.W4Linear.quantize(w[None].cuda(), m.MOE_W4_INT4, GROUP, st, zeros)
    got = lin.values()[0].cpu().numpy()
    assert np.all(np.isfinite(got))
    assert np.array_equal(got, documented(w.float().numpy(), sdt, zeros))
    # and through the product, one weight times 2^-8 at a time
    out = lin((torch.eye(K, device="cuda") * 2.0 ** -8).to(torch.bfloat16))
    assert torch.equal(out.cpu(), torch.from_numpy(got * np.float32(2.0 ** -8)).to(torch.bfloat16))


def test_the_steps_by_hand():
    """The test's own steps on groups worked by hand (host only)."""
    w = np.zeros((K, 2), np.float32)
    w[0, 0], w[1, 0] = -983040.0, 917504.0        # step 126703 (kept in bf16), past fp16's 65504
    w[0, 1] = 14.0
    v = documented(w, torch.float16, 1)
    assert v[0, 0] == -8 * 65504 and v[1, 0] == 7 * 65504 and np.all(v[2:, 0] == 0)
    v = documented(w, torch.float16, 0)
    assert v[0, 0] == -8 * 65504 and v[1, 0] == 7 * 65504 and v[0, 1] == 14
