"""The ends of the MXFP4 scale range, E8M0 bytes 253 to 255: values within
bf16's range as they are, those past it infinite, and 255 not a number (the
format's NaN), alike in the values and in the products."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_offsets_amd as m
import test_gpu_w4 as base
import w4_oracle as wo

pytestmark = pytest.mark.gpu
_built = base._built


@pytest.mark.parametrize("rows", [1, 20])
@pytest.mark.parametrize("scale", [252, 253, 254, 255])
def test_largest_scales(rows, scale):
    codes = np.zeros((1, 16, 16), np.uint8)
    codes[0, :, 0] = np.arange(16)                     # one weight beside zeros
    lin = m.W4Linear.pack(m.W4Shape(1, 16, 32), torch.from_numpy(codes).cuda(),
                          torch.full((1, 16, 1), scale, dtype=torch.uint8, device="cuda"))
    want = np.full(16, np.nan)
    if scale < 255:
        with np.errstate(over="ignore"):
            want = (wo.E2M1 * 2.0 ** (scale - 127)).astype(np.float32)
    x = torch.zeros((rows, 32), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1
    assert np.array_equal(lin.values()[0, 0].cpu().numpy(), want, equal_nan=True)
    for row in lin(x).float().cpu().numpy():
        assert np.array_equal(row, want, equal_nan=True)
