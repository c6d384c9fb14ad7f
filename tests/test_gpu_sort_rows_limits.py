"""The expert-sorted rows at the ends of their limits."""
import os

import pytest
import torch

import mixture_experts_layer_offsets_amd as m
from gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mixture_experts_layer_offsets_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_layer_offsets_amd import build
        build.build(verbose=False)
    m.load()


@pytest.mark.parametrize("experts", [1, 64, 65, 1024])
@pytest.mark.parametrize("align", [1, 16])
def test_an_empty_batch_stays_in_its_workspace(experts, align):
    """No tokens: zero counts and offsets, and nothing behind the workspace's
    reported size is written."""
    shape = m.SortShape(0, experts, 3, 64, align=align)
    note(f"empty batch, {experts} experts")
    need = m.moe_sort_workspace_bytes(shape)
    assert need >= 4 * experts
    buf = torch.full((need + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    empty = torch.empty((0, 3), **i32)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    for call in (lambda c, o, ws: m.moe_sort_layout(shape, empty, c, o, empty, empty, ws),
                 lambda c, o, ws: m.moe_sort_fwd(shape, x, empty, c, o, empty, empty, x, ws)):
        counts, offsets = torch.full((experts,), -7, **i32), torch.full((experts + 1,), -7, **i32)
        call(counts, offsets, buf[:need])
        assert torch.all(counts == 0) and torch.all(offsets == 0)
        assert torch.all(buf[need:] == 0x5A)


@pytest.mark.parametrize("T,D", [(65530, 1032), (70000, 1032), (263000, 24)])
@pytest.mark.parametrize("align", [1, 8])
def test_more_workgroups_than_a_grid_dimension(T, D, align):
    """Tokens enough that the workgroups of one call fill more than one row of
    the grid: rows, padding and gradients as by their definitions.  Copies and
    single products are exact; dw is a sum of D products in fp32."""
    k, E = 2, 5
    shape = m.SortShape(T, E, k, D, align=align)
    note(f"grid rows: {shape}")
    g = torch.Generator(device="cuda").manual_seed(T + D + align)
    bf = torch.bfloat16
    x = torch.randn((T, D), generator=g, device="cuda").to(bf)
    dout = torch.randn((T, D), generator=g, device="cuda").to(bf)
    idx = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand((T, k), generator=g, device="cuda")
    op = m.TokenSort(shape)
    xs = op.sort(x, idx, out=op.sorted_rows().fill_(7))
    end = int(op.offsets[-1])
    perm, inv = op.perm.long(), op.inv_perm.long()
    live = perm[:end] >= 0
    f = perm[:end].clamp(min=0)
    assert torch.equal(live.sum(), (idx >= 0).sum())
    assert torch.equal(xs[:end], torch.where(live[:, None], x[f // k], 0))
    dy, dw = op.unsort_backward(dout, xs, w, dy=op.sorted_rows().fill_(7))
    want = (dout[f // k].float() * w.reshape(-1)[f][:, None]).to(bf)
    assert torch.equal(dy[:end], torch.where(live[:, None], want, 0))
    assert torch.all(xs[end:] == 7) and torch.all(dy[end:] == 7)
    # a kept slot's row is its token's, so dw = <dout, x>
    dot, size = (torch.where(inv >= 0, v[:, None], 0.0) for v in
                 ((dout.double() * x.double()).sum(1), (dout.double() * x.double()).abs().sum(1)))
    assert torch.all((dw.double() - dot).abs() <= D * 2.0 ** -24 * size)
    out = op.unsort(xs, w)
    ws = torch.where(inv >= 0, w.double(), 0.0).sum(1, keepdim=True)
    ref = x.double() * ws
    assert torch.all((out.double() - ref).abs() <= ref.abs() * (2.0 ** -8 + (k + 2) * 2.0 ** -23))


@pytest.mark.parametrize("width,type", [(1032, "bf16"), (77, "f16"), (3, "f32")])
def test_gradient_of_the_unweighted_return(width, type):
    """The same rows, bit for bit, as with weights of one."""
    code, dtype = {"bf16": (m.MOE_ROW_BF16, torch.bfloat16), "f16": (m.MOE_ROW_F16, torch.float16),
                   "f32": (m.MOE_ROW_F32, torch.float32)}[type]
    op = m.TokenSort(m.SortShape(50, 6, 3, width, code, align=4, first_expert=1))
    g = torch.Generator(device="cuda").manual_seed(width)
    idx = torch.randint(0, 8, (50, 3), generator=g, device="cuda", dtype=torch.int32)
    x, dout = (torch.randn((50, width), generator=g, device="cuda").to(dtype) for _ in range(2))
    y = op.sort(x, idx)
    dy, none = op.unsort_backward(dout, y, None, dy=op.sorted_rows().fill_(7))
    ones, _ = op.unsort_backward(dout, y, torch.ones((50, 3), device="cuda"),
                                 dy=op.sorted_rows().fill_(7))
    assert none is None and torch.equal(dy, ones)
