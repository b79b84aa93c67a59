"""Workspaces of the gated delta calls: what is refused before anything is launched, and one that is used again."""
import pytest
import torch

import linear_attention_recurrence_simple_gb300 as gla
from tests.delta_helpers import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    gla.load_library()
    yield
    assert gla.gla_get_device_error() == 0


def calls(b, ws):
    x, dO = b.inputs(), b.dev("dO")[0]
    return ([*gla.gla_delta_fwd(*x, h0=b.h0.cuda(), cu_seqlens=b.cu_dev, workspace=ws)],
            [*gla.gla_delta_bwd(*x, dO, h0=b.h0.cuda(), cu_seqlens=b.cu_dev, workspace=ws)])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_workspaces_that_the_kernels_cannot_write_are_refused(dtype):
    b = Batch(61, [70, 3], 2, dtype)
    x, dO = b.inputs(), b.dev("dO")[0]
    size = gla.gla_delta_bwd_workspace_bytes(2, 73, 2, True, 0 if dtype == torch.bfloat16 else 1)
    wide = torch.empty(2 * size, dtype=torch.uint8, device="cuda")
    for bad, error in ((torch.empty(size, dtype=torch.uint8), ValueError), (wide[::2], ValueError), (wide.tolist, TypeError),
                       (wide[:1000], gla.GlaError), (wide[4:size + 4], gla.GlaError)):
        for call in (lambda: gla.gla_delta_fwd(*x, cu_seqlens=b.cu_dev, workspace=bad),
                     lambda: gla.gla_delta_bwd(*x, dO, cu_seqlens=b.cu_dev, workspace=bad)):
            with pytest.raises(error):
                call()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_workspace_for_calls_of_every_size(dtype):
    """What an earlier call left in it does not show, NaN least of all; nothing is written behind its stated size."""
    code = 0 if dtype == torch.bfloat16 else 1
    batches = [Batch(62 + i, lens, 2, dtype) for i, lens in enumerate([[300, 40], [1], [64, 0, 65], [129] * 5])]
    size = max(gla.gla_delta_bwd_workspace_bytes(len(b.lens), sum(b.lens), 2, True, code) for b in batches)
    ws = torch.full((size + 4096,), 255, dtype=torch.uint8, device="cuda")
    for b in batches + batches[::-1]:
        for got, want in zip(calls(b, ws[:size]), calls(b, None)):
            assert all(torch.equal(g, w) for g, w in zip(got, want))
    assert bool((ws[size:] == 255).all())
    for b in batches:  # exactly as large as it says
        own = torch.full((gla.gla_delta_bwd_workspace_bytes(len(b.lens), sum(b.lens), 2, True, code) + 512,), 255,
                         dtype=torch.uint8, device="cuda")
        calls(b, own[:-512])
        assert bool((own[-512:] == 255).all())
