"""Packed calls of the gated delta rule whose offsets leave rows over: the gradients of rows of no sequence are zeros."""
import pytest
import torch

import linear_attention_recurrence_simple_gb300 as gla
from tests.delta_helpers import DK, DV, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    gla.load_library()
    yield
    assert gla.gla_get_device_error() == 0


def dirty(x):
    """Memory that the next outputs of these sizes get, filled with NaN."""
    junk = [torch.full_like(t, float("nan")) for t in x for _ in range(2)]
    torch.cuda.synchronize()
    del junk


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,spare", [([70, 0, 64], 1), ([1], 200), ([65, 3], 127), ([0, 0], 70), ([], 9), ([64, 128], 64), ([5] * 40, 4000)])
def test_gradients_of_rows_of_no_sequence_are_zero(lens, spare, dtype):
    H, used, T = 3, sum(lens), sum(lens) + spare
    b = Batch(41, lens or [0], H, dtype, spare=spare)
    x, dO = b.inputs(), b.dev("dO")[0]
    for t in (*x, dO):
        t[used:] = float("nan")  # nothing may come from there either
    cu = b.cu_dev if lens else torch.zeros(1, dtype=torch.int32, device="cuda")
    h0 = b.h0.cuda() if lens else None
    own = [t[:used].clone() for t in x]
    want = gla.gla_delta_bwd(*own, dO[:used].clone(), h0=h0, cu_seqlens=cu) if used else None
    dirty(x)
    got = gla.gla_delta_bwd(*x, dO, h0=h0, cu_seqlens=cu)
    for i, g in enumerate(got[:5]):
        assert g.shape[0] == T and not bool(g[used:].any()), i  # (a NaN counts as true)
        if want:
            assert torch.equal(g[:used], want[i])
    if want:
        assert torch.equal(got[5], want[5])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_offsets_that_begin_behind_the_first_row(dtype):
    b = Batch(42, [30, 100, 20], 2, dtype)
    x, dO = b.inputs(), b.dev("dO")[0]
    cu = torch.tensor([30, 130], dtype=torch.int32, device="cuda")
    dirty(x)
    got = gla.gla_delta_bwd(*x, dO, cu_seqlens=cu, need_dh0=False)
    want = gla.gla_delta_bwd(*[t[30:130].clone() for t in x], dO[30:130].clone(), need_dh0=False,
                             cu_seqlens=torch.tensor([0, 100], dtype=torch.int32, device="cuda"))
    for g, w in zip(got[:5], want[:5]):
        assert torch.equal(g[30:130], w) and not bool(g[:30].any()) and not bool(g[130:].any())


def test_captured_with_offsets_that_change():
    """One graph, offsets of fewer and of more tokens: rows are cleared again where there were gradients."""
    b = Batch(43, [90, 60], 2, torch.bfloat16)
    x, dO, cu = b.inputs(), b.dev("dO")[0], b.cu_dev
    full = gla.gla_delta_bwd(*x, dO, cu_seqlens=cu)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gla.gla_delta_bwd(*x, dO, cu_seqlens=cu)
    graph.replay()
    assert all(torch.equal(g, w) for g, w in zip(got, full))
    cu.copy_(torch.tensor([0, 90, 90], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    for g, w in zip(got[:5], full):
        assert torch.equal(g[:90], w[:90]) and not bool(g[90:].any())
    assert got[5].shape == (2, 2, DK, DV)
