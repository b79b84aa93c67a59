"""Slot plans of more requests than a thread keeps in registers (8 each of 1,024), and of more than have their offsets in
shared memory, where the tokens' places come from a second launch; with rows written over those held, and captured."""
import pytest
import torch

import linear_attention_recurrence_simple_gb300 as gla
from tests.delta_helpers import plan_ref
from tests.test_gpu_delta import i32, plan_inputs

pytestmark = pytest.mark.gpu
SIZES = [(8192, 4096, 9000), (8193, 4096, 9000), (20000, 2 ** 19, 30000), (60000, 4096, 70000), (60001, 2 ** 19, 12345)]


@pytest.fixture(scope="module", autouse=True)
def _setup():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    gla.load_library()
    yield
    assert gla.gla_get_device_error() == 0


def same(got, want):
    for name, x, w in zip(gla.SlotPlan._fields, got, want):
        assert torch.equal(x.cpu(), torch.tensor(w, dtype=torch.int32)), name


@pytest.mark.parametrize("long", [3, 300])
@pytest.mark.parametrize("N,rows,budget", SIZES)
def test_many_requests(N, rows, budget, long):
    """(Short lengths: the tokens of the last requests are within the budget, too.)"""
    new, held, seen = plan_inputs(71, N, rows, long)
    for s in (seen, None):
        same(gla.gla_slot_plan(i32(new), i32(held), None if s is None else i32(s), rows, budget),
             plan_ref(new, held, s, rows, budget))


@pytest.mark.parametrize("N,rows,budget", SIZES)
def test_many_requests_with_rows_over_those_held(N, rows, budget):
    new, held, seen = plan_inputs(72, N, rows, 3)
    a, h, s = i32(new), i32(held), i32(seen)
    out = gla.gla_slot_plan(a, h, s, rows, budget)
    over = gla.SlotPlan(out[0], out[1], out[2], h, out[4], out[5])
    for _ in range(3):  # each step goes on from the rows that the last one left
        want = plan_ref(new, held, seen, rows, budget)
        gla.gla_slot_plan(a, h, s, rows, budget, out=over)
        same(over, want)
        held = want[3]


def test_the_most_requests_captured():
    """2^20 requests of a token each, a quarter of a million rows: rows in order until there are none, as one graph."""
    N, rows, budget = 2 ** 20, 2 ** 18, 2 ** 18 + 1000
    new, held = torch.ones(N, dtype=torch.int32, device="cuda"), torch.full((N,), -1, dtype=torch.int32, device="cuda")
    held[5] = 7
    graph = torch.cuda.CUDAGraph()
    gla.gla_slot_plan(new, held, None, rows, budget)
    with torch.cuda.graph(graph):
        p = gla.gla_slot_plan(new, held, None, rows, budget)
    graph.replay()
    torch.cuda.synchronize()
    want = torch.arange(rows, dtype=torch.int32)
    row = torch.cat([want[:5], want[7:8], want[5:7], want[8:]])
    assert torch.equal(p.row.cpu()[:rows], row) and bool((p.row[rows:] == -1).all())
    assert torch.equal(p.slot, p.row) and p.start_row.nonzero().numel() == N and int(p.start_row[5]) == 7
    assert int(p.start_row.sum()) == 7 - (N - 1)
    assert torch.equal(p.cu_seqlens.cpu(), torch.arange(N + 1, dtype=torch.int32).clamp(max=rows))
    assert torch.equal(p.token_seq.cpu()[:rows], want) and bool((p.token_seq[rows:] == -1).all())
    assert not bool(p.token_pos[:rows].any()) and bool((p.token_pos[rows:] == -1).all())
