"""Decode steps of the gated delta rule that start from rows of their own or from zeros, and serving loops driven by slot
plans alone: rows go from one request to the next on the device, and nothing waits for the host."""
import pytest
import torch

import linear_attention_recurrence_simple_gb300 as gla
from tests.delta_helpers import DK, DV, Batch, check

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
SHAPE_ERR = -2


@pytest.fixture(scope="module", autouse=True)
def _setup():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    gla.load_library()
    yield
    assert gla.gla_get_device_error() == 0


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def kind(dtype):
    return "bf16" if dtype == BF else "f32"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sdtype", [F32, BF])
def test_decode_from_rows_of_its_own(sdtype, dtype):
    """From zeros over a row that holds NaN, from another row (two sequences from one), in place, and left alone."""
    H, N = 3, 6
    b = Batch(31, [1] * N, H, dtype)
    pool = (torch.randn(9, H, DK, DV, generator=torch.Generator().manual_seed(32)) * 0.1).to(sdtype)
    slot, start = [4, 2, 0, 7, -1, 8], [-1, 6, 6, 7, 3, -1]
    pool[4] = float("nan")
    pool[8] = float("inf")
    dev, o = pool.cuda(), torch.full((N, H, DV), 5.0, dtype=dtype, device="cuda")
    assert gla.gla_delta_decode_step(*b.inputs(), dev, slot=i32(slot), start_row=i32(start), o=o) is o
    assert gla.gla_get_device_error() == 0
    for n, s in enumerate(slot):
        if s < 0:
            assert bool((o[n] == 5.0).all())
            continue
        ro, rS = b.ref(n, pool[start[n]] if start[n] >= 0 else torch.zeros(H, DK, DV))
        check(o[n:n + 1], ro, kind(dtype), "o")
        check(dev[s], rS, kind(sdtype), "state")
    for s in set(range(9)) - set(slot):
        assert torch.equal(dev[s].cpu(), pool[s])


@pytest.mark.parametrize("sdtype", [F32, BF])
def test_decode_start_rows_as_the_slots(sdtype):
    """Start rows that are the slots, or no slots and start rows 0 .. N - 1: the same bits as the step without them."""
    b = Batch(33, [1] * 5, 2, BF)
    pool, x = (torch.randn(5, 2, DK, DV) * 0.1).to(sdtype).cuda(), b.inputs()
    slot = i32([3, 0, 4, 1, 2])
    a, c, d, e = (pool.clone() for _ in range(4))
    assert torch.equal(gla.gla_delta_decode_step(*x, a, slot=slot), gla.gla_delta_decode_step(*x, c, slot=slot, start_row=slot))
    assert torch.equal(a, c)
    assert torch.equal(gla.gla_delta_decode_step(*x, d), gla.gla_delta_decode_step(*x, e, start_row=i32(range(5))))
    assert torch.equal(d, e)


def test_decode_start_rows_outside_are_reported():
    b = Batch(34, [1, 1], 1, BF)
    pool = torch.full((3, 1, DK, DV), float("nan"), device="cuda")
    o = gla.gla_delta_decode_step(*b.inputs(), pool, slot=i32([0, 2]), start_row=i32([3, -2]))
    assert gla.gla_get_device_error() == SHAPE_ERR
    for n, s in enumerate((0, 2)):  # from zeros
        ro, rS = b.ref(n, torch.zeros(1, DK, DV))
        check(o[n:n + 1], ro, "bf16", "o")
        check(pool[s], rS, "f32", "state")


def test_decode_start_row_arguments():
    b = Batch(35, [1, 1], 1, BF)
    pool = torch.zeros(3, 1, DK, DV, device="cuda")
    for bad in (i32([0]), i32([[0, 1]]), torch.tensor([0, 1], device="cuda"), torch.tensor([0, 1], dtype=torch.int32)):
        with pytest.raises((ValueError, TypeError)):
            gla.gla_delta_decode_step(*b.inputs(), pool, start_row=bad)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sdtype", [F32, BF])
@pytest.mark.parametrize("captured", [False, True])
def test_single_tokens_over_a_pool_that_changes_hands(captured, sdtype, dtype):
    """More requests than rows, one token each a step: every step is the plan and the decode step by its maps, eager or as
    one graph's replays.  A row that becomes free goes to the next request, whose output must not see what it holds."""
    H, R = 2, 3
    total = [4, 2, 5, 3, 1, 4, 2]
    N = len(total)
    b = Batch(36, total, H, dtype)
    x = b.inputs()
    base, todo = torch.from_numpy(b.cu[:-1]).cuda(), i32(total)
    pool = torch.full((R, H, DK, DV), float("nan"), dtype=sdtype, device="cuda")
    held, seen = i32([-1] * N), torch.zeros(N, dtype=torch.int32, device="cuda")
    new, o = torch.empty_like(seen), torch.zeros(N, H, DV, dtype=dtype, device="cuda")
    got = torch.full((int(b.cu[-1]) + 1, H, DV), float("nan"), dtype=dtype, device="cuda")  # (the last row: no one's)
    last = int(b.cu[-1])

    def step():
        new.copy_(torch.where(seen < todo, 1, -1))
        p = gla.gla_slot_plan(new, held, seen, R, N)
        at = (base + seen).clamp(max=last - 1).long()
        gla.gla_delta_decode_step(*[t[at] for t in x], pool, slot=p.slot, start_row=p.start_row, o=o)
        there = p.slot >= 0
        got.index_copy_(0, torch.where(there, at, last), o)
        held.copy_(p.row)
        seen.add_(there.to(torch.int32))

    run = step
    if captured:
        gla.gla_delta_decode_step(*[t[:N].contiguous() for t in x], pool.clone()[:1].expand(N, -1, -1, -1).contiguous(),
                                  start_row=i32([-1] * N))  # (a first call before the capture)
        gla.gla_slot_plan(i32([1]), i32([-1]), None, R, 1)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            step()
        run = graph.replay
    for _ in range(12):
        run()
    torch.cuda.synchronize()
    assert seen.tolist() == total and held.tolist() == [-1] * N
    want = torch.cat([b.ref(n, torch.zeros(H, DK, DV))[0] for n in range(N)])
    # a bf16 pool rounds the state at each of up to 5 steps: 5 x 2^-9 of it at most, within the bf16 bound
    check(got[:-1], want, "bf16" if BF in (dtype, sdtype) else "f32", "o")
