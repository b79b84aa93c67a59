"""Host-only checks of limits that the gated delta calls and the slot plan state: sizes past them are refused before any
CUDA call (fake addresses, never dereferenced)."""
import ctypes

import pytest
import torch

import linear_attention_recurrence_simple_gb300 as gla

NULL, SHAPE, UNSUP = -1, -2, -5
P, A = ctypes.c_void_p, 0x10000


@pytest.fixture(scope="module")
def lib():
    return gla.load_library()


@pytest.mark.parametrize("budget", [2 ** 30 + 1, 2 ** 31 - 65536, 2 ** 31 - 1])
def test_plan_budgets_that_token_places_cannot_count_are_refused(lib, budget):
    """Places of tokens are counted in 32 bits, a whole grid at a time."""
    def plan(seq, pos, cu=None, N=0):
        return lib.gla_slot_plan(P(A), P(A), None, N, 9, budget, P(cu), P(A), P(A), P(A), P(seq), P(pos), None)

    assert plan(A, A) == UNSUP       # (before the missing cu_seqlens is looked at)
    assert plan(None, A) == UNSUP and plan(A, None) == UNSUP
    assert plan(None, None) == NULL  # without places a budget is a number to compare with


def test_plan_binding_refuses_before_a_c_int_wraps():
    x = torch.zeros(3, dtype=torch.int32)
    for rows, budget, status in ((2 ** 32 + 4, 8, UNSUP), (2 ** 19 + 1, 8, UNSUP), (4, 2 ** 30 + 1, UNSUP), (4, 2 ** 32 + 8, UNSUP),
                                 (0, 8, SHAPE), (-2 ** 32 + 4, 8, SHAPE)):
        with pytest.raises(gla.GlaError) as e:
            gla.gla_slot_plan(x, x, None, rows, budget)
        assert e.value.status == status


def test_decode_from_rows_argument_errors(lib):
    NULL, DTYPE, ALIGN = -1, -3, -4

    def step(q=A, state=A, sdt=1, slot=None, start=A, rows=9, o=A, N=3, H=2, dk=96, dt=0):
        return lib.gla_delta_decode_step_rows(P(q), P(A), P(A), P(A), P(A), 0.1, P(state), sdt, P(slot), P(start), rows, P(o),
                                              N, H, dk, 192, dt, None)

    for sdt in (0, 1):
        assert step(sdt=sdt, dt=2) == DTYPE and step(sdt=sdt, dk=95) == UNSUP
        assert step(sdt=sdt, rows=2) == SHAPE and step(sdt=sdt, N=2 ** 30, slot=A) == SHAPE
        assert step(sdt=sdt, q=None) == NULL and step(sdt=sdt, state=None) == NULL
        assert step(sdt=sdt, start=A + 2) == ALIGN and step(sdt=sdt, o=A + 4) == ALIGN
        assert step(sdt=sdt, N=0, q=None, start=None) == 0
    assert step(sdt=2) == DTYPE and step(sdt=-1) == DTYPE


def test_workspace_sizes_are_those_stated():
    """Bytes of a (chunk place, head) as include/gla.h has them, beside 256 bytes, the order and dbeta's parts."""
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gla.h")).read()
    stated = [int(x.replace(",", "")) for x in re.search(r"Workspaces: ([\d,]+) bytes.*?\(fp32 ([\d,]+)\).*?forward, ([\d,]+).*?\(fp32 ([\d,]+)\)",
                                                         re.sub(r"\n \* ?", " ", text)).groups()]
    N, T, H = 5, 64 * 700, 7
    places = T // 64 + N
    sizes = [(gla.gla_delta_workspace_bytes, 0), (gla.gla_delta_workspace_bytes, 1), (gla.gla_delta_bwd_workspace_bytes, 0),
             (gla.gla_delta_bwd_workspace_bytes, 1)]
    for (f, code), bytes_ in zip(sizes, stated):
        size, least = f(N, T, H, True, code), places * H * bytes_
        assert least <= size <= least + 256 + 4 * N + (48 * T * H if f is gla.gla_delta_bwd_workspace_bytes else 0), (f, code)
