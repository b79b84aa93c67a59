"""Host-only checks of the gated delta rule and of the slot plan: argument errors of the C ABI (before any CUDA call)
and of the binding, workspace sizes, and the tests' reference against differences."""
import ctypes

import pytest
import torch

import linear_attention_recurrence_simple_gb300 as gla
from tests.delta_helpers import DK, DV, ref_bwd, ref_fwd

OK, NULL, SHAPE, DTYPE, ALIGN, UNSUP, WS = 0, -1, -2, -3, -4, -5, -6
A, MIS = 0x10000, 0x10004  # fake device addresses, never dereferenced
GATES = ("g", "beta", "dg", "dbeta")  # aligned to their element
P = ctypes.c_void_p
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return gla.load_library()


def fwd(lib, q=A, k=A, v=A, g=A, beta=A, h0=A, h0_rows=9, h0_row=None, o=A, hT=A, hT_rows=9, hT_row=None, cu=None, n=3, T=7,
        H=2, dk=96, dv=192, dt=0, ws=A, wsb=BIG):
    return lib.gla_delta_fwd(P(q), P(k), P(v), P(g), P(beta), P(h0), h0_rows, P(h0_row), 0.1, P(o), P(hT), hT_rows,
                             P(hT_row), P(cu), n, T, H, dk, dv, dt, P(ws), wsb, None)


def bwd(lib, q=A, k=A, v=A, g=A, beta=A, h0=A, dO=A, dhT=A, dq=A, dk_=A, dv_=A, dg=A, dbeta=A, dh0=A, cu=None, n=3, T=7, H=2,
        dk=96, dv=192, dt=0, ws=A, wsb=BIG):
    return lib.gla_delta_bwd(P(q), P(k), P(v), P(g), P(beta), P(h0), 0.1, P(dO), P(dhT), P(dq), P(dk_), P(dv_), P(dg),
                             P(dbeta), P(dh0), P(cu), n, T, H, dk, dv, dt, P(ws), wsb, None)


def step(lib, bf16=False, q=A, k=A, v=A, g=A, beta=A, state=A, slot=None, rows=9, o=A, N=3, H=2, dk=96, dv=192, dt=0):
    f = lib.gla_delta_decode_step_bf16_state if bf16 else lib.gla_delta_decode_step
    return f(P(q), P(k), P(v), P(g), P(beta), 0.1, P(state), P(slot), rows, P(o), N, H, dk, dv, dt, None)


def plan(lib, new=A, held=A, seen=A, N=5, rows=9, budget=100, cu=A, slot=A, start=A, row=A, seq=A, pos=A):
    return lib.gla_slot_plan(P(new), P(held), P(seen), N, rows, budget, P(cu), P(slot), P(start), P(row), P(seq), P(pos), None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_chunked_argument_errors(lib, call):
    assert call(lib, dt=7) == DTYPE
    assert call(lib, dk=64) == UNSUP
    assert call(lib, dv=128) == UNSUP
    for kw in (dict(n=-1), dict(T=-1), dict(H=0), dict(n=2 ** 20, H=2 ** 10), dict(n=2 ** 16, T=2 ** 16)):
        assert call(lib, **kw) == SHAPE, kw
    assert call(lib, cu=A, n=3, T=2 ** 31 - 1, H=128) == SHAPE  # chunk places times heads
    assert call(lib, cu=A + 2) == ALIGN
    names = ["q", "k", "v", "g", "beta"] + (["o"] if call is fwd else ["dO", "dq", "dk_", "dv_", "dg", "dbeta"])
    for name in names:
        assert call(lib, **{name: None}) == NULL, name
    for name in names + ["h0"] + (["hT"] if call is fwd else ["dhT", "dh0"]):
        assert call(lib, **{name: A + 1 if name in GATES else MIS}) == ALIGN, name
    assert call(lib, ws=None) == WS
    assert call(lib, wsb=1000) == WS
    assert call(lib, ws=MIS) == ALIGN
    assert call(lib, n=0, q=None, ws=None) == OK


def test_forward_row_errors(lib):
    assert fwd(lib, h0_rows=2) == SHAPE                # three sequences, two rows, no map
    assert fwd(lib, hT_rows=2) == SHAPE
    assert fwd(lib, h0=None, h0_row=A) == NULL
    assert fwd(lib, hT=None, hT_row=A) == NULL
    assert fwd(lib, h0_row=A, h0_rows=-1) == SHAPE
    assert fwd(lib, h0_row=A + 2) == ALIGN
    assert fwd(lib, hT_row=A + 1) == ALIGN
    assert fwd(lib, hT_row=A, hT_rows=2 ** 24) == SHAPE


def test_decode_argument_errors(lib):
    for bf16 in (False, True):
        assert step(lib, bf16, dt=2) == DTYPE
        assert step(lib, bf16, dk=95) == UNSUP
        for kw in (dict(N=-1), dict(H=0), dict(rows=-1), dict(rows=2), dict(N=2 ** 30, slot=A)):
            assert step(lib, bf16, **kw) == SHAPE, kw
        for name in ("q", "k", "v", "g", "beta", "state", "o"):
            assert step(lib, bf16, **{name: None}) == NULL, name
            assert step(lib, bf16, **{name: A + 1 if name in GATES else MIS}) == ALIGN, name
        assert step(lib, bf16, slot=A + 2) == ALIGN
        assert step(lib, bf16, N=0, q=None) == OK


def test_plan_argument_errors(lib):
    for kw in (dict(N=-1), dict(rows=0), dict(budget=-1)):
        assert plan(lib, **kw) == SHAPE, kw
    assert plan(lib, rows=2 ** 19 + 1) == UNSUP
    assert plan(lib, N=2 ** 20 + 1) == UNSUP
    for name in ("new", "held", "cu", "slot", "start", "row", "seq", "pos"):
        assert plan(lib, **{name: None}) == NULL, name
    for name in ("new", "held", "seen", "cu", "slot", "start", "row", "seq", "pos"):
        assert plan(lib, **{name: A + 2}) == ALIGN, name


def test_workspace_bytes(lib):
    for f in (gla.gla_delta_workspace_bytes, gla.gla_delta_bwd_workspace_bytes):
        for packed in (False, True):
            for dt in (0, 1):
                sizes = [f(3, T, 4, packed, dt) for T in (0, 1, 64, 65, 1000, 100000)]
                assert sizes == sorted(sizes) and sizes[0] > 0
        assert f(-1, 5, 1, True, 0) == 0 and f(1, -1, 1, True, 0) == 0 and f(1, 1, 0, True, 0) == 0


def test_binding_refuses_host_tensors():
    x = [torch.zeros(1, 4, 2, d) for d in (DK, DK, DV)] + [torch.zeros(1, 4, 2)] * 2
    for call in (lambda: gla.gla_delta_fwd(*x), lambda: gla.gla_delta_bwd(*x, x[2]),
                 lambda: gla.gla_delta_decode_step(*[t[0] for t in x], torch.zeros(4, 2, DK, DV)),
                 lambda: gla.gla_slot_plan(torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), None, 4, 8)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_reference_against_differences():
    """The reference's gradients against central differences of the reference's forward, in 64 bits."""
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    L, H = 5, 2
    x = [r(L, H, DK) / 10, r(L, H, DK) / 10, r(L, H, DV), -r(L, H).abs(), torch.sigmoid(r(L, H)), r(H, DK, DV) * 0.1]
    dO, dS = r(L, H, DV), r(H, DK, DV)
    grads = ref_bwd(*x, dO, dS)

    def loss(y):
        o, S = ref_fwd(*y)
        return float((o * dO).sum() + (S * dS).sum())

    for i in range(6):
        d = r(*x[i].shape)
        e = 1e-5
        hi, lo = list(x), list(x)
        hi[i], lo[i] = x[i] + e * d, x[i] - e * d
        numeric, slope = (loss(hi) - loss(lo)) / (2 * e), float((grads[i] * d).sum())
        assert abs(numeric - slope) <= 1e-6 * (1 + float((grads[i] * d).norm())), i
