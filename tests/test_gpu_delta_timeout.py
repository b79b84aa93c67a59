"""The give-up paths of the gated delta rule's bf16 kernels, each of their waits in turn: in the debug-bounds build the
threads of a role are told to give up at a phase of an mbarrier, as if its limit had passed.  The other roles learn of
it through the CTA's flag; copies, products and stores in flight end, tensor memory is freed, the kernels return and
GLA_ERR_TIMEOUT is reported; the next calls give what they give without."""
import pytest
import torch

import linear_attention_recurrence_simple_gb300 as gla
from tests.delta_helpers import Batch

pytestmark = pytest.mark.gpu
TIMEOUT = -8
COPIES, PRODUCTS, ROWS = 0, 1, 2
PREP, SCAN, RSCAN, GRADS = 0, 1, 2, 3
# barriers by the order of the kernels' enumerations
A, C, O, KQ, V, KD, PH, SR, WR, OF, MX = range(11)  # scan
E0, E1, EF0, EF1, K, KR, RA, RC, Z, RSR, RWR, RDRAIN, ZF0, ZF1, GT0, GT1, X0, X1, MX0, MX1, QT = range(21)  # reverse scan
GKQ, IN0, IN1, FR0, FR1, MMA0, MMA1, ONE, EF, TWO = range(10)  # gradients

SCAN_WAITS = ([(COPIES, b, k) for b in (A, WR, C, O, V) for k in (0, 1, 3)] + [(COPIES, SR, 0), (PRODUCTS, MX, 0), (PRODUCTS, MX, 4)] +
              [(PRODUCTS, b, k) for b in (KQ, SR, KD, WR, PH) for k in (0, 1, 4)] + [(PRODUCTS, OF, k) for k in (0, 3)] +
              [(ROWS, b, k) for b in (V, A, C, O) for k in (0, 1, 4)])
RSCAN_WAITS = ([(COPIES, b, k) for b in (RA, RC, Z) for k in (0, 1, 4)] + [(COPIES, ZF0, 0), (COPIES, ZF1, 1)] +
               [(PRODUCTS, b, k) for b in (K, RSR, KR, RWR) for k in (0, 1, 4)] +
               [(PRODUCTS, b, k) for b, k in ((EF0, 0), (EF1, 0), (EF0, 2), (ZF0, 0), (ZF1, 1), (MX0, 0), (MX1, 1), (QT, 0), (QT, 4))] +
               [(ROWS, RSR, 0)] + [(ROWS, b, k) for b in (GT0, GT1, E0, E1, X0, X1, EF0, EF1) for k in (0, 1)] + [(ROWS, b, k) for b in (RA, RC, Z) for k in (0, 1, 4)])
GRADS_WAITS = ([(PRODUCTS, b, 0) for b in (IN0, IN1, FR0, FR1, MMA0, MMA1, EF)] + [(PRODUCTS, IN0, 1)] +
               [(ROWS, b, 0) for b in (IN0, IN1, GKQ, ONE, TWO)] + [(ROWS, IN0, 1)])


@pytest.fixture(scope="module")
def case():
    """Sequences of five chunks, of ragged ones, of one token and of none, more than fit on the GPU at a time."""
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    gla.load_library()
    b = Batch(81, [320, 300, 0, 1, 65, 64] * 8, 16, torch.bfloat16)
    x, dO, h0, dhT, cu = b.inputs(), b.dev("dO")[0], b.h0.cuda(), b.dhT.cuda(), b.cu_dev
    fwd = lambda: gla.gla_delta_fwd(*x, h0=h0, cu_seqlens=cu)  # noqa: E731
    bwd = lambda: gla.gla_delta_bwd(*x, dO, h0=h0, dhT=dhT, cu_seqlens=cu)  # noqa: E731
    out = {"fwd": (fwd, fwd()), "bwd": (bwd, bwd())}
    assert gla.gla_get_device_error() == 0
    return out


def gives_up(case, way, role, kernel, bar, k):
    call, want = case[way]
    with gla.debug_bounds_library():
        gla.gla_debug_give_up(role, kernel << 10 | bar << 5 | k)
        try:
            call()
            status = gla.gla_get_device_error()
        finally:
            gla.gla_debug_give_up(-1)
        assert status == TIMEOUT
        assert all(torch.equal(a, c) for a, c in zip(call(), want))
        assert gla.gla_get_device_error() == 0


@pytest.mark.parametrize("way", ["fwd", "bwd"])
def test_prep_gives_up(case, way):
    gives_up(case, way, ROWS, PREP, 0, 0)


@pytest.mark.parametrize("way", ["fwd", "bwd"])
@pytest.mark.parametrize("role,bar,k", SCAN_WAITS)
def test_scan_gives_up(case, role, bar, k, way):
    gives_up(case, way, role, SCAN, bar, k)


@pytest.mark.parametrize("role,bar,k", RSCAN_WAITS)
def test_reverse_scan_gives_up(case, role, bar, k):
    gives_up(case, "bwd", role, RSCAN, bar, k)


@pytest.mark.parametrize("role,bar,k", GRADS_WAITS)
def test_gradients_give_up(case, role, bar, k):
    gives_up(case, "bwd", role, GRADS, bar, k)


def test_a_phase_that_nobody_waits_for(case):
    for way, kernel, bar in (("fwd", SCAN, A), ("bwd", RSCAN, Z)):
        call, want = case[way]
        with gla.debug_bounds_library():
            gla.gla_debug_give_up(ROWS, kernel << 10 | bar << 5 | 31)
            try:
                got = call()
                assert gla.gla_get_device_error() == 0
            finally:
                gla.gla_debug_give_up(-1)
            assert all(torch.equal(a, c) for a, c in zip(got, want))
