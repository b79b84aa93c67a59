"""Every shared-prefix call through the debug-bounds build, whose kernels check their computed accesses (tail
places, pool and output rows, packed rows): no error, and the release build's results and tails, on ragged
cases; and a host check that each of these kernels has such checks."""
import os
import re

import pytest
import torch

import linear_attention_recurrence_simple_gb300 as gla
from tests.gpu_helpers import within_one_bf16_rounding
from tests.prefix_helpers import DK, DV, SCALE
from tests.test_gpu_prefix import Case, bits, i32, packed

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "linear_attention_recurrence_simple_gb300", "csrc")


def test_every_kernel_of_the_tails_checks_its_indexes():
    found = 0
    for name in ("gla_prefix.cu", "gla_tail.cu"):
        text = open(os.path.join(CSRC, name)).read()
        parts = re.split(r"__global__", text)[1:]
        for part in parts:
            kernel = re.search(r"(\w+_kernel)\(", part).group(1)
            body = part[:part.index("\n}\n")]
            assert re.search(r"GLA_IN_BOUNDS|tail_in_bounds|state_in_bounds", body), kernel
            found += 1
    assert found == 6  # two decodes, the pool's gradient; the copies, two folds


def through_both(fn):
    """fn() in the release build and in the debug-bounds build, where it must record nothing."""
    rel = fn()
    assert gla.gla_get_device_error() == 0
    with gla.debug_bounds_library():
        dbg = fn()
        err = gla.gla_get_device_error()
    assert err == 0, gla.gla_status_string(err)
    return rel, dbg


LENS, H, ROWS = [0, 1, 33, 16, 65, 129, 40], 3, [1, 1, 0, 2, 2, 0, 0]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["native", "mxfp8"])
@pytest.mark.parametrize("bf16", [True, False])
def test_decode_and_fold(bf16, fmt):
    cases = [Case(980, LENS, H, ROWS, 3, bf16, fmt, cap=144) for _ in range(2)]
    it = iter(cases)

    def run():
        c = next(it)
        return [c.decode(), c.fold()] + [x for x in c.tail if x is not None]
    for x, y in zip(*through_both(run)):
        assert torch.equal(bits(x), bits(y))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["native", "mxfp8"])
@pytest.mark.parametrize("bf16", [True, False])
def test_append_and_read(bf16, fmt):
    cases = [Case(990, LENS, H, ROWS, 3, bf16, fmt, room=31) for _ in range(2)]
    it = iter(cases)
    T = sum(LENS)
    k, v = (torch.randn(T, H, d, device="cuda").to(cases[0].dt) for d in (DK, DV))
    cu = i32([sum(LENS[:i]) for i in range(len(LENS) + 1)])

    def run():
        c = next(it)
        pos = i32([c.cap - n for n in LENS])
        gla.gla_tail_append(k, v, c.tail, pos, cu, tail_slot=i32(c.slots))
        return list(gla.gla_tail_read(c.tail, pos, cu, T, tail_slot=i32(c.slots), dtype=c.dt)) + [x for x in c.tail if x is not None]
    for x, y in zip(*through_both(run)):
        assert torch.equal(bits(x), bits(y))


@pytest.mark.gpu
@pytest.mark.parametrize("bf16", [True, False])
def test_packed_forward_and_backward(bf16):
    d, g, rg = packed(995, LENS, H, ROWS, 4, bf16)

    def run():
        o = gla.gla_prefix_fwd(g["q"], g["k"], g["v"], g["ll"], g["pool"], rg, g["cu"], SCALE)
        return list(o) + list(gla.gla_prefix_bwd(g["q"], g["k"], g["v"], g["ll"], g["dO"], g["pool"], rg, g["cu"], SCALE,
                                                 dhT=g["dhT"]))
    for i, (x, y) in enumerate(zip(*through_both(run))):
        if bf16 and i in (2, 3):  # dq, dk: partial sums in arrival order
            assert within_one_bf16_rounding(x.float().cpu().numpy(), y.float().cpu().numpy())
        else:
            assert torch.equal(bits(x), bits(y))
