"""The gated delta rule's calls and the slot plan through the debug-bounds build, whose kernels check their computed places
(sequences' rows and chunk places, the order, pool rows, tokens' places): no error, and the release build's results, on
ragged cases; and a host check that each of these kernels has such checks."""
import os
import re

import pytest
import torch

import linear_attention_recurrence_simple_gb300 as gla
from tests.delta_helpers import DK, DV, Batch
from tests.test_gpu_delta import i32, plan_inputs

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "linear_attention_recurrence_simple_gb300", "csrc")
CHECKS = r"GLA_IN_BOUNDS|\bdelta_seq\(|\bchunk_of_slot\(|\bdelta_unit\(|\btoken_place\("


def test_every_kernel_checks_its_places():
    shared = open(os.path.join(CSRC, "gla_delta.cuh")).read()
    for name in ("delta_seq", "chunk_of_slot", "delta_unit"):
        body = shared[re.search(r"inline__ \w+ " + name + r"\(", shared).start():]
        assert "GLA_IN_BOUNDS" in body[:body.index("\n}\n")], name
    found = 0
    for name in ("gla_delta_tc.cu", "gla_delta_simt.cu", "gla_delta_decode.cu", "gla_slot_plan.cu"):
        text = open(os.path.join(CSRC, name)).read()
        for part in re.split(r"__global__", text)[1:]:
            kernel = re.search(r"(\w+_kernel)\(", part).group(1)
            assert re.search(CHECKS, part[:part.index("\n}\n")]), kernel
            found += 1
    assert found == 11  # prep, scan, reverse scan and gradients twice; the decode step; the plan and its tokens


def through_both(fn):
    """fn() in the release build and in the debug-bounds build, where it must record nothing."""
    rel = fn()
    assert gla.gla_get_device_error() == 0
    with gla.debug_bounds_library():
        dbg = fn()
        err = gla.gla_get_device_error()
    assert err == 0, gla.gla_status_string(err)
    for x, y in zip(rel, dbg):
        assert torch.equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,spare", [([1], 0), ([0, 200, 1, 64, 0, 65, 130], 0), ([70, 3], 190), ([2] * 300, 5), ([128] * 9, 0)])
def test_packed_forward_and_backward(lens, spare, dtype):
    b = Batch(91, lens, 3, dtype, spare=spare)
    x, dO, used = b.inputs(), b.dev("dO")[0], sum(lens)
    N = len(lens)
    pool0 = torch.randn(N + 2, 3, DK, DV, generator=torch.Generator().manual_seed(92)).cuda()
    rows = torch.randperm(N + 2, generator=torch.Generator().manual_seed(93))[:N].tolist()

    def run():
        pool = pool0.clone()
        o, _ = gla.gla_delta_fwd(*x, h0=pool, h0_row=i32([r if n % 3 else -1 for n, r in enumerate(rows)]), hT=pool,
                                 hT_row=i32([r if n % 4 else -1 for n, r in enumerate(rows)]), cu_seqlens=b.cu_dev)
        return [o[:used], pool, *gla.gla_delta_bwd(*x, dO, h0=b.h0.cuda(), dhT=b.dhT.cuda(), cu_seqlens=b.cu_dev)]
    through_both(run)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,T", [(3, 65), (7, 1), (2, 256), (3, 0)])
def test_equal_lengths(N, T, dtype):
    b = Batch(94, [T] * N, 2, dtype, packed=False)
    x, dO, h0 = b.inputs(), b.dev("dO")[0], b.h0.cuda()
    through_both(lambda: [*gla.gla_delta_fwd(*x, h0=h0), *gla.gla_delta_bwd(*x, dO, h0=h0)])


@pytest.mark.gpu
@pytest.mark.parametrize("sdtype", [torch.bfloat16, torch.float32])
def test_decode(sdtype):
    b = Batch(95, [1] * 5, 3, torch.bfloat16)
    x, pool0 = b.inputs(), torch.randn(8, 3, DK, DV).to(sdtype).cuda()

    def run():
        a, c, o = pool0.clone(), pool0.clone(), torch.zeros(5, 3, DV, dtype=torch.bfloat16, device="cuda")
        return [gla.gla_delta_decode_step(*x, a, slot=i32([7, 0, -1, 3, 5]), o=o), a,
                gla.gla_delta_decode_step(*x, c, slot=i32([7, 0, 2, 3, 5]), start_row=i32([-1, 0, 1, 1, 6])), c]
    through_both(run)


@pytest.mark.gpu
@pytest.mark.parametrize("N,rows,budget", [(1, 1, 1), (64, 64, 4096), (9000, 700, 3000), (60000, 4096, 70000), (5, 40, 0)])
def test_plans(N, rows, budget):
    new, held, seen = (i32(x) for x in plan_inputs(96, N, rows))
    through_both(lambda: list(gla.gla_slot_plan(new, held, seen, rows, budget)))
