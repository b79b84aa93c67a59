"""Packed forward and backward from shared states where a CTA runs several (sequence, head, tile) units one
after another: many more units than SMs, with several chunks, odd chunk counts, partial last chunks and
empty sequences between them; past the most units that a CTA takes; and at the average length where the
launch goes over to one CTA per unit.

Against the oracle, and against gla_chunk_fwd and gla_chunk_bwd on copies of the states, which run one
CTA per unit: bit for bit, dq and dk within the order of their fp32 partial sums."""
import numpy as np
import pytest
import torch

import linear_attention_recurrence_simple_gb300 as gla
import oracle
from tests.gpu_helpers import BF16_TOL, F32_TOL, rel_err, within_one_bf16_rounding
from tests.prefix_helpers import SCALE
from tests.test_gpu_prefix import packed

pytestmark = pytest.mark.gpu

MIXED = [300, 0, 1, 127, 513, 128, 129, 0, 0, 385, 64, 256, 255, 257, 1, 640, 2, 0, 383, 130]
CASES = {
    # 480 units: the lengths mixed over them, empty sequences first, last and side by side
    "mixed": (MIXED, 8, [i % 3 for i in range(20)], 4, True),
    "mixed the other way": (MIXED[::-1] + [0], 8, [2 - i % 3 for i in range(21)], 3, True),
    # 5,760 units: more than 32 for each of 152 SMs
    "many short": ([(7 * i) % 41 for i in range(120)], 16, [i // 30 for i in range(120)], 4, True),
    # 168 units, at most and just above twelve chunks a sequence on average
    "twelve chunks": ([1536, 1537, 1408, 1664, 1536, 1535, 1536], 8, [0, 1, 0, 1, 1, 1, 0], 2, False),
    "above twelve chunks": ([1536, 1537, 1409, 1664, 1536, 1535, 1536], 8, [0, 1, 0, 1, 1, 1, 0], 2, False),
}


@pytest.fixture(scope="module", autouse=True)
def _setup():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    gla.load_library()
    yield
    assert gla.gla_get_device_error() == 0


@pytest.mark.parametrize("name", list(CASES))
def test_forward_over_many_units(name):
    lens, H, rows, P, with_oracle = CASES[name]
    d, g, rg = packed(800 + len(name), lens, H, rows, P, True)
    o, hT = gla.gla_prefix_fwd(g["q"], g["k"], g["v"], g["ll"], g["pool"], rg, g["cu"], SCALE)
    o2, hT2 = gla.gla_chunk_fwd(g["q"], g["k"], g["v"], g["ll"], SCALE, h0=g["pool"][rg.long()].contiguous(),
                                cu_seqlens=g["cu"])
    assert torch.equal(o, o2) and torch.equal(hT, hT2)
    if with_oracle:
        o_ref, hT_ref = oracle.fwd(d["q"], d["k"], d["v"], d["ll"], SCALE, h0=d["pool"][rows], cu_seqlens=d["cu"])
        assert rel_err(o.float().cpu().numpy(), o_ref, True) <= BF16_TOL
        assert rel_err(hT.cpu().numpy(), hT_ref) <= F32_TOL


@pytest.mark.parametrize("with_dhT", [True, False])
@pytest.mark.parametrize("name", list(CASES))
def test_backward_over_many_units(name, with_dhT):
    lens, H, rows, P, with_oracle = CASES[name]
    d, g, rg = packed(820 + len(name), lens, H, rows, P, True)
    dhT = g["dhT"] if with_dhT else None
    got = gla.gla_prefix_bwd(g["q"], g["k"], g["v"], g["ll"], g["dO"], g["pool"], rg, g["cu"], SCALE, dhT=dhT)
    plain = gla.gla_chunk_bwd(g["q"], g["k"], g["v"], g["ll"], g["dO"], SCALE, h0=g["pool"][rg.long()].contiguous(),
                              dhT=dhT, cu_seqlens=g["cu"])
    acc = torch.zeros_like(g["pool"])
    for n, r in enumerate(rows):
        acc[r] += plain[3][n]
    assert torch.equal(got[2], plain[2]) and torch.equal(got[3], acc)
    for i in (0, 1):
        assert within_one_bf16_rounding(got[i].float().cpu().numpy(), plain[i].float().cpu().numpy())
    if with_oracle:
        ref = oracle.bwd(d["q"], d["k"], d["v"], d["ll"], SCALE, d["dO"], h0=d["pool"][rows],
                         dhT=d["dhT"] if with_dhT else None, cu_seqlens=d["cu"])
        dpool_ref = np.zeros(d["pool"].shape)
        for n, r in enumerate(rows):
            dpool_ref[r] += ref[3][n]
        for x, y in zip(got[:3], ref[:3]):
            assert rel_err(x.float().cpu().numpy(), y, True) <= BF16_TOL
        assert rel_err(got[3].cpu().numpy(), dpool_ref) <= F32_TOL
