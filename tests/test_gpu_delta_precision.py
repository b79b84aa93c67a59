"""How near the gated delta rule's calls come to the recurrence in 64 bits, held at what they are meant to keep (2-norm of
the error over that of the result).

An output of dtype bf16 is off by its own rounding at least: at most half a step, 2^-8 of a value at the low end of its
binade and 2^-9 at the high end, at random places in the step 1 / sqrt(3) of that in the mean square; 2^-8 x 0.72 (the rms over
a binade) / sqrt(3) = 1.6e-3.  One more rounding of that size on the way gives sqrt(2) of it, 2.3e-3, two give sqrt(3) of it,
2.8e-3: 2.5e-3 leaves room for one, and not for two; dg has two (the states before and after a chunk): 3e-3.  fp32 calls keep 22 bits of each operand, sums of 16 terms are cut off
in the tensor cores and the rest is fp32: 2^-22 x 0.72 / sqrt(3) = 1e-7 for each of the up to eight operands in a row, 3e-7 at
random signs, and the cut of 2^-23 a sum with a sign of its own, 1.2e-7 for each of up to three in a row: 6e-7 (long sums in
the tensor cores cut off ten times as often).  dg is what is left of three dot products (q . dq and two of k), each with an
error of its own: sqrt(3) of that, 1.05e-6."""
import pytest
import torch

import linear_attention_recurrence_simple_gb300 as gla
from tests.delta_helpers import Batch, far

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAMES = ("dq", "dk", "dv", "dg", "dbeta")
LENS = [300, 64, 0, 190, 129]


@pytest.fixture(scope="module", autouse=True)
def _setup():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    gla.load_library()
    yield
    assert gla.gla_get_device_error() == 0


def outputs(b):
    """{name: (result, reference)} of a forward and a backward."""
    o, hT = gla.gla_delta_fwd(*b.inputs(), h0=b.h0.cuda(), cu_seqlens=b.cu_dev)
    grads = gla.gla_delta_bwd(*b.inputs(), *b.dev("dO"), h0=b.h0.cuda(), dhT=b.dhT.cuda(), cu_seqlens=b.cu_dev)
    f, r = [b.ref(n, b.h0[n]) for n in range(len(b.lens))], [b.ref_bwd(n, b.h0[n], b.dhT[n]) for n in range(len(b.lens))]
    out = {"o": (o, torch.cat([x[0] for x in f])), "hT": (hT, torch.stack([x[1] for x in f])),
           "dh0": (grads[5], torch.stack([x[5] for x in r]))}
    out.update({n: (grads[i], torch.cat([x[i] for x in r])) for i, n in enumerate(NAMES)})
    return out


def hold(b, bounds):
    out = {n: far(*x)[0] for n, x in outputs(b).items()}
    print({n: f"{x:.2e}" for n, x in out.items()})
    over = {n: x for n, x in out.items() if not x <= bounds(n)}
    assert not over, over


def bf16(name):
    return 2e-5 if name in ("hT", "dh0") else 3e-3 if name == "dg" else 2.5e-3


@pytest.mark.parametrize("seed", [101, 102])
def test_bf16(seed):
    hold(Batch(seed, LENS, 4, BF), bf16)


@pytest.mark.parametrize("seed", [101, 102])
def test_fp32(seed):
    hold(Batch(seed, LENS, 4, F32), lambda name: 1.05e-6 if name == "dg" else 6e-7)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size,beta", [(1.0, 2.0), (0.3, 2.0), (4.0, 0.1), (1e-3, 1.0), (300.0, 1e-5)])
def test_keys_of_other_lengths(size, beta, dtype):
    """Keys of no common length, the strength times their squared length up to 2."""
    b = Batch(103, LENS[:4], 3, dtype, unit=False)
    b.x["k"] = b.x["k"] * 30 / 96 ** 0.5 * size
    b.x["beta"] = b.x["beta"] * beta / max(1.0, size * size * beta / 1.6)
    hold(b, bf16 if dtype == BF else lambda name: 2e-6)
