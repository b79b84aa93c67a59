"""How near the gated delta rule's calls come to the recurrence in 64 bits, held at what they are meant to keep (2-norm of
the error over that of the result).

An output of dtype bf16 is off by its own rounding at least: at most half a step, 2^-8 of a value at the low end of its
binade and 2^-9 at the high end, at random places in the step 1 / sqrt(3) of that in the mean square; 2^-8 x 0.72 (the rms over
a binade) / sqrt(3) = 1.6e-3.  One more rounding of that size on the way gives sqrt(2) of it, 2.3e-3, two give sqrt(3) of it,
2.8e-3: 2.5e-3 leaves room for one, and not for two; dg has two (the states before and after a chunk): 3e-3.  fp32 calls keep 22 bits of each operand, sums of 16 terms are cut off
in the tensor cores and the rest is fp32: 2^-22 x 0.72 / sqrt(3) = 1e-7 for each of the up to eight operands in a row, 3e-7 at
random signs, and the cut of 2^-23 a sum with a sign of its own, 1.2e-7 for each of up to three in a row: 6e-7 (long sums in
the tensor cores cut off ten times as often).  dg is what is left of three dot products (q . dq and two of k), each with an
error of its own: sqrt(3) of that, 1.05e-6.  States of bf16 calls: what is split into two bf16 (the state itself, and P in the
backward) keeps 2^-17 x 0.72 / sqrt(3) = 3.2e-6 of its part of the result, a quarter of it or less (what a chunk adds is made from
one state, of which it replaces a part), 0.8e-6; what is split into two fp16 2^-22; sums are cut off at 2^-23 three times
in a row, 0.3e-6 with a sign of its own: 1.5e-6 with room for few sequences."""
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
    return 1.5e-6 if name in ("hT", "dh0") else 3e-3 if name == "dg" else 2.5e-3


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


@pytest.mark.parametrize("size", [1e-25, 1e-8, 1e4, 1e20])
def test_values_of_other_sizes(size):
    """Everything is linear in (v, h0) and in (dO, dhT): sizes far outside fp16's range, or fp32's of squares, change nothing.
    (dbeta, dg and dk are products of both, so that one goes up as the other goes down.)"""
    b = Batch(104, LENS[:4], 3, BF)
    for name, by in (("v", size), ("dO", 1 / size)):
        b.x[name] = b.x[name] * by
    b.h0, b.dhT = b.h0 * size, b.dhT / size
    hold(b, bf16)


@pytest.mark.parametrize("what", ["outliers", "quiet", "silent", "keys", "states"])
def test_sizes_side_by_side(what):
    """Tokens of very different sizes in one chunk and from chunk to chunk: each bound that the kernels go by is far above most of
    what it bounds."""
    b = Batch(105, [400, 64, 130, 1], 2, BF)
    T = int(b.cu[-1])
    if what == "outliers":      # a few values a thousand times the others
        b.x["v"][::67] *= 1000
        b.x["dO"][5::71] *= 1000
    elif what == "quiet":       # large first, small after
        b.x["v"] *= torch.where(torch.arange(T) % 400 < 100, 1000.0, 1.0)[:, None, None]
    elif what == "silent":      # nothing is written: what there is comes from the first state
        b.x["v"][:] = 0
        b.x["v"][300:] = torch.randn(T - 300, 2, 192, generator=torch.Generator().manual_seed(6))
    elif what == "keys":        # lengths over five orders, writing strengths against them
        s = 10.0 ** (torch.arange(T) % 6 - 3.0)
        b.x["k"] *= s[:, None, None]
        b.x["beta"] /= (s * s)[:, None].clamp(min=1.0)
    else:                       # first states far above what is written
        b.h0, b.dhT = b.h0 * 1e5, b.dhT * 1e5
    # (where all of a gradient comes from S0, dS1 and dR, it has three roundings beside its own: sqrt(4) of 1.6e-3)
    hold(b, lambda name: bf16(name) if name in ("o", "hT", "dv", "dh0") or what not in ("keys", "states") else 3.3e-3)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", [1e-6, 1e-2, 1e3])
@pytest.mark.parametrize("gate", [-float("inf"), -100.0, -60.0])
def test_resets_with_keys_of_other_lengths(gate, size, dtype):
    """Resets and all but resets, at a chunk's first token, its last one and between, beside short and long keys: finite, and as
    near as elsewhere."""
    b = Batch(107, [200, 64, 65], 2, dtype)
    b.x["k"] *= size
    b.x["beta"] /= size * size
    b.x["g"][[0, 63, 64, 100, 200, 263, 264, 328], 0] = gate
    hold(b, bf16 if dtype == BF else lambda name: 2e-6)


@pytest.mark.parametrize("size", [1e3, 1e6])
@pytest.mark.parametrize("decay", [False, True])
def test_states_that_are_lost(decay, size):
    """First states (and, in the backward, last gradients) far above what comes beside them, which lose in a few hundred tokens what
    no decay says: a write takes out what stands under its key.  An error made in a chunk loses the same, so that each of up to 11
    chunks leaves the 1.5e-6 of one chunk's states, 1.65e-5 if all had one sign.
    With decay the state is lost within one chunk (head 0: e^-51), whose last tokens' residuals are small beside the bound that
    brings the chunk's to fp16: 10 of the largest element, 4.4 rms, of the state (unit keys), brought to 2^13 at least, where
    half of fp16's smallest step is 2^-38 of it.  With columns of K^ up to 2, sqrt(64) x 2 x 2^-38 x 44 / sqrt(96) = 2^-31.8 of the
    first state's norm, which is 2.7e-10.  (K^'s own smallest steps stand at tokens that the state had reached in full, but
    whose part decays away.)"""
    b = Batch(108, [700, 300, 64, 33], 2, BF)
    if not decay:
        b.x["g"][:] = 0
    b.h0, b.dhT = b.h0 * size, b.dhT * size
    got = outputs(b)
    out = {n: far(*got[n])[0] for n in ("hT", "dh0")}
    print({n: f"{x:.2e}" for n, x in out.items()})
    for n, first in (("hT", b.h0), ("dh0", b.dhT)):
        assert out[n] <= 1.65e-5 + 2.0 ** -31.8 * float(first.norm()) / float(got[n][1].norm()), (n, out)


@pytest.mark.parametrize("strength", ["usual", "one", "two"])
def test_long_sequences_without_decay(strength):
    """States over thousands of tokens that forget nothing: against the fp32 call on the same values, whose states are 6e-7 of
    the norm from the exact ones."""
    b = Batch(106, [6000, 3000], 1, BF)
    b.x["g"][:] = 0
    if strength != "usual":
        b.x["beta"][:] = 1.0 if strength == "one" else 1.9
    x, dO, cu = b.inputs(), b.dev("dO")[0], b.cu_dev
    wide = [t.float() for t in x]
    got = [*gla.gla_delta_fwd(*x, h0=b.h0.cuda(), cu_seqlens=cu), *gla.gla_delta_bwd(*x, dO, h0=b.h0.cuda(), dhT=b.dhT.cuda(), cu_seqlens=cu)]
    want = [*gla.gla_delta_fwd(*wide, h0=b.h0.cuda(), cu_seqlens=cu),
            *gla.gla_delta_bwd(*wide, dO.float(), h0=b.h0.cuda(), dhT=b.dhT.cuda(), cu_seqlens=cu)]
    errors = {n: far(g, w)[0] for n, g, w in zip(("o", "hT", *NAMES, "dh0"), got, want)}
    print({n: f"{x:.2e}" for n, x in errors.items()})
    # (what states have gathered over thousands of tokens outweighs what a chunk adds: as with first states above)
    # (a strength of 1.9 leaves 0.81 of the square of what stands under a key, one of 0.5 a quarter: errors live four times as long,
    # twice in the norm: 1.6e-3 and twice sqrt(3) of it)
    rest = 5.8e-3 if strength == "two" else 3.3e-3
    # (and a state that forgets nothing gathers the errors of 94 chunks, at random signs: 10 times a chunk's, of which a write
    # takes back its part)
    assert all(x <= (1.5e-5 if n in ("hT", "dh0") else bf16(n) if n in ("o", "dv") else rest) for n, x in errors.items())
