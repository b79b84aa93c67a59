"""Values far apart in the shared-prefix calls: infinities in MXFP8 tails, blocks with one element far
above the rest, queries and keys near the ends of the range.

An MXFP8 element's value is code x 2^(scale - 127) in fp32 (2^128 and more: an infinity), and the
decode step's result is the formula's on those values, whatever the elements beside it hold: the bounds
are those of tests/test_gpu_prefix.py, per entry, with M the sum of the magnitudes of that entry's own
terms."""
import numpy as np
import pytest
import torch

import glasynth as gs
import linear_attention_recurrence_simple_gb300 as gla
import oracle
from tests.prefix_helpers import DK, DV, SCALE, powers, ref_decode, ref_fold
from tests.test_gpu_prefix import Case, bits, i32, tol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    gla.load_library()
    yield
    assert gla.gla_get_device_error() == 0


def requantise(c, k, v):
    """The case's tails from these values (places that hold no token keep what they hold)."""
    (c.t.kc, c.t.ks), (c.t.vc, c.t.vs) = oracle.mxfp8_quantize(np.nan_to_num(k)), oracle.mxfp8_quantize(np.nan_to_num(v))
    c.t.k, c.t.v = oracle.mxfp8_dequantize(c.t.kc, c.t.ks), oracle.mxfp8_dequantize(c.t.vc, c.t.vs)
    c.t.spoil(c.slots, c.lens)
    c.tail = c.t.device()


def check_columns(c, o, keep=None):
    """The decode step's outputs against the 64-bit reference, where `keep` [N, H, 192] says so."""
    o = o.float().cpu().numpy().astype(np.float64)
    with np.errstate(all="ignore"):
        ref, mag = ref_decode(c.q, c.k, c.v, c.ll, SCALE, c.pool, c.rows, c.t.k, c.t.v, c.slots, c.lens)
        bound = tol(ref, mag, max(c.lens) + 2 * DK, c.bf16, c.bf16)
        bad = ~(np.abs(o - ref) <= bound)  # (a NaN is bad)
    if keep is not None:
        bad &= keep
    assert not bad.any(), (np.argwhere(bad)[:4].tolist(), [(o[tuple(i)], ref[tuple(i)], mag[tuple(i)]) for i in np.argwhere(bad)[:4]])


# ---- infinities --------------------------------------------------------------------------------
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("place", [0, 17, 70, 99])
def test_an_infinite_value_in_an_mxfp8_tail_stays_infinite(place, bf16):
    """Appended and quantised, read back as an infinity, and the decode step's column is the infinity of
    its weight's sign (weights of a few tenths); every other column is what it is without it."""
    lens, H, n, h, col = [100, 100, 37], 3, 1, 0, 40
    c = Case(900, lens, H, [0, 0, 1], 2, bf16, "mxfp8")
    c.k[:], c.v[:] = 0.0, 0.0                            # (the new tokens add nothing)
    for x in "kv":
        c.g[x].zero_()
    for sign in (1.0, -1.0):
        k, v = c.t.k[c.slots[n], :, place].copy(), c.t.v[c.slots[n], :, place].copy()
        v[h, col] = sign * np.inf
        kg, vg = (torch.from_numpy(x[None].astype(np.float32)).cuda().to(c.dt) for x in (k, v))
        gla.gla_tail_append(kg, vg, c.tail, i32([place]), i32([0, 1]), tail_slot=i32([c.slots[n]]))
        _, back = gla.gla_tail_read(c.tail, i32([place]), i32([0, 1]), 1, tail_slot=i32([c.slots[n]]), dtype=c.dt)
        assert float(back[0, h, col]) == sign * np.inf
        c.t.v[c.slots[n], h, place, 32:64] = 0.0         # (the infinity costs its block's other values)
        o = c.decode()
        x = c.t.k[c.slots[n], h, place] @ c.q[n, h].astype(np.float64) * powers(c.ll[h], lens[n] - place)
        assert 2.0 ** -40 < abs(x) < 0.57
        assert float(o[n, h, col]) == sign * np.sign(x) * np.inf
        keep = np.ones((3, H, DV), bool)
        keep[n, h, col] = False
        check_columns(c, o, keep)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("place", [0, 31, 64])
def test_an_infinite_key_in_an_mxfp8_tail_reaches_its_head_alone(place, bf16):
    """An infinite key element makes that token's weight infinite: every column of its head is an infinity
    or a NaN; other heads and sequences come out bit for bit as without it."""
    lens, H, n, h = [65, 80, 3], 3, 1, 0
    c = Case(910, lens, H, [0, 0, 0], 1, bf16, "mxfp8")
    clean = c.decode()
    k, v = c.t.k[c.slots[n], :, place].copy(), c.t.v[c.slots[n], :, place].copy()
    k[h, 70] = -np.inf
    kg, vg = (torch.from_numpy(x[None].astype(np.float32)).cuda().to(c.dt) for x in (k, v))
    gla.gla_tail_append(kg, vg, c.tail, i32([place]), i32([0, 1]), tail_slot=i32([c.slots[n]]))
    o = c.decode()
    assert not bool(torch.isfinite(o[n, h]).any())
    for i in range(3):
        for j in range(H):
            if (i, j) != (n, h):
                assert torch.equal(bits(o[i, j]), bits(clean[i, j])), (i, j)


def test_infinities_of_an_mxfp8_tail_in_the_fold():
    """The state of a tail with an infinite value has its column infinite or NaN, of one with an infinite
    key its row; everything else is what it is without them."""
    lens, H = [50, 40], 2
    c = Case(920, lens, H, [0, 1], 2, True, "mxfp8")
    # as the quantiser leaves a block with an infinity: code 448 under 2^120, the others zero
    for codes, scales, at, e, code in ((c.t.vc, c.t.vs, (c.slots[0], 0, 7), 40, 0x7E), (c.t.kc, c.t.ks, (c.slots[1], 1, 20), 33, 0xFE)):
        codes[at][32:64], scales[at][1] = 0, 247
        codes[at][e] = code
    c.t.k, c.t.v = oracle.mxfp8_dequantize(c.t.kc, c.t.ks), oracle.mxfp8_dequantize(c.t.vc, c.t.vs)
    c.tail = c.t.device()
    s = c.fold().cpu().numpy().astype(np.float64)
    with np.errstate(all="ignore"):
        ref, mag = ref_fold(c.ll, c.pool, c.rows, c.t.k, c.t.v, c.slots, c.lens)
        keep = np.ones(s.shape, bool)
        keep[0, 0, :, 40] = False
        keep[1, 1, 33, :] = False
        assert not np.isfinite(s[~keep]).any()
        assert np.all((np.abs(s - ref) <= tol(ref, mag, max(lens) + 2, True, False))[keep])


@pytest.mark.parametrize("bf16", [True, False])
def test_keys_and_values_near_the_top_of_the_range(bf16):
    """Keys of 2^118 against values of 2^-118, and a value of 2^126 whose own column overflows: no product
    on the way passes the range where the result does not."""
    lens, H = [40, 33, 70], 2
    c = Case(930, lens, H, [0, 1, 1], 2, bf16, "mxfp8")
    k, v = c.t.k.copy(), c.t.v.copy()
    k[c.slots[0]] *= 2.0 ** 118
    v[c.slots[0]] *= 2.0 ** -118
    k[c.slots[1]] *= 2.0 ** 20
    v[c.slots[1], :, 5, 70] = 2.0 ** 126
    requantise(c, k, v)
    o = c.decode()
    keep = np.ones((3, H, DV), bool)
    keep[1, :, 70] = False
    check_columns(c, o, keep)


# ---- one element far above the rest ------------------------------------------------------------
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("ratio", [16, 20, 24, 40, 90])
def test_a_value_far_above_its_block_leaves_the_other_columns_alone(ratio, bf16):
    """One element 2^ratio times the others in one token's value, early, late and twice: the tokens
    without it keep their weights' bits in the block's other 31 columns."""
    lens, H = [70, 8, 140, 40], 3
    c = Case(940 + ratio, lens, H, [0, 0, 1, 1], 2, bf16, "mxfp8")
    v = c.t.v.copy()
    for n, places in enumerate(([3], [6], [20, 120], [39])):
        for j in places:
            v[c.slots[n], :, j, 40] = 2.0 ** ratio
            v[c.slots[n], :, j, 191] = -(2.0 ** ratio)
    requantise(c, c.t.k, v)
    check_columns(c, c.decode())


@pytest.mark.parametrize("bf16", [True, False])
def test_tokens_whose_weights_are_far_apart(bf16):
    """Weights of one sequence spread over 2^60 by their keys, the large ones on tokens whose values are
    zero in most columns; and a head with lambda = 0.5."""
    lens, H = [64, 33, 90], 5
    c = Case(950, lens, H, [0, 1, 1], 2, bf16, "mxfp8")
    rng = np.random.default_rng(7)
    k, v = c.t.k.copy(), c.t.v.copy()
    e = rng.integers(-30, 31, k.shape[:3])
    k *= np.exp2(e)[..., None]
    v[e > -10] = 0.0
    v[..., 100] = 1.0                                    # (a column that has them all)
    requantise(c, k, v)
    check_columns(c, c.decode())


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("ratio", [20, 30, 60])
def test_a_query_element_far_above_the_rest_over_keys_without_it(ratio, bf16):
    """One element of q 2^ratio times the others, keys that are zero there: what the rest of q gives is
    all there is."""
    lens, H = [50, 20, 33], 2
    c = Case(960 + ratio, lens, H, [0, 1, 1], 2, bf16, "mxfp8")
    k = c.t.k.copy()
    k[..., 3] = 0.0
    requantise(c, k, c.t.v)
    c.q[:, :, 3] = 2.0 ** ratio
    c.k[:, :, 3] = 0.0
    c.pool[:, :, 3] = 0.0
    c.poolg = torch.from_numpy(c.pool).cuda()
    for x in "qk":
        c.g[x] = torch.from_numpy(getattr(c, x)).cuda().to(c.dt)
    check_columns(c, c.decode())


@pytest.mark.parametrize("bf16", [True, False])
def test_queries_of_zeros(bf16):
    c = Case(970, [40, 100, 7], 2, [0, 1, 1], 2, bf16, "mxfp8")
    c.q[:2] = 0.0
    c.g["q"][:2] = 0.0
    o = c.decode()
    assert bool((o[:2] == 0).all())
    check_columns(c, o)
