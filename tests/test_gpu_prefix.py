"""GPU parity of the calls on sequences that continue a shared prefix: the decode step over shared
states and tails, the tails' writes and reads, the fold, and the packed forward and backward from
shared states.

Bounds.  With M the sum of the magnitudes of an entry's terms (in 64 bits, from the references):
  fp32 arithmetic over n terms: n 2^-23 M (a product and a sum, 2^-24 each), plus the weights
      lambda^j = expf(j log lambda): 2^-22 for expf and 2^-24 |j log lambda| for its argument, which
      stays below 104 where the weight is not zero: together (n + 110) 2^-23 M.
  bf16 calls: operands that are not bf16 (states, weighted keys, weights) may be held as the sum of two
      bf16 (each rounding half an ulp, 2^-8: together 2^-16 of the operand); products of two such
      operands do not occur, so 2^-15 M covers the split and its second-order terms.
  the rounding of a bf16 output: 2^-8 of its value.
The tails' contents are compared bit for bit."""
import threading

import numpy as np
import pytest
import torch

import glasynth as gs
import linear_attention_recurrence_simple_gb300 as gla
import oracle
from tests.gpu_helpers import BF16_TOL, F32_TOL, rel_err, within_one_bf16_rounding
from tests.prefix_helpers import DK, DV, SCALE, Tails, ref_decode, ref_fold

pytestmark = pytest.mark.gpu
SHAPE_ERR = -2


@pytest.fixture(scope="module", autouse=True)
def _setup():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    gla.load_library()
    yield
    assert gla.gla_get_device_error() == 0


def tol(ref, mag, terms, bf16, bf16_out):
    t = (terms + 110) * 2.0 ** -23 * mag
    if bf16:
        t = t + 2.0 ** -15 * mag
    return t + (2.0 ** -8 * np.abs(ref) if bf16_out else 0.0)


def lambdas(H):
    """log lambda of H heads: the schedule, with lambda = 1, 0 and 0.5 among them."""
    ll = gs.laplace_log_lambda(max(H, 2))[:H].astype(np.float32)
    for at, x in ((1, 0.0), (2, -np.inf), (4, np.log(0.5))):
        if at < H:
            ll[at] = x
    return ll


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


class Case:
    def __init__(self, seed, lens, H, rows, P, bf16, fmt, cap=None, spare=2, room=1):
        rng = np.random.default_rng(seed)
        N = len(lens)
        self.N, self.H, self.lens, self.rows, self.bf16, self.fmt = N, H, list(lens), list(rows), bf16, fmt
        self.cap = cap or max(16, -(-(max(lens, default=0) + room) // 16) * 16)
        self.R = N + spare
        self.slots = rng.permutation(self.R)[:N].tolist()
        self.t = Tails(seed, self.R, H, self.cap, fmt, bf16)
        self.t.spoil(self.slots, lens)
        self.ll = lambdas(H)
        self.pool = gs.normal(seed, 4, (P, H, DK, DV), 0.1)
        rnd = gs.bf16_round if bf16 else (lambda x: x)
        self.q, self.k = (rnd(gs.normal(seed, 5 + i, (N, H, DK), 1 / np.sqrt(DK))) for i in range(2))
        self.v = rnd(gs.normal(seed, 7, (N, H, DV)))
        self.dt = torch.bfloat16 if bf16 else torch.float32
        self.tail = self.t.device()
        self.g = {n: torch.from_numpy(getattr(self, n)).cuda().to(self.dt) for n in "qkv"}
        self.llg, self.poolg = torch.from_numpy(self.ll).cuda(), torch.from_numpy(self.pool).cuda()

    def decode(self, **kw):
        return gla.gla_prefix_decode_step(self.g["q"], self.g["k"], self.g["v"], self.llg, self.poolg, i32(self.rows),
                                          self.tail, i32(self.lens), tail_slot=i32(self.slots), scale=SCALE, **kw)

    def fold(self, **kw):
        return gla.gla_tail_fold(self.llg, self.poolg, i32(self.rows), self.tail, i32(self.lens),
                                 tail_slot=i32(self.slots), **kw)

    def written(self):
        """The tails as the decode step leaves them, on the host."""
        out = [x.clone() for x in self.t.device("cpu") if x is not None]
        for n, (s, L) in enumerate(zip(self.slots, self.lens)):
            if self.fmt == "mxfp8":
                new = [torch.from_numpy(x) for x in (*oracle.mxfp8_quantize(self.k[n]), *oracle.mxfp8_quantize(self.v[n]))]
                new = [new[0], new[2], new[1], new[3]]
            else:
                new = [torch.from_numpy(self.k[n]).to(self.dt), torch.from_numpy(self.v[n]).to(self.dt)]
            for a, b in zip(out, new):
                a[s, :, L] = b
        return out


def bits(x):
    return x.view(torch.int16) if x.dtype == torch.bfloat16 else x.view(torch.int32) if x.dtype == torch.float32 else x


def same_tails(tail, want):
    for x, y in zip([x for x in tail if x is not None], want):
        differ = (bits(x.cpu()) != bits(y)).nonzero()
        assert differ.numel() == 0, differ[:4].tolist()


def check_decode(c, o=None):
    o = (c.decode() if o is None else o).float().cpu().numpy().astype(np.float64)
    ref, mag = ref_decode(c.q, c.k, c.v, c.ll, SCALE, c.pool, c.rows, c.t.k, c.t.v, c.slots, c.lens)
    terms = (max(c.lens, default=0) + DK + DK)
    bad = np.abs(o - ref) > tol(ref, mag, terms, c.bf16, c.bf16)
    assert not bad.any(), (np.argwhere(bad)[:4].tolist(), np.nanmax(np.abs(o - ref) / np.maximum(mag, 1e-30)))
    assert np.isfinite(o).all()


# (lens, H, rows, P): empty and one-token tails; lengths around 16 and 32; one prefix for all, one
# each, runs that end inside a group of 16, rows that return; more heads than a power of two
DECODE = [
    ([0], 1, [0], 1),
    ([1], 2, [2], 3),
    ([0, 1, 2, 15, 16, 17, 31, 32, 33], 3, [1] * 9, 2),
    ([5, 0, 64], 5, [2, 0, 1], 3),
    (list(range(0, 37)), 2, [0] * 20 + [3] * 16 + [1], 4),
    ([7, 9, 8, 3, 0, 12, 40], 7, [1, 0, 1, 1, 0, 0, 1], 2),
    ([100, 255, 0, 129, 200, 96, 97, 191, 193], 3, [0] * 5 + [1] * 4, 2),
    ([600, 1], 2, [0, 0], 1),
    ([3] * 70, 1, [0] * 33 + [1] * 37, 2),
]


@pytest.mark.parametrize("fmt", ["native", "mxfp8"])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("case", range(len(DECODE)))
def test_decode(case, bf16, fmt):
    lens, H, rows, P = DECODE[case]
    c = Case(100 + case, lens, H, rows, P, bf16, fmt)
    check_decode(c)
    same_tails(c.tail, c.written())


@pytest.mark.parametrize("fmt", ["native", "mxfp8"])
def test_decode_at_the_last_place_and_default_rows(fmt):
    """Tails one token short of full; no slots (row n) and the default scale."""
    c = Case(150, [31, 31, 0], 2, [0, 0, 0], 1, True, fmt, cap=32, spare=0)
    c.slots = [0, 1, 2]
    c.t = Tails(150, 3, 2, 32, fmt, True)
    c.tail = c.t.device()
    o = gla.gla_prefix_decode_step(c.g["q"], c.g["k"], c.g["v"], c.llg, c.poolg, i32(c.rows), c.tail, i32(c.lens))
    check_decode(c, o)
    same_tails(c.tail, c.written())


@pytest.mark.parametrize("fmt", ["native", "mxfp8"])
@pytest.mark.parametrize("bf16", [True, False])
def test_decode_skips_bad_sequences(bf16, fmt):
    """Sequences with a row, a slot or a length out of range are skipped (output and tails as they
    were) and reported; the others come out as they should."""
    lens = [3, 20, 33, 5, 6, 7, 8, 9]
    c = Case(160, lens, 2, [0] * 8, 2, bf16, fmt, cap=48)
    before = [x.clone().cpu() for x in c.tail if x is not None]
    rows, slots, bad_lens = list(c.rows), list(c.slots), list(lens)
    rows[1], rows[2] = 2, -1
    slots[3], slots[4] = c.R, -5
    bad_lens[5], bad_lens[6] = 48, -1
    o = torch.full((8, 2, DV), 7.0, device="cuda", dtype=c.dt)
    gla.gla_prefix_decode_step(c.g["q"], c.g["k"], c.g["v"], c.llg, c.poolg, i32(rows), c.tail, i32(bad_lens),
                               tail_slot=i32(slots), scale=SCALE, o=o)
    assert gla.gla_get_device_error() == SHAPE_ERR
    assert bool((o[1:7] == 7.0).all())
    good = [0, 7]
    ref, mag = ref_decode(c.q[good], c.k[good], c.v[good], c.ll, SCALE, c.pool, [0, 0], c.t.k, c.t.v,
                          [c.slots[i] for i in good], [lens[i] for i in good])
    got = o[good].float().cpu().numpy()
    assert np.all(np.abs(got - ref) <= tol(ref, mag, 40 + 2 * DK, bf16, bf16))
    want = c.written()
    for i in range(1, 7):  # the skipped ones' rows
        for x, y in zip(want, before):
            x[c.slots[i]] = y[c.slots[i]]
    same_tails(c.tail, want)


@pytest.mark.parametrize("fmt", ["native", "mxfp8"])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("case", range(len(DECODE)))
def test_fold(case, bf16, fmt):
    lens, H, rows, P = DECODE[case]
    c = Case(200 + case, lens, H, rows, P, bf16, fmt)
    s = c.fold().cpu().numpy().astype(np.float64)
    ref, mag = ref_fold(c.ll, c.pool, c.rows, c.t.k, c.t.v, c.slots, c.lens)
    bad = np.abs(s - ref) > tol(ref, mag, max(lens) + 2, bf16 or fmt == "mxfp8", False)
    assert not bad.any(), (np.argwhere(bad)[:4].tolist(), np.max(np.abs(s - ref) / np.maximum(mag, 1e-30)))


@pytest.mark.parametrize("bf16", [True, False])
def test_fold_into_pool_rows(bf16):
    """Into chosen rows of the pool itself: other rows stay, and one sequence is folded into the row
    that it alone continues."""
    c = Case(230, [20, 5, 130], 3, [1, 1, 3], 6, bf16, "native")
    before = c.poolg.clone()
    c.fold(out=c.poolg, out_row=i32([5, 0, 3]))
    ref, mag = ref_fold(c.ll, c.pool, c.rows, c.t.k, c.t.v, c.slots, c.lens)
    for i, r in enumerate([5, 0, 3]):
        s = c.poolg[r].cpu().numpy()
        assert np.all(np.abs(s - ref[i]) <= tol(ref[i], mag[i], 140, bf16, False))
    for r in (1, 2, 4):
        assert torch.equal(c.poolg[r], before[r])


def test_fold_skips_bad_sequences():
    c = Case(240, [20, 5, 9, 4, 6], 2, [0, 0, 0, 0, 0], 1, True, "mxfp8", cap=32)
    out = torch.full((5, 2, DK, DV), 3.0, device="cuda")
    gla.gla_tail_fold(c.llg, c.poolg, i32([0, 1, 0, 0, 0]), c.tail, i32([20, 5, 33, 4, 6]),
                      tail_slot=i32(c.slots[:3] + [99, c.slots[4]]), out=out, out_row=i32([0, 1, 2, 3, 5]))
    assert gla.gla_get_device_error() == SHAPE_ERR
    assert bool((out[1:] == 3.0).all())
    ref, mag = ref_fold(c.ll, c.pool, c.rows[:1], c.t.k, c.t.v, c.slots[:1], c.lens[:1])
    assert np.all(np.abs(out[:1].cpu().numpy() - ref) <= tol(ref, mag, 22, True, False))


@pytest.mark.parametrize("fmt", ["native", "mxfp8"])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("lens", [[1], [0, 3, 64, 1, 65, 0, 130], [1] * 40, [1, 0, 2] * 400])
def test_append_and_read(lens, bf16, fmt):
    """Written places hold the tokens (quantised bit for bit as the oracle does), the others are
    untouched; the read gives the values back exactly, rows behind the last sequence left alone."""
    N, H, extra = len(lens), 3, 5
    c = Case(300 + N, lens, H, [0] * N, 1, bf16, fmt, room=9)
    T = sum(lens)
    rnd = gs.bf16_round if bf16 else (lambda x: x)
    k, v = rnd(gs.normal(300, 1, (T + extra, H, DK), 0.1)), rnd(gs.normal(300, 2, (T + extra, H, DV)))
    k[0, 0, :32] = 0.0                                   # an all-zero block
    v[0, 0, :32] *= 2.0 ** -130                          # a block of tiny values
    if bf16:
        v = gs.bf16_round(v)
    pos = [c.cap - n if i % 2 else (c.cap - n) // 2 for i, n in enumerate(lens)]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    want = [x.clone().cpu() for x in c.tail if x is not None]
    kg, vg = torch.from_numpy(k).cuda().to(c.dt), torch.from_numpy(v).cuda().to(c.dt)
    gla.gla_tail_append(kg, vg, c.tail, i32(pos), i32(cu), tail_slot=i32(c.slots))
    vals = []
    if fmt == "mxfp8":
        (kc, ks), (vc, vs) = oracle.mxfp8_quantize(k), oracle.mxfp8_quantize(v)
        vals = [oracle.mxfp8_dequantize(kc, ks), oracle.mxfp8_dequantize(vc, vs)]
        new = [torch.from_numpy(x) for x in (kc, vc, ks, vs)]
    else:
        vals = [k, v]
        new = [kg.cpu(), vg.cpu()]
    for i in range(N):
        for a, b in zip(want, new):
            a[c.slots[i], :, pos[i]:pos[i] + lens[i]] = b[cu[i]:cu[i + 1]].transpose(0, 1)
    same_tails(c.tail, want)
    ko = torch.full((T + extra, H, DK), 9.0, device="cuda", dtype=c.dt)
    vo = torch.full((T + extra, H, DV), 9.0, device="cuda", dtype=c.dt)
    gla.gla_tail_read(c.tail, i32(pos), i32(cu), T + extra, tail_slot=i32(c.slots), k=ko, v=vo)
    for got, val in ((ko, vals[0]), (vo, vals[1])):
        ref = torch.from_numpy(val[:T]).to(c.dt)
        assert torch.equal(got[:T].cpu(), ref)
        assert bool((got[T:] == 9.0).all())


def test_append_skips_bad_sequences():
    lens = [4, 4, 4, 4]
    c = Case(340, lens, 2, [0] * 4, 1, True, "mxfp8", cap=16)
    before = [x.clone() for x in c.tail]
    T = sum(lens)
    k, v = torch.ones(T, 2, DK, device="cuda", dtype=c.dt), torch.ones(T, 2, DV, device="cuda", dtype=c.dt)
    slots = list(c.slots)
    slots[1] = 77
    gla.gla_tail_append(k, v, c.tail, i32([13, 0, -1, 2]), i32([0, 4, 8, 12, 16]), tail_slot=i32(slots))
    assert gla.gla_get_device_error() == SHAPE_ERR
    for x, y in zip(c.tail, before):
        y[c.slots[3], :, 2:6] = x[c.slots[3], :, 2:6]
        assert torch.equal(x, y)
    assert bool((c.tail.k[c.slots[3], :, 2:6].view(torch.float8_e4m3fn).float() == 256.0).all())
    # offsets that decrease or pass the total: no access outside, and an error
    gla.gla_tail_append(k, v, c.tail, i32([0, 0, 0]), i32([0, 12, 4, 40]), tail_slot=i32(c.slots[:3]))
    assert gla.gla_get_device_error() == SHAPE_ERR


# ---- packed forward and backward from shared states -------------------------------------------
PACKED = [([200, 0, 1, 128, 129, 33], 3, [1, 0, 1, 1, 2, 0], 4), ([64], 2, [0], 1), ([5] * 40, 2, [3] * 25 + [0] * 15, 5)]


def packed(seed, lens, H, rows, P, bf16):
    rnd = gs.bf16_round if bf16 else (lambda x: x)
    T = sum(lens)
    d = {"q": rnd(gs.normal(seed, 1, (T, H, DK), 1 / np.sqrt(DK))), "k": rnd(gs.normal(seed, 2, (T, H, DK), 1 / np.sqrt(DK))),
         "v": rnd(gs.normal(seed, 3, (T, H, DV))), "dO": rnd(gs.normal(seed, 5, (T, H, DV))),
         "pool": gs.normal(seed, 4, (P, H, DK, DV), 0.1), "dhT": gs.normal(seed, 6, (len(lens), H, DK, DV), 0.01),
         "ll": gs.laplace_log_lambda(max(H, 2))[:H].astype(np.float32), "cu": gs.cu_seqlens_of(lens)}
    dt = torch.bfloat16 if bf16 else torch.float32
    g = {n: torch.from_numpy(x).cuda().to(dt) if n in ("q", "k", "v", "dO") else torch.from_numpy(x).cuda()
         for n, x in d.items()}
    return d, g, i32(rows)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("case", range(len(PACKED)))
def test_packed_forward(case, bf16):
    lens, H, rows, P = PACKED[case]
    d, g, rg = packed(400 + case, lens, H, rows, P, bf16)
    o, hT = gla.gla_prefix_fwd(g["q"], g["k"], g["v"], g["ll"], g["pool"], rg, g["cu"], SCALE)
    o_ref, hT_ref = oracle.fwd(d["q"], d["k"], d["v"], d["ll"], SCALE, h0=d["pool"][rows], cu_seqlens=d["cu"])
    bar = BF16_TOL if bf16 else F32_TOL
    assert rel_err(o.float().cpu().numpy(), o_ref, bf16) <= bar
    assert rel_err(hT.cpu().numpy(), hT_ref) <= F32_TOL  # the state path holds about 16 bits in bf16 calls
    # the same kernels from copies of the states: bit for bit
    o2, hT2 = gla.gla_chunk_fwd(g["q"], g["k"], g["v"], g["ll"], SCALE, h0=g["pool"][rg.long()].contiguous(),
                                cu_seqlens=g["cu"])
    assert torch.equal(o, o2) and torch.equal(hT, hT2)


@pytest.mark.parametrize("with_dhT", [True, False])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("case", range(len(PACKED)))
def test_packed_backward(case, bf16, with_dhT):
    lens, H, rows, P = PACKED[case]
    d, g, rg = packed(420 + case, lens, H, rows, P, bf16)
    dhT = g["dhT"] if with_dhT else None
    got = gla.gla_prefix_bwd(g["q"], g["k"], g["v"], g["ll"], g["dO"], g["pool"], rg, g["cu"], SCALE, dhT=dhT)
    ref = oracle.bwd(d["q"], d["k"], d["v"], d["ll"], SCALE, d["dO"], h0=d["pool"][rows],
                     dhT=d["dhT"] if with_dhT else None, cu_seqlens=d["cu"])
    bar = BF16_TOL if bf16 else F32_TOL
    for x, y in zip(got[:3], ref[:3]):
        assert rel_err(x.float().cpu().numpy(), y, bf16) <= bar
    dpool_ref = np.zeros(d["pool"].shape)
    for n, r in enumerate(rows):
        dpool_ref[r] += ref[3][n]
    assert rel_err(got[3].cpu().numpy(), dpool_ref) <= F32_TOL
    # dh0 of the plain backward from copies of the states, added up in the sequences' order
    plain = gla.gla_chunk_bwd(g["q"], g["k"], g["v"], g["ll"], g["dO"], SCALE, h0=g["pool"][rg.long()].contiguous(),
                              dhT=dhT, cu_seqlens=g["cu"])
    acc = torch.zeros_like(g["pool"])
    for n, r in enumerate(rows):
        acc[r] += plain[3][n]
    assert torch.equal(got[3], acc)
    assert torch.equal(got[2], plain[2])
    for i in (0, 1):
        if bf16:
            assert within_one_bf16_rounding(got[i].float().cpu().numpy(), plain[i].float().cpu().numpy())
        else:
            assert torch.equal(got[i], plain[i])
    none = gla.gla_prefix_bwd(g["q"], g["k"], g["v"], g["ll"], g["dO"], g["pool"], rg, g["cu"], SCALE, dhT=dhT,
                              need_dpool=False)
    assert none[3] is None and torch.equal(none[2], got[2])


def test_packed_gradients_against_differences():
    """L = sum(o * dO) + sum(hT * dhT) in fp32 calls: L is linear in the pool, in v and in q, so
    (L(x + d) - L(x - d)) / 2 = <dL/dx, d> for a step d of any size.  Both sides are sums of m = T H 192
    + n H 96 192 rounded products taken in 64 bits; an fp32 output carries at most 2^-20 of the
    magnitude of its terms, so 2^-18 of the sum of |terms| bounds the difference."""
    lens, H, rows, P = PACKED[0]
    d, g, rg = packed(440, lens, H, rows, P, False)

    def out(**kw):
        x = dict(g, **kw)
        o, hT = gla.gla_prefix_fwd(x["q"], x["k"], x["v"], x["ll"], x["pool"], rg, x["cu"], SCALE)
        t = (o.double() * g["dO"].double()), (hT.double() * g["dhT"].double())
        return float(t[0].sum() + t[1].sum()), float(t[0].abs().sum() + t[1].abs().sum())

    dq, dk, dv, dpool = gla.gla_prefix_bwd(g["q"], g["k"], g["v"], g["ll"], g["dO"], g["pool"], rg, g["cu"], SCALE,
                                           dhT=g["dhT"])
    for name, grad in (("pool", dpool), ("v", dv), ("q", dq)):
        step = torch.from_numpy(gs.normal(441, 1, tuple(grad.shape), 0.5)).cuda()
        (a, ma), (b, mb) = out(**{name: g[name] + step}), out(**{name: g[name] - step})
        want = float((grad.double() * step.double()).sum())
        assert abs((a - b) / 2 - want) <= 2.0 ** -18 * (ma + mb), name


def test_packed_calls_report_bad_rows():
    """A pool row out of range: that sequence starts from zeros, takes no part in the pool's gradient,
    and the error is recorded."""
    lens, H, rows, P = [40, 30, 20], 2, [0, 7, -1], 2
    d, g, _ = packed(450, lens, H, rows, P, True)
    o, hT = gla.gla_prefix_fwd(g["q"], g["k"], g["v"], g["ll"], g["pool"], i32(rows), g["cu"], SCALE)
    assert gla.gla_get_device_error() == SHAPE_ERR
    h0 = np.stack([d["pool"][0], np.zeros_like(d["pool"][0]), np.zeros_like(d["pool"][0])])
    o_ref, hT_ref = oracle.fwd(d["q"], d["k"], d["v"], d["ll"], SCALE, h0=h0, cu_seqlens=d["cu"])
    assert rel_err(o.float().cpu().numpy(), o_ref, True) <= BF16_TOL
    got = gla.gla_prefix_bwd(g["q"], g["k"], g["v"], g["ll"], g["dO"], g["pool"], i32(rows), g["cu"], SCALE)
    assert gla.gla_get_device_error() == SHAPE_ERR
    assert bool((got[3][1] == 0).all()) and bool((got[3][0] != 0).any())


def test_empty_calls():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    pool, ll, cu = z(3, 2, DK, DV, dt=torch.float32), z(2, dt=torch.float32), i32([0])
    none = i32([])
    t = gla.gla_tail_alloc(1, 2, 16)
    assert gla.gla_prefix_decode_step(z(0, 2, DK), z(0, 2, DK), z(0, 2, DV), ll, pool, none, t, none).shape == (0, 2, DV)
    assert gla.gla_tail_fold(ll, pool, none, t, none).shape == (0, 2, DK, DV)
    gla.gla_tail_append(z(0, 2, DK), z(0, 2, DV), t, none, cu)
    assert gla.gla_tail_read(t, none, cu, 0)[0].shape == (0, 2, DK)
    o, hT = gla.gla_prefix_fwd(z(0, 2, DK), z(0, 2, DK), z(0, 2, DV), ll, pool, none, cu)
    assert hT.shape == (0, 2, DK, DV)
    dpool = torch.ones_like(pool)
    gla.gla_prefix_bwd(z(0, 2, DK), z(0, 2, DK), z(0, 2, DV), ll, z(0, 2, DV), pool, none, cu, dpool=dpool)
    assert bool((dpool == 0).all())  # nobody continues any row
    # sequences without tokens: hT is the shared state, its gradient dhT
    pool.normal_()
    rows, cu = i32([2, 2]), i32([0, 0, 0])
    for dt in (torch.bfloat16, torch.float32):
        e = [z(0, 2, d, dt=dt) for d in (DK, DK, DV, DV)]
        _, hT = gla.gla_prefix_fwd(*e[:3], ll, pool, rows, cu)
        assert torch.equal(hT, pool[rows.long()])
        dhT = torch.randn_like(hT)
        got = gla.gla_prefix_bwd(*e[:3], ll, e[3], pool, rows, cu, dhT=dhT)
        assert torch.equal(got[3][2], dhT[0] + dhT[1]) and bool((got[3][:2] == 0).all())


# ---- together, as they are used ---------------------------------------------------------------
@pytest.mark.parametrize("fmt", ["native", "mxfp8"])
def test_sampling_from_shared_prompts(fmt):
    """Two prompts run once; five continuations of them decode 40 tokens over the shared states, the
    first few tokens of each given as a prompt suffix; then the tails are folded and each goes on
    with a state of its own.  Against the oracle's recurrence token by token (fp64 states)."""
    H, P, N, steps = 4, 2, 5, 40
    rows, suffix = [0, 0, 0, 1, 1], [0, 3, 17, 1, 33]
    ll = gs.laplace_log_lambda(H).astype(np.float32)
    llg = torch.from_numpy(ll).cuda()
    dt = torch.bfloat16

    def rnd(seed, *shape, sigma=0.1):
        return gs.bf16_round(gs.normal(seed, 9, shape, sigma))

    def dev(x):
        return torch.from_numpy(x).cuda().to(dt)
    # the prompts, once
    lens = [150, 77]
    k, v = rnd(500, sum(lens), H, DK), rnd(501, sum(lens), H, DV, sigma=1.0)
    cu = gs.cu_seqlens_of(lens)
    _, pool = gla.gla_chunk_fwd(dev(k), dev(k), dev(v), llg, SCALE, cu_seqlens=torch.from_numpy(cu).cuda())
    _, pool_ref = oracle.fwd(k, k, v, ll, SCALE, cu_seqlens=cu)
    state = pool_ref[rows].copy()
    # the suffixes: outputs from the shared states, keys and values to the tails
    Ts = sum(suffix)
    q, k, v = rnd(502, Ts, H, DK), rnd(503, Ts, H, DK), rnd(504, Ts, H, DV, sigma=1.0)
    cu = gs.cu_seqlens_of(suffix)
    cug, rg = torch.from_numpy(cu).cuda(), i32(rows)
    tail = gla.gla_tail_alloc(N, H, 80, torch.float8_e4m3fn if fmt == "mxfp8" else dt)
    length = torch.zeros(N, dtype=torch.int32, device="cuda")
    o, _ = gla.gla_prefix_fwd(dev(q), dev(k), dev(v), llg, pool, rg, cug, SCALE)
    gla.gla_tail_append(dev(k), dev(v), tail, length, cug)
    length += i32(suffix)
    o_ref, _ = oracle.fwd(q, k, v, ll, SCALE, h0=state, cu_seqlens=cu)
    assert rel_err(o.float().cpu().numpy(), o_ref, True) <= BF16_TOL
    deq = lambda x: oracle.mxfp8_dequantize(*oracle.mxfp8_quantize(x)) if fmt == "mxfp8" else x  # noqa: E731
    _, state = oracle.fwd(q, deq(k), deq(v), ll, SCALE, h0=state, cu_seqlens=cu)
    for t in range(steps):
        q, k, v = rnd(600 + 3 * t, N, H, DK), rnd(601 + 3 * t, N, H, DK), rnd(602 + 3 * t, N, H, DV, sigma=1.0)
        o = gla.gla_prefix_decode_step(dev(q), dev(k), dev(v), llg, pool, rg, tail, length, scale=SCALE)
        length += 1
        after = state.copy()
        o_ref = oracle.decode_step(q, k, v, ll, SCALE, after)
        assert rel_err(o.float().cpu().numpy(), o_ref, True) <= BF16_TOL
        # what later tokens see of this one is what the tail holds
        oracle.decode_step(q, deq(k), deq(v), ll, SCALE, state)
    own = gla.gla_tail_fold(llg, pool, rg, tail, length)
    assert rel_err(own.cpu().numpy(), state) <= F32_TOL
    q, k, v = rnd(700, N, H, DK), rnd(701, N, H, DK), rnd(702, N, H, DV, sigma=1.0)
    o = gla.gla_decode_step(dev(q), dev(k), dev(v), llg, own, SCALE)
    assert rel_err(o.float().cpu().numpy(), oracle.decode_step(q, k, v, ll, SCALE, state), True) <= BF16_TOL


@pytest.mark.parametrize("fmt", ["native", "mxfp8"])
def test_captured_decode_replays_as_it_runs(fmt):
    """A step captured into a graph (with the advance of the lengths), replayed on new inputs, gives
    the eager calls' outputs and tails bit for bit; on a stream that is not the default."""
    c = Case(520, [0, 5, 16, 40, 7, 31], 3, [0, 0, 1, 1, 1, 1], 2, True, fmt, cap=64)
    other = c.t.device()
    rows, slots = i32(c.rows), i32(c.slots)
    len_a, len_b = i32(c.lens), i32(c.lens)
    x = {n: torch.empty_like(y) for n, y in c.g.items()}
    o_b = torch.empty(c.N, c.H, DV, device="cuda", dtype=c.dt)
    for n in "qkv":
        x[n].copy_(c.g[n])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        gla.gla_prefix_decode_step(x["q"], x["k"], x["v"], c.llg, c.poolg, rows, other, len_b, tail_slot=slots,
                                   scale=SCALE, o=o_b)
        len_b += 1
    for step in range(4):
        new = {n: (y * (1 + step)).contiguous() for n, y in c.g.items()}
        o_a = gla.gla_prefix_decode_step(new["q"], new["k"], new["v"], c.llg, c.poolg, rows, c.tail, len_a,
                                         tail_slot=slots, scale=SCALE)
        len_a += 1
        for n in "qkv":
            x[n].copy_(new[n])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(o_a), bits(o_b))
    for a, b in zip(c.tail, other):
        if a is not None:
            assert torch.equal(bits(a), bits(b))


def test_repeated_calls_are_bitwise_equal_and_streams_are_independent():
    c = Case(530, list(range(0, 60, 3)), 4, [0] * 11 + [1] * 9, 2, True, "mxfp8")
    o = c.decode()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    f = c.fold()
    torch.cuda.synchronize()
    out = []
    for s in (s1, s2, s1, s2):
        with torch.cuda.stream(s):
            out.append((c.fold(), gla.gla_prefix_fwd(*[c.g[n] for n in "qkv"], c.llg, c.poolg, i32(c.rows),
                                                     i32(range(c.N + 1)))[0]))
    torch.cuda.synchronize()
    assert torch.equal(o, c.decode())
    for x, y in out:
        assert torch.equal(x, f) and torch.equal(y, out[0][1])


@pytest.mark.parametrize("fmt", ["native", "mxfp8"])
def test_debug_bounds_build_gives_the_same(fmt):
    c = Case(540, [0, 1, 16, 33, 70, 5], 3, [0, 0, 1, 1, 1, 0], 2, True, fmt)
    o, f = c.decode(), c.fold()
    with gla.debug_bounds_library():
        o2, f2 = c.decode(), c.fold()
        assert gla.gla_get_device_error() == 0
    assert torch.equal(o, o2) and torch.equal(f, f2)


@pytest.mark.parametrize("fmt", ["native", "mxfp8"])
def test_offsets_past_32_bits(fmt):
    """A tail whose last rows start past 2^32 bytes (values) and 2^31 elements."""
    H, cap = 16, 512
    R = 2 ** 32 // (H * cap * DV) + 3 if fmt == "mxfp8" else 2 ** 31 // (H * cap * DV) + 3
    t = gla.gla_tail_alloc(R, H, cap, torch.float8_e4m3fn if fmt == "mxfp8" else torch.bfloat16)
    lens, rows = [33, 511], [0, 0]
    small = Case(550, lens, H, rows, 1, True, fmt, cap=cap, spare=0)
    slots = [R - 1, R - 2]
    for big, x in zip(t, small.tail):
        if big is not None:
            for i in range(2):
                big[slots[i]] = x[small.slots[i]]
    o = gla.gla_prefix_decode_step(small.g["q"], small.g["k"], small.g["v"], small.llg, small.poolg, i32(rows), t,
                                   i32(lens), tail_slot=i32(slots), scale=SCALE)
    check_decode(small, o)
    f = gla.gla_tail_fold(small.llg, small.poolg, i32(rows), t, i32(lens), tail_slot=i32(slots))
    want = small.decode()
    assert torch.equal(o, want)
    assert torch.equal(f, small.fold())
    for big, x in zip(t, small.tail):
        if big is not None:
            for i in range(2):
                assert torch.equal(bits(big[slots[i]]), bits(x[small.slots[i]]))


# ---- values at the edges -----------------------------------------------------------------------
@pytest.mark.parametrize("fmt", ["native", "mxfp8"])
@pytest.mark.parametrize("bf16", [True, False])
def test_infinities_and_nan_stay_with_their_sequence(bf16, fmt):
    """A NaN state, an infinity or a NaN in a sequence's tail or new token: the other sequences of the
    tile come out as without it."""
    c = Case(600, [20, 33, 7, 64, 0, 5, 18], 2, [0, 1, 1, 2, 0, 2, 2], 4, bf16, fmt)
    clean = c.decode()
    rows = list(c.rows)
    rows[3] = 3
    c.poolg[3] = float("nan")
    if fmt == "mxfp8":
        c.tail.v[c.slots[1], :, 4, 40] = 0x7F
    else:
        c.tail.v[c.slots[1], :, 4, 40] = float("inf")
        c.tail.k[c.slots[5], :, 2, 3] = float("nan")
    c.g["q"][6, :, 5] = float("nan")
    o = gla.gla_prefix_decode_step(c.g["q"], c.g["k"], c.g["v"], c.llg, c.poolg, i32(rows), c.tail, i32(c.lens),
                                   tail_slot=i32(c.slots), scale=SCALE)
    for n in (0, 2, 4):
        assert torch.equal(bits(o[n]), bits(clean[n])), n
    bad = {1: (slice(None), 40), 3: (slice(None), slice(None)), 6: (slice(None), slice(None))}
    if fmt != "mxfp8":
        bad[5] = (slice(None), slice(None))
    for n, at in bad.items():
        assert not bool(torch.isfinite(o[n][at]).any()), n
    ok = torch.ones(DV, dtype=torch.bool)
    ok[40] = False
    assert torch.equal(bits(o[1][:, ok.cuda()]), bits(clean[1][:, ok.cuda()]))


@pytest.mark.parametrize("bf16", [True, False])
def test_mxfp8_tails_of_many_magnitudes(bf16):
    """Keys and values whose blocks differ by up to 2^24 from token to token, growing and shrinking
    along the tail: the decode's running power of two per block follows them."""
    lens, H = [70, 40, 33, 130], 3
    c = Case(610, lens, H, [0, 0, 1, 1], 2, bf16, "mxfp8")
    rng = np.random.default_rng(5)
    k, v = c.t.k.copy(), c.t.v.copy()
    e = rng.integers(-12, 13, v.shape[:3] + (6,))
    e[c.slots[0]] = np.sort(e[c.slots[0]], axis=1)            # growing along the tail
    e[c.slots[1]] = -np.sort(-e[c.slots[1]], axis=1)          # shrinking
    v = np.nan_to_num(v) * np.exp2(e).repeat(32, axis=3)
    k = np.nan_to_num(k) * np.exp2(rng.integers(-6, 7, k.shape[:3] + (3,))).repeat(32, axis=3)
    (c.t.kc, c.t.ks), (c.t.vc, c.t.vs) = oracle.mxfp8_quantize(k), oracle.mxfp8_quantize(v)
    c.t.k, c.t.v = oracle.mxfp8_dequantize(c.t.kc, c.t.ks), oracle.mxfp8_dequantize(c.t.vc, c.t.vs)
    c.tail = c.t.device()
    check_decode(c)
    s = c.fold().cpu().numpy().astype(np.float64)
    ref, mag = ref_fold(c.ll, c.pool, c.rows, c.t.k, c.t.v, c.slots, c.lens)
    assert np.all(np.abs(s - ref) <= tol(ref, mag, max(lens) + 2, True, False))


@pytest.mark.parametrize("scale_q", [2.0 ** -60, 2.0 ** 40])
@pytest.mark.parametrize("fmt", ["native", "mxfp8"])
def test_decode_with_tiny_and_huge_queries(fmt, scale_q):
    c = Case(620, [30, 5, 17], 2, [0, 1, 1], 2, True, fmt)
    c.q = gs.bf16_round((c.q * scale_q).astype(np.float32))
    c.q[1, :, 3] *= 2.0 ** 20                                # one dimension far above the others
    c.g["q"] = torch.from_numpy(c.q).cuda().to(c.dt)
    check_decode(c)


def test_one_tail_row_for_read_only_use_and_repeated_rows():
    """Two sequences may fold the same tail row (it is only read), into rows of their own."""
    c = Case(630, [20, 20], 2, [0, 1], 2, True, "mxfp8")
    out = gla.gla_tail_fold(c.llg, c.poolg, i32([0, 1]), c.tail, i32([20, 12]), tail_slot=i32([c.slots[0]] * 2))
    for n, (r, L) in enumerate(((0, 20), (1, 12))):
        ref, mag = ref_fold(c.ll, c.pool, [r], c.t.k, c.t.v, [c.slots[0]], [L])
        assert np.all(np.abs(out[n:n + 1].cpu().numpy() - ref) <= tol(ref, mag, 24, True, False))


# ---- bounded waits -----------------------------------------------------------------------------
def test_short_wait_limit_reports_timeout_and_the_context_survives():
    """With a wait limit of 1 ns, waits that the hardware's own first try does not see through give up
    (many in a decode whose loads queue up behind each other, maybe none in a fold): the kernels
    drain their copies and MMAs and return, GLA_ERR_TIMEOUT is reported, and the next calls are right."""
    N, H = 640, 16
    c = Case(640, [40] * 4, 2, [0] * 4, 1, True, "mxfp8")
    tail = gla.gla_tail_alloc(N, H, 160, torch.float8_e4m3fn)
    for x in (tail.k, tail.v):
        x.random_(0, 0x7E)
    for x in (tail.k_scales, tail.v_scales):
        x.random_(118, 122)
    pool, rows, lens = torch.randn(2, H, DK, DV, device="cuda"), i32([0] * 300 + [1] * 340), i32([159] * N)
    ll = torch.full((H,), -0.01, device="cuda")
    q, k, v = (torch.randn(N, H, d, device="cuda", dtype=torch.bfloat16) for d in (DK, DK, DV))
    calls = (lambda: gla.gla_prefix_decode_step(q, k, v, ll, pool, rows, tail, lens),
             lambda: gla.gla_tail_fold(ll, pool, rows, tail, lens))
    want = [f() for f in calls]
    assert gla.gla_get_device_error() == 0
    for f, w in zip(calls, want):
        gla.gla_set_wait_limit_ns(1)
        try:
            f()
            err = gla.gla_get_device_error()
        finally:
            gla.gla_set_wait_limit_ns(2_000_000_000)
        assert err in (0, -8)
        assert gla.gla_get_device_error() == 0
        assert torch.equal(f(), w)
    check_decode(c)


# ---- several calls at once ---------------------------------------------------------------------
def test_two_graphs_and_eager_calls_on_several_streams():
    """Two captured steps on pools of their own, replayed at once on two streams beside eager calls
    on a third: the calls share no workspace, so each gives what it gives alone."""
    cases = [Case(650 + i, [40, 3, 90, 17] * 6, 3, [0, 1] * 12, 2, True, "mxfp8") for i in range(3)]
    alone = [x.decode() for x in cases]
    folds = [x.fold() for x in cases]
    idx = [[i32(x.rows), i32(x.lens), i32(x.slots)] for x in cases]
    streams = [torch.cuda.Stream() for _ in range(3)]
    graphs, outs = [], []
    torch.cuda.synchronize()
    for x, (rows, lens, slots), s in zip(cases[:2], idx, streams):
        g, o = torch.cuda.CUDAGraph(), torch.empty_like(alone[0])
        f = torch.empty_like(folds[0])
        with torch.cuda.graph(g, stream=s):
            gla.gla_prefix_decode_step(x.g["q"], x.g["k"], x.g["v"], x.llg, x.poolg, rows, x.tail, lens,
                                       tail_slot=slots, scale=SCALE, o=o)
            gla.gla_tail_fold(x.llg, x.poolg, rows, x.tail, lens, tail_slot=slots, out=f)
        graphs.append(g)
        outs.append((o, f))
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            x, (rows, lens, slots) = cases[2], idx[2]
            o = gla.gla_prefix_decode_step(x.g["q"], x.g["k"], x.g["v"], x.llg, x.poolg, rows, x.tail, lens,
                                           tail_slot=slots, scale=SCALE)
            f = gla.gla_tail_fold(x.llg, x.poolg, rows, x.tail, lens, tail_slot=slots)
    torch.cuda.synchronize()
    for (a, b), d, e in zip(outs + [(o, f)], alone, folds):
        assert torch.equal(a, d) and torch.equal(b, e)


@pytest.mark.parametrize("bf16", [True, False])
def test_captured_packed_calls(bf16):
    """Forward and backward from shared states, captured (the backward's side streams fork and join
    inside the capture) and replayed on new inputs."""
    lens, H, rows, P = PACKED[0]
    d, g, rg = packed(660, lens, H, rows, P, bf16)
    _, g2, _ = packed(661, lens, H, rows, P, bf16)

    def both(x):
        fwd = gla.gla_prefix_fwd(x["q"], x["k"], x["v"], x["ll"], x["pool"], rg, x["cu"], SCALE)
        return fwd + gla.gla_prefix_bwd(x["q"], x["k"], x["v"], x["ll"], x["dO"], x["pool"], rg, x["cu"], SCALE,
                                        dhT=x["dhT"])
    want = both(g2)
    both(g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(g)
    for name in ("q", "k", "v", "dO", "pool", "dhT"):
        g[name].copy_(g2[name])
    graph.replay()
    torch.cuda.synchronize()
    for i, (x, y) in enumerate(zip(got, want)):
        if bf16 and i in (2, 3):  # dq, dk: partial sums in arrival order
            assert within_one_bf16_rounding(x.float().cpu().numpy(), y.float().cpu().numpy())
        else:
            assert torch.equal(x, y)


def backward_into(x, rg):
    """A function that runs the backward into tensors of its own (nothing is allocated by the call)."""
    n_seq, T, H = rg.numel(), x["q"].shape[0], x["q"].shape[1]
    code = 0 if x["q"].dtype == torch.bfloat16 else 1
    out = {"d" + n: torch.empty_like(x[n]) for n in ("q", "k", "v", "pool")}
    out["workspace"] = torch.empty(gla.gla_prefix_bwd_workspace_bytes(n_seq, T, H, code), dtype=torch.uint8,
                                   device="cuda")
    return lambda: gla.gla_prefix_bwd(x["q"], x["k"], x["v"], x["ll"], x["dO"], x["pool"], rg, x["cu"], SCALE,
                                      dhT=x["dhT"], **out)


def same_gradients(got, want, bf16):
    for i, (x, y) in enumerate(zip(got, want)):
        if bf16 and i < 2:  # dq, dk: partial sums in arrival order
            assert within_one_bf16_rounding(x.float().cpu().numpy(), y.float().cpu().numpy())
        else:
            assert torch.equal(x, y)


@pytest.mark.parametrize("bf16", [True, False])
def test_backward_beside_an_open_capture(bf16):
    """An eager backward on one stream, and a second capture's on another, while a capture that holds a
    backward is open: the captures' side streams are their own."""
    lens, H, rows, P = PACKED[0]
    cases = [packed(662 + i, lens, H, rows, P, bf16) for i in range(3)]
    runs = [backward_into(g, rg) for _, g, rg in cases]
    want = [[t.clone() for t in run()] for run in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.stream(streams[0]):
        graphs[0].capture_begin(capture_error_mode="thread_local")
        first = runs[0]()
        with torch.cuda.stream(streams[2]):
            eager = runs[2]()
        runs[0]()  # (twice in one capture)
        graphs[0].capture_end()
    same_gradients(eager, want[2], bf16)
    with torch.cuda.stream(streams[1]):
        graphs[1].capture_begin(capture_error_mode="thread_local")
        second = runs[1]()
        graphs[1].capture_end()
    for t in first + second:
        t.zero_()
    torch.cuda.synchronize()
    for g, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    same_gradients(first, want[0], bf16)
    same_gradients(second, want[1], bf16)


@pytest.mark.parametrize("bf16", [True, False])
def test_backwards_of_several_threads(bf16):
    """Threads that run backwards on streams of their own, eagerly, one of them capturing its calls."""
    lens, H, rows, P = PACKED[0]
    cases = [packed(665 + i, lens, H, rows, P, bf16) for i in range(4)]
    runs = [backward_into(g, rg) for _, g, rg in cases]
    want = [[t.clone() for t in run()] for run in runs]
    torch.cuda.synchronize()
    got, failed = [None] * 4, []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(8):
                    if i == 0:
                        g = torch.cuda.CUDAGraph()
                        g.capture_begin(capture_error_mode="thread_local")
                        got[i] = runs[i]()
                        g.capture_end()
                        for t in got[i]:
                            t.zero_()
                        g.replay()
                    else:
                        got[i] = runs[i]()
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001 (reported below)
            failed.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for x, y in zip(got, want):
        same_gradients(x, y, bf16)
