"""GPU parity of the gated delta rule against the recurrence in 64 bits, its refusals on the device, and the way it
is used: slot plans, packed prefills into a pool, decode steps, gradients.  Bounds: tests/delta_helpers.py."""
import threading

import pytest
import torch

import linear_attention_recurrence_simple_gb300 as gla
from tests.delta_helpers import DK, DV, SCALE, Batch, check, far, plan_ref, ref_fwd

pytestmark = pytest.mark.gpu
SHAPE_ERR = -2
BF, F32 = torch.bfloat16, torch.float32
NAMES = ("dq", "dk", "dv", "dg", "dbeta")


@pytest.fixture(scope="module", autouse=True)
def _setup():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    gla.load_library()
    yield
    assert gla.gla_get_device_error() == 0


def kinds(dtype):
    return ("bf16", "state") if dtype == BF else ("f32", "f32")


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def check_fwd(b, o, hT, h0):
    out, state = kinds(b.dtype)
    refs = [b.ref(n, h0[n]) for n in range(len(b.lens))]
    check(b.rows(o), torch.cat([r[0] for r in refs]), out, "o")
    if hT is not None:
        check(hT, torch.stack([r[1] for r in refs]), state, "hT")


def check_bwd(b, grads, h0, dhT):
    out, state = kinds(b.dtype)
    refs = [b.ref_bwd(n, h0[n], dhT[n]) for n in range(len(b.lens))]
    for i, name in enumerate(NAMES):
        check(b.rows(grads[i]), torch.cat([r[i] for r in refs]), out, name)
    if grads[5] is not None:
        check(grads[5], torch.stack([r[5] for r in refs]), state, "dh0")


LENS = [[1], [2], [63], [64], [65], [127, 129], [128], [200, 0, 1, 64, 33, 300]]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("H", [1, 3])
def test_forward(lens, H, dtype):
    b = Batch(1, lens, H, dtype)
    h0 = b.h0 if H == 3 else torch.zeros_like(b.h0)
    o, hT = gla.gla_delta_fwd(*b.inputs(), h0=b.h0.cuda() if H == 3 else None, cu_seqlens=b.cu_dev)
    check_fwd(b, o, hT, h0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,T,H", [(1, 1, 1), (3, 70, 2), (2, 256, 16), (0, 5, 2), (4, 0, 2)])
def test_forward_equal_lengths(N, T, H, dtype):
    b = Batch(2, [T] * N, H, dtype, packed=False) if N else None
    if N == 0:
        x = [torch.empty(0, T, H, d, dtype=dtype, device="cuda") for d in (DK, DK, DV)]
        o, hT = gla.gla_delta_fwd(*x, *[torch.empty(0, T, H, dtype=dtype, device="cuda")] * 2)
        assert o.numel() == 0 and hT.shape == (0, H, DK, DV)
        return
    o, hT = gla.gla_delta_fwd(*b.inputs(), scale=0.3, h0=b.h0.cuda())
    refs = [ref_fwd(*(b.host(n, m) for m in ("q", "k", "v", "g", "beta")), b.h0[n].double(), 0.3) for n in range(N)]
    check(b.rows(o), torch.cat([r[0] for r in refs]), kinds(dtype)[0], "o")
    check(hT, torch.stack([r[1] for r in refs]), kinds(dtype)[1], "hT")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_pool_in_place_and_rows(dtype):
    """Sequences go on from pool rows, from zeros, or from a row that two of them share, and end in rows of the same
    pool; rows without a sequence and packed rows behind the last one stay."""
    b = Batch(3, [70, 0, 5, 130, 64], 2, dtype, spare=9)
    pool = torch.randn(9, 2, DK, DV, generator=torch.Generator().manual_seed(4)) * 0.1
    start, to = [3, -1, -1, 7, 7], [3, -1, 0, 5, 8]
    before, dev = pool.clone(), pool.cuda()
    o = torch.full((int(b.cu[-1]) + 9, 2, DV), 7.0, dtype=dtype, device="cuda")
    o2, out = gla.gla_delta_fwd(*b.inputs(), h0=dev, h0_row=i32(start), hT=dev, hT_row=i32(to), cu_seqlens=b.cu_dev, o=o)
    assert out is dev and o2 is o and bool((o[-9:] == 7.0).all())
    h0 = [before[r] if r >= 0 else torch.zeros(2, DK, DV) for r in start]
    check_fwd(b, o, None, h0)
    for n, r in enumerate(to):
        if r >= 0:
            check(dev[r], b.ref(n, h0[n])[1], kinds(dtype)[1], f"row {r}")
    for r in set(range(9)) - set(to):
        assert torch.equal(dev[r].cpu(), before[r])


def test_rows_outside_are_reported():
    b = Batch(5, [10, 20], 1, BF)
    pool = (torch.randn(3, 1, DK, DV) * 0.1).cuda()
    kept = pool.clone()
    o, _ = gla.gla_delta_fwd(*b.inputs(), h0=pool, h0_row=i32([3, 1]), hT=pool, hT_row=i32([0, 9]), cu_seqlens=b.cu_dev)
    assert gla.gla_get_device_error() == SHAPE_ERR
    check_fwd(b, o, None, [torch.zeros(1, DK, DV), kept[1].cpu()])
    assert torch.equal(pool[1:], kept[1:])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_bad_offsets_are_clamped_and_reported(dtype):
    b = Batch(6, [40, 60, 30], 2, dtype)
    for cu in ([0, 90, 50, 130], [0, -5, 100, 130], [0, 40, 100, 500]):
        gla.gla_delta_fwd(*b.inputs(), cu_seqlens=i32(cu))
        assert gla.gla_get_device_error() == SHAPE_ERR
        gla.gla_delta_bwd(*b.inputs(), *b.dev("dO"), cu_seqlens=i32(cu))
        assert gla.gla_get_device_error() == SHAPE_ERR


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", LENS[:6] + [[150, 0, 1, 64, 33]], ids=str)
def test_backward(lens, dtype):
    b = Batch(7, lens, 2, dtype)
    grads = gla.gla_delta_bwd(*b.inputs(), *b.dev("dO"), h0=b.h0.cuda(), dhT=b.dhT.cuda(), cu_seqlens=b.cu_dev)
    check_bwd(b, grads, b.h0, b.dhT)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_backward_equal_lengths_and_no_states(dtype):
    b = Batch(8, [100] * 2, 3, dtype, packed=False)
    grads = gla.gla_delta_bwd(*b.inputs(), *b.dev("dO"), need_dh0=False)
    assert grads[5] is None
    zero = torch.zeros_like(b.h0)
    check_bwd(b, grads, zero, zero)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_sequences_and_heads(dtype):
    """More (sequence, head)s than the GPU runs at a time, of several chunks and a ragged last one."""
    b = Batch(21, [200] * 4, 40, dtype, packed=False)
    o, hT = gla.gla_delta_fwd(*b.inputs(), h0=b.h0.cuda())
    check_fwd(b, o, hT, b.h0)
    grads = gla.gla_delta_bwd(*b.inputs(), *b.dev("dO"), h0=b.h0.cuda(), dhT=b.dhT.cuda())
    check_bwd(b, grads, b.h0, b.dhT)


@pytest.mark.parametrize("N,T,H", [(13, 200, 16), (51, 65, 1), (1, 700, 103), (5, 128, 32), (40, 300, 16), (304, 70, 1)])
def test_equal_lengths_as_packed(N, T, H):
    """The same bits from a call of equal lengths and from a packed one of those sequences."""
    b = Batch(22, [T] * N, H, BF, packed=False)
    x, dO, h0, dhT = b.inputs(), b.dev("dO")[0], b.h0.cuda(), b.dhT.cuda()
    cu = i32(range(0, N * T + 1, T))
    flat = [t.reshape(N * T, *t.shape[2:]) for t in (*x, dO)]
    for _ in range(3):
        o, hT = gla.gla_delta_fwd(*x, h0=h0)
        o2, hT2 = gla.gla_delta_fwd(*flat[:5], h0=h0, cu_seqlens=cu)
        assert torch.equal(o.reshape(o2.shape), o2) and torch.equal(hT, hT2)
    grads = gla.gla_delta_bwd(*x, dO, h0=h0, dhT=dhT)
    for a, c in zip(grads, gla.gla_delta_bwd(*flat, h0=h0, dhT=dhT, cu_seqlens=cu)):
        assert torch.equal(a.reshape(c.shape), c)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_packed_sequences(dtype):
    """Offsets of thousands of sequences: places of chunks, the order of the scans, empty sequences among them."""
    lens = [(7 * i) % 5 for i in range(1100)] + [130, 0, 64, 1] + [i % 3 for i in range(1500)]
    b = Batch(23, lens, 1, dtype)
    o, hT = gla.gla_delta_fwd(*b.inputs(), h0=b.h0.cuda(), cu_seqlens=b.cu_dev)
    check_fwd(b, o, hT, b.h0)
    grads = gla.gla_delta_bwd(*b.inputs(), *b.dev("dO"), h0=b.h0.cuda(), dhT=b.dhT.cuda(), cu_seqlens=b.cu_dev)
    check_bwd(b, grads, b.h0, b.dhT)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_backward_without_tokens(dtype):
    x = [torch.empty(2, 0, 1, d, dtype=dtype, device="cuda") for d in (DK, DK, DV)]
    g = torch.empty(2, 0, 1, dtype=dtype, device="cuda")
    dhT = torch.randn(2, 1, DK, DV, device="cuda")
    grads = gla.gla_delta_bwd(*x, g, g, x[2], dhT=dhT)
    assert torch.equal(grads[5], dhT) and all(t.numel() == 0 for t in grads[:5])


def harsh(name, T, H):
    """Gates and strengths where a chunk's form could go wrong."""
    g = -0.1 * torch.rand(T, H, generator=torch.Generator().manual_seed(11))
    beta = torch.rand(T, H, generator=torch.Generator().manual_seed(12))
    if name == "resets":
        g[::37] = -float("inf")
        g[5::41] = -1000.0
    elif name == "strong":
        g = g * 300
    elif name == "mixed":  # strong decay, then almost none: what is left is a difference of large sums
        g = torch.where(torch.arange(T)[:, None] % 20 < 3, -90.0, -1e-3) * torch.ones(T, H)
    elif name == "none":
        g = torch.zeros(T, H)
    elif name == "beta0":
        beta[::3] = 0
    elif name == "beta2":
        beta = 2 * beta
    return g, beta


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("name", ["resets", "strong", "mixed", "none", "beta0", "beta2"])
def test_harsh_gates(name, dtype):
    b = Batch(9, [150, 90], 2, dtype)
    b.x["g"], b.x["beta"] = harsh(name, 240, 2)
    o, hT = gla.gla_delta_fwd(*b.inputs(), h0=b.h0.cuda(), cu_seqlens=b.cu_dev)
    check_fwd(b, o, hT, b.h0)
    grads = gla.gla_delta_bwd(*b.inputs(), *b.dev("dO"), h0=b.h0.cuda(), dhT=b.dhT.cuda(), cu_seqlens=b.cu_dev)
    check_bwd(b, grads, b.h0, b.dhT)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_key_again_and_again(dtype):
    """The same key at every token: M is as large as it gets."""
    b = Batch(10, [130], 2, dtype)
    b.x["k"] = b.x["k"][:1].expand_as(b.x["k"]).clone()
    b.x["g"] = b.x["g"] * 0.01
    o, hT = gla.gla_delta_fwd(*b.inputs(), h0=b.h0.cuda(), cu_seqlens=b.cu_dev)
    check_fwd(b, o, hT, b.h0)
    grads = gla.gla_delta_bwd(*b.inputs(), *b.dev("dO"), h0=b.h0.cuda(), dhT=b.dhT.cuda(), cu_seqlens=b.cu_dev)
    check_bwd(b, grads, b.h0, b.dhT)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nonfinite_stays_in_its_sequence(bad, dtype):
    """What a token with an infinity or a NaN reaches: its chunk and what follows, in its sequence and head."""
    b = Batch(11, [100, 200, 65], 2, dtype)
    clean, cleanT = gla.gla_delta_fwd(*b.inputs(), cu_seqlens=b.cu_dev)
    b.x["v"][100 + 130, 1, 17] = bad
    o, hT = gla.gla_delta_fwd(*b.inputs(), cu_seqlens=b.cu_dev)
    assert torch.equal(o[:, 0], clean[:, 0]) and torch.equal(hT[:, 0], cleanT[:, 0])
    assert torch.equal(o[:228], clean[:228]) and torch.equal(o[300:], clean[300:])
    assert torch.equal(hT[0], cleanT[0]) and torch.equal(hT[2], cleanT[2])
    assert not bool(torch.isfinite(o[230, 1, 17]))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_same_bits_again_other_stream_and_captured(dtype):
    b = Batch(12, [90, 130], 3, dtype)
    x, dO, h0, cu = b.inputs(), b.dev("dO")[0], b.h0.cuda(), b.cu_dev
    first = [*gla.gla_delta_fwd(*x, h0=h0, cu_seqlens=cu), *gla.gla_delta_bwd(*x, dO, h0=h0, cu_seqlens=cu)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = [*gla.gla_delta_fwd(*x, h0=h0, cu_seqlens=cu), *gla.gla_delta_bwd(*x, dO, h0=h0, cu_seqlens=cu)]
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [*gla.gla_delta_fwd(*x, h0=h0, cu_seqlens=cu), *gla.gla_delta_bwd(*x, dO, h0=h0, cu_seqlens=cu)]
    for t in got:
        t.fill_(9.0)
    graph.replay()
    torch.cuda.synchronize()
    for a, c, d in zip(first, again, got):
        assert torch.equal(a, c) and torch.equal(a, d)


def test_two_threads_two_streams():
    b = Batch(13, [200, 70], 4, BF)
    x, dO, cu = b.inputs(), b.dev("dO")[0], b.cu_dev
    want = [*gla.gla_delta_fwd(*x, cu_seqlens=cu), *gla.gla_delta_bwd(*x, dO, cu_seqlens=cu)]
    torch.cuda.synchronize()
    bad = []

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(8):
                got = [*gla.gla_delta_fwd(*x, cu_seqlens=cu), *gla.gla_delta_bwd(*x, dO, cu_seqlens=cu)]
                torch.cuda.current_stream().synchronize()
                bad.extend(i for i, (a, c) in enumerate(zip(want, got)) if not torch.equal(a, c))

    threads = [threading.Thread(target=work) for _ in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sdtype", [F32, BF])
@pytest.mark.parametrize("N,H", [(1, 1), (5, 3), (40, 16)])
def test_decode(N, H, sdtype, dtype):
    b = Batch(14, [1] * N, H, dtype)
    pool = (torch.randn(N + 3, H, DK, DV, generator=torch.Generator().manual_seed(15)) * 0.1).to(sdtype)
    slot = torch.randperm(N + 3, generator=torch.Generator().manual_seed(16))[:N].tolist()
    b.x["g"][0] = -float("inf")
    dev = pool.cuda()
    o = gla.gla_delta_decode_step(*b.inputs(), dev, slot=i32(slot))
    for n, s in enumerate(slot):
        ro, rS = b.ref(n, pool[s])
        check(o[n:n + 1], ro, "bf16" if dtype == BF else "f32", "o")
        check(dev[s], rS, "bf16" if sdtype == BF else "f32", "state")
    for s in set(range(N + 3)) - set(slot):
        assert torch.equal(dev[s].cpu(), pool[s])


def test_decode_without_rows():
    b = Batch(17, [1] * 3, 2, BF)
    pool = (torch.randn(4, 2, DK, DV) * 0.1).cuda()
    kept, o = pool.clone(), torch.full((3, 2, DV), 5.0, dtype=BF, device="cuda")
    gla.gla_delta_decode_step(*b.inputs(), pool, slot=i32([-1, 2, -1]), o=o)
    assert gla.gla_get_device_error() == 0
    assert bool((o[[0, 2]] == 5.0).all()) and torch.equal(pool[[0, 1, 3]], kept[[0, 1, 3]])
    check(pool[2], b.ref(1, kept[2].cpu())[1], "f32")
    gla.gla_delta_decode_step(*b.inputs(), pool, slot=i32([-1, 4, -2]), o=o)
    assert gla.gla_get_device_error() == SHAPE_ERR


def test_decode_captured():
    b = Batch(18, [1] * 6, 4, BF)
    x, pool = b.inputs(), (torch.randn(6, 4, DK, DV) * 0.1).cuda()
    eager, o = pool.clone(), torch.empty(6, 4, DV, dtype=BF, device="cuda")
    gla.gla_delta_decode_step(*x, eager.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gla.gla_delta_decode_step(*x, pool, o=o)
    for _ in range(3):
        graph.replay()
        want = gla.gla_delta_decode_step(*x, eager)
    torch.cuda.synchronize()
    assert torch.equal(pool, eager) and torch.equal(o, want)


# --------------------------------------------------------------------------------------- slot plans
def plan_inputs(seed, N, rows, long=300):
    g = torch.Generator().manual_seed(seed)
    free = torch.randperm(rows, generator=g).tolist()
    new, held, seen = [], [], []
    for u, w in zip(torch.rand(N, generator=g).tolist(), torch.randint(0, long, (N,), generator=g).tolist()):
        held.append(free.pop() if free and u < 0.7 else -1)
        new.append(-1 if u < 0.1 or 0.95 < u else 0 if u < 0.2 else 1 if u < 0.6 else w)
        seen.append(w if held[-1] >= 0 else 0)
    return new, held, seen


@pytest.mark.parametrize("N,rows,budget", [(1, 1, 1), (1, 5, 0), (3, 2, 100), (33, 31, 50), (64, 64, 4096), (1000, 700, 3000),
                                           (1025, 2000, 100000), (5000, 4097, 20000), (2500, 1, 77)])
@pytest.mark.parametrize("seed", range(3))
def test_plan(N, rows, budget, seed):
    new, held, seen = plan_inputs(seed, N, rows)
    for s in (seen, None):
        got = gla.gla_slot_plan(i32(new), i32(held), None if s is None else i32(s), rows, budget)
        for name, x, want in zip(gla.SlotPlan._fields, got, plan_ref(new, held, s, rows, budget)):
            assert x.tolist() == want, name


def test_plan_large_lengths_and_pools():
    new, held = [2 ** 31 - 1] * 40, [-1] * 20 + list(range(20))
    got = gla.gla_slot_plan(i32(new), i32(held), None, 1 << 19, 1000)
    for x, want in zip(got, plan_ref(new, held, None, 1 << 19, 1000)):
        assert x.tolist() == want
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    got = gla.gla_slot_plan(e, e, e, 4, 3)
    assert got.cu_seqlens.tolist() == [0] and got.token_seq.tolist() == [-1] * 3


def test_plan_refusals_on_the_device():
    got = gla.gla_slot_plan(i32([2, 2, 2]), i32([9, -1, 1]), None, 3, 10)  # a row outside the pool
    assert gla.gla_get_device_error() == SHAPE_ERR
    assert got.row.tolist() == [-1, 0, 1] and got.cu_seqlens.tolist() == [0, 0, 2, 4]
    gla.gla_slot_plan(i32([1, 1]), i32([2, 2]), None, 3, 10)  # one row twice
    assert gla.gla_get_device_error() == SHAPE_ERR


def test_plan_row_over_held_and_captured():
    new, held, seen = plan_inputs(5, 200, 150)
    a, h, s = i32(new), i32(held), i32(seen)
    out = gla.gla_slot_plan(a, h, s, 150, 500)
    want = plan_ref(new, held, seen, 150, 500)
    over = gla.SlotPlan(out[0], out[1], out[2], h, out[4], out[5])
    gla.gla_slot_plan(a, h, s, 150, 500, out=over)  # row written where held stands
    for x, w in zip(over, want):
        assert x.tolist() == w
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gla.gla_slot_plan(a, h, s, 150, 500, out=over)
    graph.replay()
    torch.cuda.synchronize()
    for x, w in zip(over, plan_ref(new, want[3], seen, 150, 500)):
        assert x.tolist() == w


# ------------------------------------------------------------------------------------ used together
@pytest.mark.parametrize("dtype", [BF, F32])
def test_serving_steps(dtype):
    """Requests come, are prefilled in pieces under a token budget, decode, and leave; every token's output against the
    recurrence over the request's whole sequence."""
    H, R, budget = 2, 4, 100
    prompts, extra = [30, 150, 7, 64, 90, 3], 3  # tokens of each request, and decode steps after its prompt
    total = [p + extra for p in prompts]
    b = Batch(20, total, H, dtype)
    x = {m: b.dev(m)[0] for m in ("q", "k", "v", "g", "beta")}
    want = torch.cat([b.ref(n, torch.zeros(H, DK, DV))[0] for n in range(len(total))])
    got = torch.full_like(want, float("nan"))
    pool = torch.full((R, H, DK, DV), float("nan"), device="cuda")  # nothing may come from a row's last user
    N = len(total)
    held, seen = i32([-1] * N), [0] * N
    for _ in range(60):
        left = [t - s for t, s in zip(total, seen)]
        if not any(left):
            break
        new = [-1 if n == 0 else max(1, n - extra) for n in left]
        p = gla.gla_slot_plan(i32(new), held, i32(seen), R, budget)
        held, cu = p.row, p.cu_seqlens.tolist()
        base = torch.from_numpy(b.cu).cuda()
        live = p.token_seq >= 0
        at = (base[p.token_seq.clamp(min=0).long()] + p.token_pos)[live].long()
        step = {m: torch.zeros((budget,) + t.shape[1:], dtype=t.dtype, device="cuda") for m, t in x.items()}
        for m, t in x.items():
            step[m][:at.numel()] = t[at]
        lens = [c - a for a, c in zip(cu, cu[1:])]
        if max(lens) == 1:  # only single tokens: the decode step
            tok = base[:N] + i32(seen)
            one = [x[m][tok.clamp(max=int(b.cu[-1]) - 1).long()].contiguous() for m in ("q", "k", "v", "g", "beta")]
            fresh = (p.start_row < 0) & (p.slot >= 0)
            pool[p.slot[fresh].long()] = 0
            o = gla.gla_delta_decode_step(*one, pool, slot=p.slot)[p.slot >= 0]
        else:
            o, _ = gla.gla_delta_fwd(*step.values(), h0=pool, h0_row=p.start_row, hT=pool, hT_row=p.slot,
                                     cu_seqlens=p.cu_seqlens)
            o = o[:at.numel()]
        got[at.cpu()] = o.double().cpu()
        seen = [s + n for s, n in zip(seen, lens)]
    assert seen == total
    check(got, want, kinds(dtype)[0], "o")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_training_step_gradients(dtype):
    """Loss over outputs and final states, by the calls' gradients and by a difference along their direction."""
    b = Batch(21, [80, 70], 2, dtype)
    x, cu, h0 = b.inputs(), b.cu_dev, b.h0.cuda()
    w, wT = b.dev("dO")[0], b.dhT.cuda()
    grads = gla.gla_delta_bwd(*x, w, h0=h0, dhT=wT, cu_seqlens=cu)
    step = [torch.randn_like(t.float()) for t in x]
    step[3], step[4] = step[3] * 0.05, step[4] * 0.05

    def loss(e):  # in 64 bits
        s = 0.0
        for n in range(2):
            sl = slice(int(b.cu[n]), int(b.cu[n + 1]))
            o, S = ref_fwd(*((t.double() + e * d.double())[sl].cpu() for t, d in zip(x, step)), b.h0[n].double())
            s += float((o * w[sl].double().cpu()).sum() + (S * wT[n].double().cpu()).sum())
        return s

    slope = sum(float((g.double() * d.double()).sum()) for g, d in zip(grads, step))
    numeric = (loss(1e-4) - loss(-1e-4)) / 2e-4
    size = sum(float((g.double() * d.double()).norm()) for g, d in zip(grads, step))
    assert abs(slope - numeric) <= (1e-2 if dtype == BF else 1e-5) * size + 1e-6 * abs(numeric)


def test_scale_default_and_debug_build():
    b = Batch(22, [70, 130], 3, BF)
    x, dO, cu, h0 = b.inputs(), b.dev("dO")[0], b.cu_dev, b.h0.cuda()
    want = [*gla.gla_delta_fwd(*x, h0=h0, cu_seqlens=cu), *gla.gla_delta_bwd(*x, dO, h0=h0, cu_seqlens=cu)]
    assert torch.equal(want[0], gla.gla_delta_fwd(*x, scale=SCALE, h0=h0, cu_seqlens=cu)[0])
    with gla.debug_bounds_library():
        got = [*gla.gla_delta_fwd(*x, h0=h0, cu_seqlens=cu), *gla.gla_delta_bwd(*x, dO, h0=h0, cu_seqlens=cu)]
        assert gla.gla_get_device_error() == 0
    for a, c in zip(want, got):
        assert torch.equal(a, c), far(a, c)


def test_waits_that_run_out():
    """With a limit of 1 us a wait that blocks gives up: the call ends, the error is reported, the next one is right."""
    b = Batch(24, [700] * 3, 16, BF, packed=False)
    x, dO, h0 = b.inputs(), b.dev("dO")[0], b.h0.cuda()
    want = [*gla.gla_delta_fwd(*x, h0=h0), *gla.gla_delta_bwd(*x, dO, h0=h0)]
    assert gla.gla_get_device_error() == 0
    for call in (lambda: gla.gla_delta_fwd(*x, h0=h0), lambda: gla.gla_delta_bwd(*x, dO, h0=h0)):
        gla.gla_set_wait_limit_ns(1000)
        try:
            call()
            assert gla.gla_get_device_error() == -8
        finally:
            gla.gla_set_wait_limit_ns(2_000_000_000)
    got = [*gla.gla_delta_fwd(*x, h0=h0), *gla.gla_delta_bwd(*x, dO, h0=h0)]
    assert gla.gla_get_device_error() == 0
    for a, c in zip(want, got):
        assert torch.equal(a, c)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta", "dO"])
def test_nan_beside_a_ragged_end(name, dtype):
    """Chunks that end inside a sequence's last 64 tokens share their rows with the next sequence's first ones: a NaN there
    stays out of every result of the sequence before it, of the one after it and of the other head."""
    b = Batch(25, [100, 70, 65], 2, dtype)

    def run():
        x, dO = b.inputs(), b.dev("dO")[0]
        o, hT = gla.gla_delta_fwd(*x, h0=b.h0.cuda(), cu_seqlens=b.cu_dev)
        *rows, dh0 = gla.gla_delta_bwd(*x, dO, h0=b.h0.cuda(), dhT=b.dhT.cuda(), cu_seqlens=b.cu_dev)
        return [o, *rows], [hT, dh0]

    rows, states = run()
    b.x[name][103, 1] = float("nan")
    rows2, states2 = run()
    for x, y in zip(rows, rows2):
        assert torch.equal(x[:100], y[:100]) and torch.equal(x[170:], y[170:]) and torch.equal(x[:, 0], y[:, 0])
    for x, y in zip(states, states2):
        assert torch.equal(x[[0, 2]], y[[0, 2]]) and torch.equal(x[:, 0], y[:, 0])
    assert not all(bool(torch.isfinite(y).all()) for y in rows2)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_slices_of_a_packed_array(dtype):
    """Three heads: a token's gates are 6 or 12 bytes, so that slices of g and beta start off 16-byte boundaries."""
    b = Batch(26, [90], 3, dtype)
    x, dO = b.inputs(), b.dev("dO")[0]
    part, cu = [t[17:80] for t in x], i32([0, 63])
    own = [t.clone() for t in part]
    for t, c in zip(gla.gla_delta_fwd(*part, cu_seqlens=cu), gla.gla_delta_fwd(*own, cu_seqlens=cu)):
        assert torch.equal(t, c)
    for t, c in zip(gla.gla_delta_bwd(*part, dO[17:80], cu_seqlens=cu), gla.gla_delta_bwd(*own, dO[17:80].clone(), cu_seqlens=cu)):
        assert torch.equal(t, c)
    pool = torch.randn(5, 3, DK, DV, device="cuda")
    a, c = pool.clone(), pool.clone()
    assert torch.equal(gla.gla_delta_decode_step(*[t[13:18] for t in x], a), gla.gla_delta_decode_step(*[t[13:18].clone() for t in x], c))
    assert torch.equal(a, c)
    flat = torch.zeros(90 * 3 * DK + 1, dtype=dtype, device="cuda")[1:].view(90, 3, DK)
    with pytest.raises(gla.GlaError):
        gla.gla_delta_fwd(flat, *x[1:], cu_seqlens=b.cu_dev)


def test_long_sequences():
    """Two sequences of dozens of chunks: the forward against the recurrence, the bf16 backward against the fp32 one on the
    same values (which lies 1e-3 of the bf16 bound from the exact result)."""
    b = Batch(27, [5000, 4033], 2, BF)
    x, dO, cu = b.inputs(), b.dev("dO")[0], b.cu_dev
    o, hT = gla.gla_delta_fwd(*x, h0=b.h0.cuda(), cu_seqlens=cu)
    check_fwd(b, o, hT, b.h0)
    wide = [t.float() for t in x]
    o32, hT32 = gla.gla_delta_fwd(*wide, h0=b.h0.cuda(), cu_seqlens=cu)
    check(o, o32, "bf16", "o")
    check(hT, hT32, "state", "hT")
    got = gla.gla_delta_bwd(*x, dO, h0=b.h0.cuda(), dhT=b.dhT.cuda(), cu_seqlens=cu)
    want = gla.gla_delta_bwd(*wide, dO.float(), h0=b.h0.cuda(), dhT=b.dhT.cuda(), cu_seqlens=cu)
    for name, g, w in zip((*NAMES, "dh0"), got, want):
        check(g, w, "state" if name == "dh0" else "bf16", name)
