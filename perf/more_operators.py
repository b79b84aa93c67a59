"""Measured cases of the gated delta rule and of the maps that feed it.

Per head a 96 x 192 state S with a decay exp(g_t) and a writing strength beta_t of every token's own:

    S_t = exp(g_t) S_{t-1} + k_t u_t^T,   u_t = beta_t (v_t - exp(g_t) S_{t-1}^T k_t),   o_t = S_t^T (scale q_t)

    fwd      chunked forward, equal lengths or packed sequences that start from and leave rows of a pool
    bwd      gradients of q, k, v, g, beta and the initial states
    decode   one token for N sequences on a pool of states, in place
    plan     one step's maps from request lengths: packed offsets, pool rows, each token's place

`own = False` computes the same in elementary torch operations in 32 bits (decays in 64, since what is
left of a decay is a difference of sums); `exact` in 64 bits, token by token.
"""
import math
import random

import torch

own = False

DK, DV, C = 96, 192, 64
SCALE = DK ** -0.5


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # A short question alone: the latency of a prefill.
        dict(name="fwd_1x16_short", op="fwd", N=1, H=16, max_len=45, ragged=False, pool=False, dtype="bf16"),
        # The training forward: 8 sequences of 2,048 tokens.
        dict(name="fwd_8x2048x16", op="fwd", N=8, H=16, max_len=2048, ragged=False, pool=False, dtype="bf16"),
        # Prompts of a serving step, an odd number of heads, from and to rows of the pool.
        dict(name="fwd_24x7_pool", op="fwd", N=24, H=7, max_len=1100, ragged=True, pool=True, dtype="bf16"),
        # The all-fp32 mode on a few ragged sequences.
        dict(name="fwd_5x3_f32", op="fwd", N=5, H=3, max_len=190, ragged=True, pool=True, dtype="f32"),
        # Gradients in fp32, a sequence ending inside a chunk.
        dict(name="bwd_2x4_f32", op="bwd", N=2, H=4, max_len=150, ragged=True, pool=False, dtype="f32"),
        # Responses of a training step, packed.
        dict(name="bwd_40x16_packed", op="bwd", N=40, H=16, max_len=500, ragged=True, pool=False, dtype="bf16"),
        # The training backward.
        dict(name="bwd_8x2048x16", op="bwd", N=8, H=16, max_len=2048, ragged=False, pool=False, dtype="bf16"),
        # One sequence's next token: latency.
        dict(name="decode_1x16", op="decode", N=1, H=16, dtype="bf16", state="f32"),
        # An odd batch and an odd number of heads over a bf16 pool.
        dict(name="decode_333x7_bf16_pool", op="decode", N=333, H=7, dtype="bf16", state="bf16"),
        # 1,280 concurrent sequences.
        dict(name="decode_1280x16", op="decode", N=1280, H=16, dtype="bf16", state="f32"),
        # A small server's step.
        dict(name="plan_48", op="plan", N=48, rows=64, budget=2048, dtype="i32"),
        # A full batch with prefills among the decodes, more requests than rows.
        dict(name="plan_5000", op="plan", N=5000, rows=4096, budget=65536, dtype="i32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "fwd", "bwd", "bwd", "decode", "decode", "plan"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    H = rng.choice([1, 2, 3, 4, 7, 8, 13, 16, 16, 16])
    if op == "plan":
        N = _log_int(rng, 1, 5000)
        return dict(op=op, N=N, rows=_log_int(rng, max(1, N // 2), max(2, 2 * N)), budget=_log_int(rng, 64, 65536),
                    dtype="i32")
    if op == "decode":
        return dict(op=op, N=_log_int(rng, 1, 1000), H=H, dtype=dtype, state=rng.choice(["f32", "f32", "bf16"]))
    tokens = 12000 if dtype == "bf16" else 1500
    max_len = _log_int(rng, 1, 2000 if dtype == "bf16" else 400)
    N = _log_int(rng, 1, max(1, min(48, tokens // max_len)))
    ragged = rng.random() < 0.6
    return dict(op=op, N=N, H=H, max_len=max_len, ragged=ragged, pool=op == "fwd" and ragged and rng.random() < 0.6,
                dtype=dtype)


def _lengths(case):
    """Host token counts: ragged calls have the longest at max_len and (from three sequences on) one
    that is empty.  Fixed by the case; the seed sets their order."""
    n, m = case["N"], case["max_len"]
    if not case["ragged"]:
        return [m] * n
    r = random.Random("lengths %s" % sorted((k, v) for k, v in case.items() if k != "name"))
    x = [m] + [r.randint(max(1, m // 8), m) for _ in range(n - 1)]
    if n >= 3:
        x[1] = 0
    return x


def work(case):
    if case["op"] == "plan":
        b = case["N"] * 4 * (3 + 4) + case["budget"] * 8
        return {"bytes": float(b), "flops": float(4 * case["N"] + 2 * case["budget"])}
    N, H, e = case["N"], case["H"], 2 if case["dtype"] == "bf16" else 4
    state = DK * DV * 4
    qkv, gates = (2 * DK + DV) * e, 2 * e
    if case["op"] == "decode":
        es = 2 if case["state"] == "bf16" else 4
        return {"bytes": float(N * H * (2 * DK * DV * es + qkv + gates + DV * e)), "flops": float(N * H * 7 * DK * DV)}
    tokens = sum(_lengths(case))
    if case["op"] == "fwd":
        states = N * H * state * (2 if case["pool"] else 1)
        return {"bytes": float(tokens * H * (qkv + gates + DV * e) + states), "flops": float(tokens * H * 7 * DK * DV)}
    return {"bytes": float(tokens * H * (2 * (qkv + gates) + DV * e) + 3 * N * H * state),
            "flops": float(tokens * H * 20 * DK * DV)}


# ----------------------------------------------------------------------------------------- inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    r = random.Random("%d rows" % seed)

    def normal(*shape, sigma=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=gen, device=dev) * sigma).to(dtype)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    s = {"case": dict(case)}
    N = case["N"]
    if case["op"] == "plan":
        # most requests bring one token, some a prompt, some none; a few have finished (-1)
        R = case["rows"]
        free = r.sample(range(R), R)
        new, held, seen = [], [], []
        for _ in range(N):
            kind = r.random()
            has = free and kind < 0.8
            held.append(free.pop() if has and r.random() < 0.9 else -1)
            new.append(-1 if kind < 0.06 else 0 if kind < 0.14 else 1 if kind < 0.8 else r.randint(2, 600))
            seen.append(r.randint(1, 4000) if held[-1] >= 0 else 0)
        s.update(new_len=ints(new), held=ints(held), seen=ints(seen))
        return s

    H, dt = case["H"], _dtype(case)

    def tokens(*lead):
        """Unit queries and keys, a gate of each head's own range, strengths in (0, 1)."""
        q, k = (torch.nn.functional.normalize(normal(*lead, H, DK), dim=-1).to(dt) for _ in range(2))
        rate = torch.exp2(torch.linspace(-7, 1, H, device=dev))
        g = (-rate * torch.nn.functional.softplus(normal(*lead, H))).to(dt)
        return dict(q=q, k=k, v=normal(*lead, H, DV, dtype=dt), g=g, beta=torch.sigmoid(normal(*lead, H)).to(dt))

    if case["op"] == "decode":
        R = N + 3
        s.update(tokens(N), slot=ints(r.sample(range(R), N)))
        s["state"] = normal(R, H, DK, DV, sigma=0.1, dtype=torch.bfloat16 if case["state"] == "bf16" else torch.float32)
        return s
    lengths = _lengths(case)
    r.shuffle(lengths)
    s["lengths"], s["max"] = lengths, max(lengths)
    if case["ragged"]:
        cu = [0]
        for x in lengths:
            cu.append(cu[-1] + x)
        T = cu[-1]
        s.update(tokens(T), cu=ints(cu))
        # of each packed row: its sequence and its place in it (a program that packs has both)
        s["seq"] = torch.repeat_interleave(torch.arange(N, device=dev), ints(lengths).long(), output_size=T)
        s["at"] = torch.arange(T, device=dev) - s["cu"].long()[s["seq"]]
        lead = (T,)
    else:
        lead = (N, lengths[0])
        s.update(tokens(*lead))
    if case["pool"]:
        # sequences that go on from their pool row and new ones (-1); an empty one has no row
        R = N + 2
        rows = r.sample(range(R), N)
        s["pool"] = normal(R, H, DK, DV, sigma=0.1)
        s["slot"] = ints([x if n else -1 for x, n in zip(rows, lengths)])
        s["start"] = ints([x if n and r.random() < 0.5 else -1 for x, n in zip(rows, lengths)])
    if case["op"] == "bwd":
        s["h0"], s["dhT"] = normal(N, H, DK, DV, sigma=0.1), normal(N, H, DK, DV, sigma=0.01)
        s["dO"] = normal(*lead, H, DV, dtype=dt)
    return s


# -------------------------------------------------------------------------------------------- run
def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import linear_attention_recurrence_simple_gb300 as gla
        if op == "plan":
            return list(gla.gla_slot_plan(s["new_len"], s["held"], s["seen"], case["rows"], case["budget"]))
        x = [s[n] for n in ("q", "k", "v", "g", "beta")]
        if op == "decode":
            o = gla.gla_delta_decode_step(*x, s["state"], slot=s["slot"], scale=SCALE)
            return [o, s["state"]]
        if op == "bwd":
            return list(gla.gla_delta_bwd(*x, s["dO"], scale=SCALE, h0=s["h0"], dhT=s["dhT"], cu_seqlens=s.get("cu")))
        if case["pool"]:
            return list(gla.gla_delta_fwd(*x, scale=SCALE, h0=s["pool"], h0_row=s["start"], hT=s["pool"],
                                          hT_row=s["slot"], cu_seqlens=s["cu"]))
        return list(gla.gla_delta_fwd(*x, scale=SCALE, cu_seqlens=s.get("cu")))
    return {"plan": _plain_plan, "decode": _plain_decode, "bwd": _plain_bwd, "fwd": _plain_fwd}[op](s)


def _plain_plan(s):
    R, budget = s["case"]["rows"], s["case"]["budget"]
    new, held, seen = s["new_len"].long(), s["held"].long(), s["seen"].long()
    dev = new.device
    keep = (held >= 0) & (new >= 0)
    taken = torch.zeros(R + 1, dtype=torch.bool, device=dev)
    taken[torch.where(keep, held, R)] = True
    free = torch.argsort(taken[:R].to(torch.int32), stable=True)  # the free rows first, lowest to highest
    wants = (new > 0) & (held < 0)
    rank = torch.cumsum(wants, 0) - 1
    placed = wants & (rank < R - taken[:R].sum())
    ends = torch.cumsum(torch.where(placed | (keep & (new > 0)), new, 0), 0).clamp(max=budget)
    cu = torch.cat([torch.zeros(1, dtype=ends.dtype, device=dev), ends])
    got = cu[1:] > cu[:-1]
    row = torch.where(keep, held, torch.where(placed & got, free[rank.clamp(min=0, max=R - 1)], -1))
    slot = torch.where(got, row, -1)
    start = torch.where(got & keep, held, -1)
    t = torch.arange(budget, device=dev)
    seq = torch.searchsorted(ends, t, right=True)
    there = t < cu[-1]
    seq = torch.where(there, seq, 0)
    pos = torch.where(there, seen[seq] + t - cu[seq], -1)
    return [x.to(torch.int32) for x in (cu, slot, start, row, torch.where(there, seq, -1), pos)]


def _plain_decode(s):
    q, k, v, g, b = (s[x].float() for x in ("q", "k", "v", "g", "beta"))
    slot = s["slot"].long()
    S = s["state"][slot].float() * torch.exp(g)[..., None, None]
    u = b[..., None] * (v - (k[..., None] * S).sum(2))
    S = S + k[..., None] * u[..., None, :]
    o = (q[..., None] * S).sum(2) * SCALE
    s["state"][slot] = S.to(s["state"].dtype)
    return [o.to(s["q"].dtype), s["state"]]


def _chunks(s, x):
    """Rows [N, L, H, ...] or packed [T, H, ...] to [N, H, chunks, C, ...], zeros behind a sequence's
    end (a key and a strength of zero leave the state as it is)."""
    n = -(-max(s["max"], 1) // C) * C
    if "cu" in s:
        out = x.new_zeros((s["case"]["N"], n) + x.shape[1:])
        out = out.index_put((s["seq"], s["at"]), x)
    else:
        out = torch.cat([x, x.new_zeros((x.shape[0], n - x.shape[1]) + x.shape[2:])], 1)
    return out.transpose(1, 2).unflatten(2, (-1, C))


def _rows(s, x):
    """[N, H, L, ...] back to the call's layout."""
    x = x.transpose(1, 2)
    return x[s["seq"], s["at"]] if "cu" in s else x[:, :s["max"]]


def _plain_delta(s, q, k, v, g, b, S):
    """The chunked form: with G the sums of g in a chunk, A_ij = b_i exp(G_i - G_j) (k_i . k_j) for
    j < i, U = (1 + A)^-1 b (V - exp(G) K S)."""
    q, k, v, g, b = (_chunks(s, x) for x in (q, k, v, g, b))
    G = torch.cumsum(g.double(), -1)
    i = torch.arange(C, device=q.device)
    D = torch.exp(torch.where(i[:, None] >= i, G[..., :, None] - G[..., None, :], -math.inf)).float()
    F, E, L = (torch.exp(x).float()[..., None] for x in (G, G[..., -1:] - G, G[..., -1:]))
    b = b[..., None]
    X = -b * torch.tril(D * (k @ k.transpose(-1, -2)), -1)
    inv = torch.eye(C, device=q.device) + X  # 1 + X + X^2 + ...: X^64 = 0
    for _ in range(5):
        X = X @ X
        inv = inv + inv @ X
    P = D * (q @ k.transpose(-1, -2))
    o = []
    for c in range(q.shape[2]):
        U = inv[:, :, c] @ (b[:, :, c] * (v[:, :, c] - F[:, :, c] * (k[:, :, c] @ S)))
        o.append(SCALE * (F[:, :, c] * (q[:, :, c] @ S) + P[:, :, c] @ U))
        S = L[:, :, c] * S + (E[:, :, c] * k[:, :, c]).transpose(-1, -2) @ U
    return _rows(s, torch.cat(o, 2)), S


def _plain_fwd(s):
    x = [s[n].float() for n in ("q", "k", "v", "g", "beta")]
    N, H = s["case"]["N"], s["case"]["H"]
    if not s["case"]["pool"]:
        o, S = _plain_delta(s, *x, torch.zeros(N, H, DK, DV, device=x[0].device))
        return [o.to(s["q"].dtype), S]
    start, slot, pool = s["start"].long(), s["slot"].long(), s["pool"]
    o, S = _plain_delta(s, *x, torch.where((start >= 0).view(-1, 1, 1, 1), pool[start.clamp(min=0)], 0.0))
    # rows that no sequence has keep what they hold: -1 writes to a row behind the last
    into = torch.cat([pool, pool[:1]])
    into[torch.where(slot >= 0, slot, pool.shape[0])] = S
    pool.copy_(into[:-1])
    return [o.to(s["q"].dtype), pool]


def _plain_bwd(s):
    with torch.enable_grad():
        x = [s[n].detach().float().requires_grad_() for n in ("q", "k", "v", "g", "beta", "h0")]
        o, S = _plain_delta(s, *x)
        d = torch.autograd.grad([o, S], x, [s["dO"].float(), s["dhT"]])
    return [y.to(s["q"].dtype) for y in d[:5]] + [d[5]]


# ------------------------------------------------------------------------------------------ exact
def exact(case, seed):
    """The same outputs from the recurrence, token by token in 64 bits.  None for the maps, which are
    whole numbers."""
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    f8 = torch.float64
    q, k, v, g, b = (s[n].to(f8) for n in ("q", "k", "v", "g", "beta"))

    def step(S, k, v, g, b):
        S = S * torch.exp(g)[..., None, None]
        e = v - (S * k[..., None]).sum(-2)
        return S, e, S + k[..., None] * (b[..., None] * e)[..., None, :]

    if case["op"] == "decode":
        slot = s["slot"].long()
        _, _, S = step(s["state"][slot].to(f8), k, v, g, b)
        out = s["state"].to(f8)
        out[slot] = S
        return [SCALE * (S * q[..., None]).sum(-2), out]

    N, H, L = case["N"], case["H"], s["max"]
    lens = s["lengths"]
    ends = [sum(lens[:n + 1]) for n in range(N)]

    def pad(x):  # [L, N, H, ...]
        out = torch.zeros((L, N) + x.shape[1 if "cu" in s else 2:], dtype=f8, device=x.device)
        for n in range(N):
            out[:lens[n], n] = x[ends[n] - lens[n]:ends[n]] if "cu" in s else x[n, :lens[n]]
        return out

    def unpad(x):
        rows = [x[:lens[n], n] for n in range(N)]
        return torch.cat(rows) if "cu" in s else torch.stack(rows)

    q, k, v, g, b = (pad(x) for x in (q, k, v, g, b))
    if case["op"] == "fwd":
        S = torch.zeros(N, H, DK, DV, dtype=f8, device=q.device)
        if case["pool"]:
            for n, row in enumerate(s["start"].tolist()):
                if row >= 0:
                    S[n] = s["pool"][row]
        o = torch.zeros_like(v)
        for t in range(L):
            _, _, S = step(S, k[t], v[t], g[t], b[t])
            o[t] = SCALE * (S * q[t][..., None]).sum(-2)
        if not case["pool"]:
            return [unpad(o), S]
        pool = s["pool"].to(f8)
        for n, row in enumerate(s["slot"].tolist()):
            if row >= 0:
                pool[row] = S[n]
        return [unpad(o), pool]

    dO = pad(s["dO"].to(f8))
    out = [torch.zeros_like(x) for x in (q, k, v, g, b)] + [torch.zeros(N, H, DK, DV, dtype=f8, device=q.device)]
    group = max(1, min(H, int(16e9 / ((L + 1) * N * DK * DV * 8))))  # heads at a time: the states of all tokens are kept
    for h0 in range(0, H, group):
        hs = slice(h0, min(H, h0 + group))
        qh, kh, vh, gh, bh, dOh = (x[:, :, hs] for x in (q, k, v, g, b, dO))
        states = torch.empty((L + 1, N, qh.shape[2], DK, DV), dtype=f8, device=q.device)
        states[0] = s["h0"][:, hs].to(f8)
        for t in range(L):
            states[t + 1] = step(states[t], kh[t], vh[t], gh[t], bh[t])[2]
        dS = s["dhT"][:, hs].to(f8)
        for t in range(L - 1, -1, -1):
            dS = dS + SCALE * qh[t][..., None] * dOh[t][..., None, :]
            out[0][t, :, hs] = SCALE * (states[t + 1] * dOh[t][..., None, :]).sum(-1)
            S, e, _ = step(states[t], kh[t], vh[t], gh[t], bh[t])
            du = (dS * kh[t][..., None]).sum(-2)
            de = bh[t][..., None] * du
            out[1][t, :, hs] = (dS * (bh[t][..., None] * e)[..., None, :]).sum(-1) - (S * de[..., None, :]).sum(-1)
            out[2][t, :, hs] = de
            out[4][t, :, hs] = (du * e).sum(-1)
            dS = dS - kh[t][..., None] * de[..., None, :]
            out[3][t, :, hs] = (dS * S).sum((-2, -1))
            dS = dS * torch.exp(gh[t])[..., None, None]
        out[5][:, hs] = dS
    return [unpad(x) for x in out[:5]] + [out[5]]
