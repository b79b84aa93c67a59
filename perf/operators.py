"""Measured cases of the shared-prefix operators: sequences that continue a common prefix.

A prefix (a prompt, a system message) is run once and leaves one 96 x 192 fp32 state per head in a
pool.  Any number of sequences then continue from that state: each has a tail of tokens of its own
(keys and values, in the call's type or as MXFP8: E4M3 codes with one E8M0 scale per 32 values).

    decode   one token for N sequences: readout of the shared states and of the tails, and the
             token's key and value written to the tail
    fold     tails folded into states of their own
    tail     packed tokens written to the tails (quantised as they are written) and read back
    fwd      packed continuations (questions after a system message, responses to a prompt)
    bwd      their gradients, with that of the shared states summed over the sequences

`own = False` computes the same in elementary torch operations in 32 bits; `exact` in 64 bits.
"""
import math
import random

import torch

own = False

DK, DV = 96, 192
SCALE = DK ** -0.5


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # Two samples of one prompt, a few tokens in: the latency of one decode step.
        dict(name="decode_2x16_bf16", op="decode", N=2, H=16, groups=1, max_len=24, dtype="bf16", tail="native"),
        # Best-of-64 sampling of one prompt, about a hundred tokens in, quantised tails.
        dict(name="decode_64x16_mxfp8", op="decode", N=64, H=16, groups=1, max_len=200, dtype="bf16", tail="mxfp8"),
        # A ragged serving batch of an odd size and an odd number of heads, five prompts, plain tails.
        dict(name="decode_333x7_bf16", op="decode", N=333, H=7, groups=5, max_len=255, dtype="bf16", tail="native"),
        # 1,280 concurrent sequences from twenty prompts, quantised tails.
        dict(name="decode_1280x16_mxfp8", op="decode", N=1280, H=16, groups=20, max_len=255, dtype="bf16", tail="mxfp8"),
        # A few tails of one chunk become states of their own.
        dict(name="fold_12x16_mxfp8", op="fold", N=12, H=16, groups=2, max_len=128, dtype="bf16", tail="mxfp8"),
        # Every tail of a batch that has outgrown its break-even length.
        dict(name="fold_256x16_bf16", op="fold", N=256, H=16, groups=8, max_len=384, dtype="bf16", tail="native"),
        # The last token of each sequence written and read back, all in fp32.
        dict(name="tail_40x16_f32", op="tail", N=40, H=16, groups=1, max_len=1, dtype="f32", tail="mxfp8"),
        # Suffix prompts written to the tails, quantised, and read back.
        dict(name="tail_200x16_mxfp8", op="tail", N=200, H=16, groups=1, max_len=500, dtype="bf16", tail="mxfp8"),
        # Eight questions after one system message.
        dict(name="fwd_8x16_bf16", op="fwd", N=8, H=16, groups=1, max_len=130, dtype="bf16", tail="native"),
        # Rollouts of a training step: eight responses to each of eight prompts.
        dict(name="fwd_64x16_bf16", op="fwd", N=64, H=16, groups=8, max_len=700, dtype="bf16", tail="native"),
        # Gradients of four short responses to one prompt, in fp32.
        dict(name="bwd_4x5_f32", op="bwd", N=4, H=5, groups=1, max_len=150, dtype="f32", tail="native"),
        # Gradients of the rollouts.
        dict(name="bwd_64x16_bf16", op="bwd", N=64, H=16, groups=8, max_len=500, dtype="bf16", tail="native"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "fold", "fold", "tail", "fwd", "bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    tail = rng.choice(["native", "mxfp8"])
    H = rng.choice([1, 3, 4, 8, 13, 16, 16, 16, 24])
    if op == "decode":
        N, max_len = _log_int(rng, 1, 1000), _log_int(rng, 1, 320)
        groups = _log_int(rng, 1, max(1, min(N, 40)))
    elif op == "fold":
        N, max_len = _log_int(rng, 1, 200), _log_int(rng, 1, 450)
        groups = _log_int(rng, 1, max(1, min(N, 20)))
    elif op == "tail":
        N, max_len = _log_int(rng, 1, 200), _log_int(rng, 1, 400)
        groups = 1
    else:
        N, max_len = _log_int(rng, 1, 60), _log_int(rng, 1, 400)
        if dtype == "f32":  # the all-fp32 mode is for checks: short runs
            N, max_len = min(N, 12), min(max_len, 200)
        groups = _log_int(rng, 1, max(1, min(N, 10)))
        H = min(H, 16)
        tail = "native"
    return dict(op=op, N=N, H=H, groups=groups, max_len=max_len, dtype=dtype, tail=tail)


def _lengths(case):
    """Host token counts of the case's sequences: ragged, with the longest at max_len and (from
    three sequences on) one that is empty.  Fixed by the case; the seed sets their order."""
    r = random.Random("lengths %s" % sorted((k, v) for k, v in case.items() if k != "name"))
    n, m = case["N"], case["max_len"]
    if m == 1:
        return [1] * n
    x = [m] + [r.randint(m // 8, m) for _ in range(n - 1)]
    if n >= 3 and case["op"] != "tail":
        x[1] = 0
    return x


def _token_bytes(case):
    """Stored bytes of one token of one head in a tail."""
    return (DK + DV) // 32 * 33 if case["tail"] == "mxfp8" else (DK + DV) * (2 if case["dtype"] == "bf16" else 4)


def work(case):
    N, H, G = case["N"], case["H"], case["groups"]
    L = sum(_lengths(case)) / N
    e = 2 if case["dtype"] == "bf16" else 4
    state, tok, qkv = DK * DV * 4, _token_bytes(case), (2 * DK + DV) * e
    if case["op"] == "decode":
        b = N * H * (L * tok + qkv + DV * e + tok) + G * H * state
        f = N * H * 2 * (DK * DV + (L + 1) * (DK + DV))
    elif case["op"] == "fold":
        b = N * H * (L * tok + state) + G * H * state
        f = N * H * 2 * DK * DV * (L + 1)
    elif case["op"] == "tail":
        b = N * H * L * 2 * (tok + (DK + DV) * e)
        f = N * H * L * 2 * (DK + DV)
    else:
        # the chunked form's least: the readout and the update of the state for every token
        tokens = N * L
        b = tokens * H * (qkv + DV * e) + G * H * state + N * H * state
        f = tokens * H * 4 * DK * DV
        if case["op"] == "bwd":
            b = tokens * H * (qkv + DV * e + qkv) + 2 * G * H * state + N * H * state
            f = tokens * H * 12 * DK * DV
    return {"bytes": float(b), "flops": float(f)}


# ----------------------------------------------------------------------------------------- inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _log_lambda(H, device):
    h = torch.arange(H, device=device, dtype=torch.float64)
    return torch.log1p(-torch.exp2(-(5 + 7 * h / max(1, H - 1)))).float()


def _mx_quantise(x):
    """fp32 [..., 32 m] to E4M3 codes (uint8) and E8M0 scales (uint8 [..., m]): the shared exponent
    is floor(log2 of the block's maximum) - 8, one more where the maximum would pass 448."""
    b = x.float().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    mant, ex = torch.frexp(top)  # top = mant 2^ex, mant in [0.5, 1)
    se = (ex - 9 + (mant > 0.875).to(ex.dtype)).clamp(-127, 127)
    se = torch.where(top < 2.0 ** -126, torch.full_like(se, -127), se)
    # 2^-se in two factors, each in range
    half = torch.div(-se, 2, rounding_mode="floor")
    y = torch.ldexp(torch.ldexp(b, half.unsqueeze(-1)), (-se - half).unsqueeze(-1))
    codes = y.to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2)
    return codes, (se + 127).to(torch.uint8)


def _mx_widen(codes, scales, dtype):
    b = codes.view(torch.float8_e4m3fn).to(dtype).unflatten(-1, (-1, 32))
    return torch.ldexp(b, (scales.to(torch.int32) - 127).unsqueeze(-1)).flatten(-2)


def _prefix_rows(case, r, P):
    """Pool row of each sequence: the sequences of a prompt stand together."""
    N, G = case["N"], case["groups"]
    cuts = sorted(r.sample(range(1, N), G - 1)) if G > 1 else []
    rows = r.sample(range(P), G)
    out = []
    for g, (a, b) in enumerate(zip([0] + cuts, cuts + [N])):
        out += [rows[g]] * (b - a)
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    r = random.Random("%d rows" % seed)
    N, H, dt = case["N"], case["H"], _dtype(case)

    def normal(*shape, sigma=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=dev) * sigma).to(dtype)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    lengths = _lengths(case)
    r.shuffle(lengths)
    P = case["groups"] + 2
    rows = _prefix_rows(case, r, P)
    s = {"case": dict(case), "log_lambda": _log_lambda(H, dev), "lengths": lengths, "max": max(lengths),
         "prefix_row": ints(rows), "len": ints(lengths)}
    if case["op"] != "tail":
        s["pool"] = normal(P, H, DK, DV, sigma=0.1, dtype=torch.float32)
    if case["op"] in ("tail", "fwd", "bwd"):
        T = sum(lengths)
        cu = [0]
        for x in lengths:
            cu.append(cu[-1] + x)
        s["T"], s["cu"] = T, ints(cu)
        s["q"], s["k"] = normal(T, H, DK, sigma=SCALE), normal(T, H, DK, sigma=SCALE)
        s["v"] = normal(T, H, DV)
        # of each packed row: its sequence and its place in it (a program that packs has both)
        s["seq"] = torch.repeat_interleave(torch.arange(N, device=dev), s["len"].long(), output_size=T)
        s["at"] = torch.arange(T, device=dev) - s["cu"].long()[s["seq"]]
    if case["op"] == "bwd":
        s["dO"] = normal(T, H, DV)
        s["dhT"] = normal(N, H, DK, DV, sigma=0.01, dtype=torch.float32)
    if case["op"] in ("decode", "fold", "tail"):
        cap = (max(lengths) + 1 + 15) // 16 * 16
        R = N + 3
        s["slot"] = ints(r.sample(range(R), N))
        # the whole cache holds tokens: what lies behind a sequence's last is an earlier one's
        k = normal(R, H, cap, DK, sigma=SCALE)
        v = normal(R, H, cap, DV)
        if case["tail"] == "mxfp8":
            (kc, ks), (vc, vs) = _mx_quantise(k), _mx_quantise(v)
            s["tail"] = (kc, vc, ks, vs)
        else:
            s["tail"] = (k, v, None, None)
    if case["op"] == "decode":
        s["q"], s["k"] = normal(N, H, DK, sigma=SCALE), normal(N, H, DK, sigma=SCALE)
        s["v"] = normal(N, H, DV)
    if case["op"] == "tail":
        # room for the new tokens behind the ones that are there
        s["pos"] = ints([0 if m == cap else r.randint(0, cap - m) for m in lengths])
    return s


# -------------------------------------------------------------------------------------------- run
def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import linear_attention_recurrence_simple_gb300 as gla
        if op == "decode":
            o = gla.gla_prefix_decode_step(s["q"], s["k"], s["v"], s["log_lambda"], s["pool"], s["prefix_row"],
                                           s["tail"], s["len"], tail_slot=s["slot"], scale=SCALE)
            return [o, _held(s["tail"])]
        if op == "fold":
            return gla.gla_tail_fold(s["log_lambda"], s["pool"], s["prefix_row"], s["tail"], s["len"],
                                     tail_slot=s["slot"])
        if op == "tail":
            gla.gla_tail_append(s["k"], s["v"], s["tail"], s["pos"], s["cu"], tail_slot=s["slot"])
            k, v = gla.gla_tail_read(s["tail"], s["pos"], s["cu"], s["T"], tail_slot=s["slot"], dtype=_dtype(case))
            return [k, v, _held(s["tail"])]
        if op == "fwd":
            return list(gla.gla_prefix_fwd(s["q"], s["k"], s["v"], s["log_lambda"], s["pool"], s["prefix_row"],
                                           s["cu"], scale=SCALE))
        return list(gla.gla_prefix_bwd(s["q"], s["k"], s["v"], s["log_lambda"], s["dO"], s["pool"], s["prefix_row"],
                                       s["cu"], scale=SCALE, dhT=s["dhT"]))
    return {"decode": _plain_decode, "fold": _plain_fold, "tail": _plain_tail, "fwd": _plain_fwd,
            "bwd": _plain_bwd}[op](s)


def _held(tail):
    """The tails as run() returns them: codes as the E4M3 values they are, scales as exponents."""
    k, v, ks, vs = tail
    return [k, v] if ks is None else [k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), ks, vs]


def _plain_tails(s, n):
    """Keys and values of the tails' first n tokens, in 32 bits: [N, H, n, 96 | 192]."""
    k, v, ks, vs = s["tail"]
    slot = s["slot"].long()
    if ks is None:
        return k[slot, :, :n].float(), v[slot, :, :n].float()
    return (_mx_widen(k[slot, :, :n], ks[slot, :, :n], torch.float32),
            _mx_widen(v[slot, :, :n], vs[slot, :, :n], torch.float32))


def _plain_write(s, row, at, k, v):
    """k, v [n, H, d] to places `at` of tail rows `row`."""
    tk, tv, tks, tvs = s["tail"]
    if tks is None:
        tk[row, :, at], tv[row, :, at] = k, v
    else:
        (tk[row, :, at], tks[row, :, at]), (tv[row, :, at], tvs[row, :, at]) = _mx_quantise(k), _mx_quantise(v)


def _plain_decode(s):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    n, ll, L = s["max"], s["log_lambda"], s["len"].long()
    S = s["pool"][s["prefix_row"].long()]
    o = (q.unsqueeze(-1) * S).sum(2) * torch.exp(ll * (L.unsqueeze(1) + 1)).unsqueeze(-1)
    tk, tv = _plain_tails(s, n)
    back = L.view(-1, 1, 1) - torch.arange(n, device=q.device)
    w = torch.where(back > 0, torch.exp(ll.view(1, -1, 1) * back.clamp(min=0)), 0.0) * (tk @ q.unsqueeze(-1)).squeeze(-1)
    o = o + (w.unsqueeze(2) @ tv).squeeze(2)
    o = o + (q * k).sum(-1, keepdim=True) * v
    _plain_write(s, s["slot"].long(), L, s["k"], s["v"])
    return [(o * SCALE).to(s["q"].dtype), _held(s["tail"])]


def _plain_fold(s):
    n, ll, L = s["max"], s["log_lambda"], s["len"].long()
    tk, tv = _plain_tails(s, n)
    back = L.view(-1, 1, 1) - 1 - torch.arange(n, device=tk.device)
    w = torch.where(back >= 0, torch.exp(ll.view(1, -1, 1) * back.clamp(min=0)), 0.0)
    out = (tk * w.unsqueeze(-1)).transpose(2, 3) @ tv
    return out + torch.exp(ll * L.unsqueeze(1)).view(*out.shape[:2], 1, 1) * s["pool"][s["prefix_row"].long()]


def _plain_tail(s):
    row, at = s["slot"].long()[s["seq"]], s["pos"].long()[s["seq"]] + s["at"]
    _plain_write(s, row, at, s["k"], s["v"])
    k, v, ks, vs = s["tail"]
    if ks is None:
        return [k[row, :, at], v[row, :, at], _held(s["tail"])]
    dt = s["k"].dtype
    return [_mx_widen(k[row, :, at], ks[row, :, at], torch.float32).to(dt),
            _mx_widen(v[row, :, at], vs[row, :, at], torch.float32).to(dt), _held(s["tail"])]


def _padded(s, x, dtype=torch.float32):
    """Packed rows [T, H, d] to [N, H, max, d], zeros behind the last row of a sequence."""
    out = torch.zeros((s["case"]["N"], s["max"]) + x.shape[1:], dtype=dtype, device=x.device)
    out[s["seq"], s["at"]] = x.to(dtype)
    return out.transpose(1, 2)


def _packed(s, x, dtype):
    return x.transpose(1, 2)[s["seq"], s["at"]].to(dtype)


def _plain_decays(s):
    """lambda^(i - j) for j <= i, else 0 [H, n, n]; lambda^(i + 1) [H, n, 1]; for every sequence
    lambda^(L - 1 - j) for j < L, else 0 [N, H, n, 1]; lambda^L [N, H, 1, 1]."""
    n, ll, L = s["max"], s["log_lambda"].view(-1, 1, 1), s["len"].view(-1, 1, 1, 1)
    i = torch.arange(n, device=ll.device)
    d = i.view(-1, 1) - i
    D = torch.where(d >= 0, torch.exp(ll * d.clamp(min=0)), 0.0)
    left = L - 1 - i.view(-1, 1)
    E = torch.where(left >= 0, torch.exp(ll * left.clamp(min=0)), 0.0)
    return D, torch.exp(ll * (i.view(-1, 1) + 1)), E, torch.exp(ll * L)


def _plain_fwd(s):
    q, k, v = (_padded(s, s[x]) for x in "qkv")
    D, F, E, G = _plain_decays(s)
    S = s["pool"][s["prefix_row"].long()]
    o = ((q @ k.transpose(2, 3)) * D) @ v + (q * F) @ S
    hT = (k * E).transpose(2, 3) @ v + G * S
    return [_packed(s, o * SCALE, s["q"].dtype), hT]


def _plain_bwd(s):
    q, k, v, dO = (_padded(s, s[x]) for x in ("q", "k", "v", "dO"))
    D, F, E, G = _plain_decays(s)
    S, R = s["pool"][s["prefix_row"].long()], s["dhT"]
    dt = s["q"].dtype
    dO = dO * SCALE
    dP = (dO @ v.transpose(2, 3)) * D
    dq = dP @ k + F * (dO @ S.transpose(2, 3))
    dk = dP.transpose(2, 3) @ q + E * (v @ R.transpose(2, 3))
    P = (q @ k.transpose(2, 3)) * D
    dv = P.transpose(2, 3) @ dO + E * (k @ R)
    dh0 = (q * F).transpose(2, 3) @ dO + G * R
    pick = (s["prefix_row"].view(1, -1) == torch.arange(s["pool"].shape[0], device=q.device).view(-1, 1)).float()
    dpool = (pick @ dh0.flatten(1)).view_as(s["pool"])
    return [_packed(s, dq, dt), _packed(s, dk, dt), _packed(s, dv, dt), dpool]


# ------------------------------------------------------------------------------------------ exact
def exact(case, seed):
    """The same outputs from the definition, S_t = lambda S_{t-1} + k_t v_t^T and
    o_t = S_t^T (scale q_t), in 64 bits, sequence by sequence and head by head in sums over pairs
    of tokens.  None for the tails: what they hold is a rounding, not a sum."""
    s = prepare(case, seed)
    op, H, f8 = case["op"], case["H"], torch.float64
    ll = s["log_lambda"].to(f8)
    rows, slots = s["prefix_row"].tolist(), s["slot"].tolist() if "slot" in s else []
    held = [None, None] if case["tail"] != "mxfp8" else [None] * 4
    if op == "tail":
        keep = []
        for name in "kv":
            x = s[name].to(f8)
            if case["tail"] == "mxfp8":
                b = x.unflatten(-1, (-1, 32))
                top = b.abs().amax(-1, keepdim=True)
                e = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
                e = torch.where(top * torch.exp2(8 - e) > 448, e + 1, e) - 8
                y = b * torch.exp2(-e)
                step = torch.exp2(torch.clamp(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -20))), min=-6) - 3)
                x = (torch.round(y / step) * step * torch.exp2(e)).flatten(-2)
            keep.append(x)
        return [keep[0], keep[1], held]

    def tail_of(n, L):
        k, v, ks, vs = (None if x is None else x[slots[n], :, :L] for x in s["tail"])
        if ks is None:
            return k.to(f8), v.to(f8)
        two = lambda c, e: c.view(torch.float8_e4m3fn).to(f8) * torch.exp2(e.to(f8) - 127).repeat_interleave(32, -1)  # noqa: E731
        return two(k, ks), two(v, vs)

    if op in ("decode", "fold"):
        out = []
        for n, L in enumerate(s["lengths"]):
            k, v = tail_of(n, L)
            S = s["pool"][rows[n]].to(f8)
            age = torch.arange(L - 1, -1, -1, device=ll.device, dtype=f8)
            w = torch.exp(ll[:, None] * age)
            if op == "fold":
                out.append(torch.exp(ll * L)[:, None, None] * S + torch.einsum("hja,hjc->hac", w[..., None] * k, v))
                continue
            q, kn, vn = (s[x][n].to(f8) for x in "qkv")
            o = torch.exp(ll * (L + 1))[:, None] * torch.einsum("ha,hac->hc", q, S)
            o = o + torch.einsum("hj,hjc->hc", torch.exp(ll)[:, None] * w * torch.einsum("ha,hja->hj", q, k), v)
            out.append(SCALE * (o + (q * kn).sum(-1, keepdim=True) * vn))
        x = torch.stack(out)
        return x if op == "fold" else [x, held]

    cu = s["cu"].tolist()
    parts = {x: [] for x in ("o", "hT", "dq", "dk", "dv")}
    dpool = torch.zeros_like(s["pool"], dtype=f8) if op == "bwd" else None
    for n, L in enumerate(s["lengths"]):
        q, k, v = (s[x][cu[n]:cu[n + 1]].to(f8).permute(1, 0, 2) for x in "qkv")
        q = q * SCALE
        S = s["pool"][rows[n]].to(f8)
        t = torch.arange(L, device=ll.device, dtype=f8)
        D = torch.exp(ll[:, None, None] * (t[:, None] - t).clamp(min=0)) * (t[:, None] >= t)
        f, e = torch.exp(ll[:, None] * (t + 1))[..., None], torch.exp(ll[:, None] * (L - 1 - t))[..., None]
        last = torch.exp(ll * L)[:, None, None]
        if op == "fwd":
            o = torch.einsum("hij,hjc->hic", torch.einsum("hia,hja->hij", q, k) * D, v) + f * torch.einsum("hia,hac->hic", q, S)
            parts["o"].append(o.permute(1, 0, 2))
            parts["hT"].append(last * S + torch.einsum("hja,hjc->hac", k * e, v))
            continue
        dO, R = s["dO"][cu[n]:cu[n + 1]].to(f8).permute(1, 0, 2), s["dhT"][n].to(f8)
        A = torch.einsum("hic,hjc->hij", dO, v) * D
        dq = torch.einsum("hij,hja->hia", A, k) + f * torch.einsum("hic,hac->hia", dO, S)
        dk = torch.einsum("hij,hia->hja", A, q) + e * torch.einsum("hjc,hac->hja", v, R)
        dv = torch.einsum("hij,hic->hjc", torch.einsum("hia,hja->hij", q, k) * D, dO) + e * torch.einsum("hja,hac->hjc", k, R)
        parts["dq"].append(SCALE * dq.permute(1, 0, 2))
        parts["dk"].append(dk.permute(1, 0, 2))
        parts["dv"].append(dv.permute(1, 0, 2))
        dpool[rows[n]] += last * R + torch.einsum("hia,hic->hac", q * f, dO)
    if op == "fwd":
        return [torch.cat(parts["o"]), torch.stack(parts["hT"])]
    return [torch.cat(parts["dq"]), torch.cat(parts["dk"]), torch.cat(parts["dv"]), dpool]
