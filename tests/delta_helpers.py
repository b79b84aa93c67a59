"""The gated delta rule in 64 bits, token by token (tests only), inputs for it, and its bounds.

Bounds (2-norm of the error over 2-norm of the result, and the largest error over its rms).
  fp32 outputs of fp32 calls: sums of at most 192 + 64 products whose operands keep 22 bits, a few of them in a row,
      errors of random sign: sqrt(256) 2^-22 each if all were the largest, 4e-6; the gates' exp 2^-22 more.  1e-5,
      and 40 times that for the largest of at most 10^6 elements (5 sigma, and operands up to 8 rms).
  states of bf16 calls: operands that are not bf16 are sums of two, each rounding off by 2^-8: 2^-16 of the
      operand.  Along the way from a state to the next, four are split (state, weighted residuals, Z, weighted updates):
      4 2^-16 = 6e-5 if all errors were the largest and of one sign; at random signs and uniform in the binade the
      rms of one is 2^-16 / sqrt(3) x 0.72, together 1.3e-5.  2e-5, and 40 times that.
  bf16 outputs: the output's own rounding (2^-8 at most) and that of two operands that are held in one bf16 (P or
      dP, a state): 3 2^-8 = 1.2e-2 if all were the largest.  1e-2 in the 2-norm, where they are not, and for the
      largest error 3 2^-8 of the largest element (8 rms at most) and of the operands' sums, 0.25 of the rms."""
import numpy as np
import torch

DK, DV = 96, 192
SCALE = DK ** -0.5
NORM = {"f32": 1e-5, "state": 2e-5, "bf16": 1e-2}
MOST = {"f32": 4e-4, "state": 8e-4, "bf16": 0.25}


def far(x, ref):
    """(2-norm error, largest error over the rms)."""
    x, ref = x.detach().double().cpu(), ref.detach().double().cpu()
    assert x.shape == ref.shape, (x.shape, ref.shape)
    if ref.numel() == 0:
        return 0.0, 0.0
    d, norm = x - ref, float(ref.norm())
    if norm == 0:
        return (0.0, 0.0) if float(d.abs().max()) == 0 else (np.inf, np.inf)
    return float(d.norm()) / norm, float(d.abs().max()) / (norm / np.sqrt(ref.numel()))


def check(x, ref, kind, name=""):
    norm, most = far(x, ref)
    assert norm <= NORM[kind] and most <= MOST[kind], f"{name}: {norm:.2e} of {NORM[kind]:.0e}, {most:.2e} of {MOST[kind]:.0e}"


def ref_fwd(q, k, v, g, beta, S, scale=SCALE):
    """One sequence: [L, H, d] and S [H, 96, 192], all in 64 bits.  Returns o and the final state."""
    o = torch.zeros_like(v)
    for t in range(q.shape[0]):
        S = S * torch.exp(g[t])[:, None, None]
        u = beta[t][:, None] * (v[t] - torch.einsum("hac,ha->hc", S, k[t]))
        S = S + k[t][:, :, None] * u[:, None, :]
        o[t] = scale * torch.einsum("hac,ha->hc", S, q[t])
    return o, S


def ref_bwd(q, k, v, g, beta, S0, dO, dS, scale=SCALE):
    """Gradients (dq, dk, dv, dg, dbeta, dS0) by the reverse recurrence."""
    states = [S0]
    for t in range(q.shape[0]):
        states.append(ref_fwd(q[t:t + 1], k[t:t + 1], v[t:t + 1], g[t:t + 1], beta[t:t + 1], states[-1])[1])
    out = [torch.zeros_like(x) for x in (q, k, v, g, beta)]
    for t in range(q.shape[0] - 1, -1, -1):
        dS = dS + scale * q[t][:, :, None] * dO[t][:, None, :]
        out[0][t] = scale * torch.einsum("hac,hc->ha", states[t + 1], dO[t])
        a = torch.exp(g[t])[:, None, None]
        D = a * states[t]
        x = v[t] - torch.einsum("hac,ha->hc", D, k[t])
        du = torch.einsum("hac,ha->hc", dS, k[t])
        dv = beta[t][:, None] * du
        out[1][t] = torch.einsum("hac,hc->ha", dS, beta[t][:, None] * x) - torch.einsum("hac,hc->ha", D, dv)
        out[2][t], out[4][t] = dv, (du * x).sum(-1)
        dD = dS - k[t][:, :, None] * dv[:, None, :]
        out[3][t] = (dD * D).sum((1, 2))
        dS = a * dD
    return out + [dS]


class Batch:
    """Packed (or equal-length) inputs on the device and their values in 64 bits on the host."""

    def __init__(self, seed, lens, H, dtype, packed=True, spare=0, unit=True):
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.H, self.dtype, self.packed = list(lens), H, dtype, packed
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        T = int(self.cu[-1]) + spare
        r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
        norm = torch.nn.functional.normalize
        self.x = {"q": norm(r(T, H, DK), dim=-1), "k": norm(r(T, H, DK), dim=-1) if unit else r(T, H, DK) / 30,
                  "v": r(T, H, DV), "g": -torch.nn.functional.softplus(r(T, H)) * 2.0 ** -torch.arange(H).float(),
                  "beta": torch.sigmoid(r(T, H)), "dO": r(T, H, DV)}
        N = len(self.lens)
        self.h0, self.dhT = r(N, H, DK, DV) * 0.1, r(N, H, DK, DV) * 0.05

    def host(self, n, name):
        x = self.x[name].to(self.dtype).double()
        return x[self.cu[n]:self.cu[n + 1]]

    def dev(self, *names):
        out = []
        for name in names:
            x = self.x[name].to(self.dtype)
            out.append((x if self.packed else x.reshape(len(self.lens), self.lens[0], *x.shape[1:])).cuda().contiguous())
        return out

    def inputs(self):
        return self.dev("q", "k", "v", "g", "beta")

    @property
    def cu_dev(self):
        return torch.from_numpy(self.cu).cuda() if self.packed else None

    def rows(self, x):
        """A device result in the packed layout, without rows behind the last sequence."""
        return (x if self.packed else x.flatten(0, 1))[:int(self.cu[-1])]

    def ref(self, n, S0):
        return ref_fwd(*(self.host(n, m) for m in ("q", "k", "v", "g", "beta")), S0.double())

    def ref_bwd(self, n, S0, dS):
        return ref_bwd(*(self.host(n, m) for m in ("q", "k", "v", "g", "beta")), S0.double(), self.host(n, "dO"), dS.double())


def plan_ref(new_len, held, seen, rows, budget):
    """The slot plan, request by request."""
    free = sorted(set(range(rows)) - {h for h, n in zip(held, new_len) if h >= 0 and n >= 0})
    left, cu, slot, start, row, seq, pos = budget, [0], [], [], [], [], []
    for i, (n, h) in enumerate(zip(new_len, held)):
        got, r = 0, h if n >= 0 else -1
        if n > 0 and left > 0:
            if h >= 0:
                got = min(n, left)
            elif free:
                r, got = free.pop(0), min(n, left)
        left -= got
        cu.append(cu[-1] + got)
        slot.append(r if got else -1)
        start.append(h if got and h >= 0 else -1)
        row.append(r)
        seq += [i] * got
        pos += [(seen[i] if seen is not None else 0) + j for j in range(got)]
    pad = [-1] * (budget - len(seq))
    return cu, slot, start, row, seq + pad, pos + pad
