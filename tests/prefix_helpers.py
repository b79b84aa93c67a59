"""Inputs and 64-bit references of the shared-prefix tests: sequences that continue pool states,
each with a tail of tokens.  The references are the written-out sums, on numpy arrays."""
import numpy as np

import glasynth as gs
import oracle

DK, DV = 96, 192
SCALE = float(gs.SCALE)


def powers(ll, n):
    """lambda^n in 64 bits (lambda^0 = 1 also for log lambda = -inf); n an integer array >= 0."""
    n = np.asarray(n, np.float64)
    with np.errstate(invalid="ignore"):
        return np.where(n == 0, 1.0, np.exp(np.float64(ll) * n))


class Tails:
    """Host tails: what the device arrays hold (elements, or codes and scales), and their values."""

    def __init__(self, seed, rows, H, cap, fmt, bf16):
        k = gs.normal(seed, 21, (rows, H, cap, DK), 1 / np.sqrt(DK))
        v = gs.normal(seed, 22, (rows, H, cap, DV))
        if bf16:
            k, v = gs.bf16_round(k), gs.bf16_round(v)
        self.fmt, self.bf16 = fmt, bf16
        if fmt == "mxfp8":
            (self.kc, self.ks), (self.vc, self.vs) = oracle.mxfp8_quantize(k), oracle.mxfp8_quantize(v)
            self.k, self.v = oracle.mxfp8_dequantize(self.kc, self.ks), oracle.mxfp8_dequantize(self.vc, self.vs)
        else:
            self.k, self.v = k.astype(np.float64), v.astype(np.float64)

    def spoil(self, slots, lens):
        """NaN in every place that no sequence's tail holds."""
        used = np.zeros(self.k.shape[:1] + self.k.shape[2:3], bool)
        for s, n in zip(slots, lens):
            used[s, :n] = True
        for r in range(used.shape[0]):
            at = ~used[r]
            if self.fmt == "mxfp8":
                self.kc[r][:, at], self.vc[r][:, at] = 0x7F, 0x7F
                self.ks[r][:, at], self.vs[r][:, at] = 255, 255
            else:
                self.k[r][:, at], self.v[r][:, at] = np.nan, np.nan

    def device(self, dev="cuda"):
        import torch

        import linear_attention_recurrence_simple_gb300 as gla
        if self.fmt == "mxfp8":
            return gla.GlaTail(*(torch.from_numpy(x.copy()).to(dev) for x in (self.kc, self.vc, self.ks, self.vs)))
        dt = torch.bfloat16 if self.bf16 else torch.float32
        return gla.GlaTail(torch.from_numpy(self.k).to(dt).to(dev), torch.from_numpy(self.v).to(dt).to(dev))  # (converted on the host: one NaN pattern)


def ref_decode(q, k, v, ll, scale, pool, prefix_row, tk, tv, slots, lens):
    """o [N, H, 192] and the sum of the magnitudes of its terms."""
    N, H = q.shape[:2]
    o, mag = np.zeros((N, H, DV)), np.zeros((N, H, DV))
    for n in range(N):
        L = lens[n]
        for h in range(H):
            S = pool[prefix_row[n], h].astype(np.float64)
            K, V = tk[slots[n], h, :L], tv[slots[n], h, :L]
            x, y, z = q[n, h].astype(np.float64), k[n, h].astype(np.float64), v[n, h].astype(np.float64)
            w = powers(ll[h], L - np.arange(L))
            lam = powers(ll[h], L + 1)
            o[n, h] = scale * (lam * (x @ S) + (w * (K @ x)) @ V + (x @ y) * z)
            a = np.abs(x)
            mag[n, h] = abs(scale) * (lam * (a @ np.abs(S)) + (w * (np.abs(K) @ a)) @ np.abs(V) + (a @ np.abs(y)) * np.abs(z))
    return o, mag


def ref_fold(ll, pool, prefix_row, tk, tv, slots, lens):
    """States [N, H, 96, 192] and the sum of the magnitudes of their terms."""
    N, H = len(lens), pool.shape[1]
    s, mag = np.zeros((N, H, DK, DV)), np.zeros((N, H, DK, DV))
    for n in range(N):
        L = lens[n]
        for h in range(H):
            S = pool[prefix_row[n], h].astype(np.float64)
            K, V = tk[slots[n], h, :L], tv[slots[n], h, :L]
            w, lam = powers(ll[h], L - 1 - np.arange(L))[:, None], powers(ll[h], L)
            s[n, h] = lam * S + (w * K).T @ V
            mag[n, h] = lam * np.abs(S) + (w * np.abs(K)).T @ np.abs(V)
    return s, mag
