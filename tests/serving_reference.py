"""Plain 64-bit CPU forms of the paged-pool operators and the sampler, for the
tests: NumPy loops written from the definitions in include/spectra.h."""
from __future__ import annotations

import numpy as np

import oracle


# ---------------------------------------------------------------- the pool's layout

class Pool:
    """A pool's buffers in host memory, in the packed layout."""

    def __init__(self, H, D, P, n_pages, rng=None):
        """Zeros, or (with a generator) what no kernel may let through: random
        codes and zero points, and scales that are infinities and NaN."""
        self.H, self.D, self.P, self.n_pages, self.G = H, D, P, n_pages, D // 32
        n, G = n_pages * H * P, D // 32
        self.codes = {w: np.zeros((n, 16 * G), np.uint8) for w in "kv"}
        self.scales = {w: np.zeros((n, G), np.uint16) for w in "kv"}
        self.zeros = {w: np.zeros(n, np.uint32) for w in "kv"}
        self.mass = np.zeros(n, np.float32)
        if rng is not None:
            for w in "kv":
                self.codes[w][:] = rng.integers(0, 256, self.codes[w].shape)
                self.scales[w][:] = rng.choice([0x7C00, 0xFC00, 0x7E00, 0xFE01], self.scales[w].shape)
                self.zeros[w][:] = rng.integers(0, 1 << (4 * G), n, dtype=np.uint64).astype(np.uint32)
            self.mass[:] = np.nan

    def slot(self, ts, h):
        return (ts // self.P * self.H + h) * self.P + ts % self.P

    def put(self, which, ts, h, codes, scales, zeros):
        """One vector: codes [D], FP16 scale bits [G], zero points [G]."""
        s, G = self.slot(ts, h), self.G
        c = codes.astype(np.uint8).reshape(G, 16, 2)
        rec = c[..., 0] | (c[..., 1] << 4)  # 16 bytes of a group, lowest channel first
        cut = 4 if which == "k" else 2
        self.codes[which][s] = rec.reshape(G, 16 // cut, cut).transpose(1, 0, 2).ravel()
        self.scales[which][s] = scales
        self.zeros[which][s] = sum(int(z) << (4 * g) for g, z in enumerate(zeros))

    def value(self, which, ts, h):
        """One vector, dequantised (FP64 [D]), from the packed bytes."""
        s, G = self.slot(ts, h), self.G
        cut = 4 if which == "k" else 2
        rec = self.codes[which][s].reshape(16 // cut, G, cut).transpose(1, 0, 2).reshape(G, 16)
        code = np.stack([rec & 15, rec >> 4], -1).reshape(G, 32).astype(np.float64)
        z = np.array([(int(self.zeros[which][s]) >> (4 * g)) & 15 for g in range(G)], np.float64)
        sc = self.scales[which][s].view(np.float16).astype(np.float64)
        return ((code - z[:, None]) * sc[:, None]).reshape(self.D)

    def append(self, k_bits, v_bits, slots):
        """The oracle's quantiser on BF16 bits [n_tok][H][D], into the slots."""
        n = len(slots)
        for which, x in (("k", k_bits), ("v", v_bits)):
            c = oracle.kv_cache(self.H, max(n, 1), self.D)
            if n:
                oracle.kv_quantize(c, x, 0)
            for t, ts in enumerate(slots):
                if ts < 0:
                    continue
                for h in range(self.H):
                    self.put(which, int(ts), h, c.codes[h, t], c.scales[h, t], c.zeros[h, t])
                    self.mass[self.slot(int(ts), h)] = 0.0

    def buffers(self):
        return [self.codes["k"], self.scales["k"], self.zeros["k"], self.codes["v"], self.scales["v"],
                self.zeros["v"]]


# ---------------------------------------------------------------- attention

def attention(pool, pages, lengths, q, q_start, scale, softcap=0.0, slopes=None, window=0, half=False):
    """(out, lse, mass to add by slot, tolerances of out, lse and mass without
    the output type's rounding) in FP64; q is FP64 [rows][Hq][D].

    Tolerances.  The products of a 4-bit difference (5 bits with its sign) and
    a BF16 query (8 bits) are exact; a group's 32 of them are added in FP32, a
    rounding (at most 2^-23 of the running sum of magnitudes, should the tensor
    core truncate) each, then G groups times their scales: with S = scale *
    sum |q k_hat| a score is off by (32 + 2G + 4) * 2^-23 * S at most.  The
    cap's tanh adds 2^-20 of the cap, the bias' rounding 2^-23 of itself, and
    the exponent in base 2 2^-22 of the largest score; all of them together
    are `ds`.  Weights then lie within a factor exp(2 ds) of the true ones
    (their own rounding: 2^-20).  Their sum, T positive FP32 terms in any order,
    is off by (T - 1) * 2^-24 of itself, and so are the weights, and lse by as
    much.  V's values and the weights enter the tensor core in two FP16
    pieces each: V's are exact, of a weight 2^-22 is lost, and so is the product
    of the two second pieces, 2^-22 too; 2^-16 covers these.  A weight under
    FP16's normal range (2^-14, where the largest one is 2^7 or more) is off by
    half of the last place there, 2^-25, which is 2^-32 of the largest weight and
    so of the sum; this counts where all larger weights meet a zero value.  The
    sum of T positions costs (T/16 + 64) roundings of 2^-23.

    `half` (BF16 output): one piece each, with two FP16 roundings: of the weight
    and of V's value, or of the weight and of its product with V's scale, which
    is then multiplied with the exact c - z.  Half a step each, 2^-11.  (A value
    under the normal range has a subnormal scale and is exact.)  A product under
    the normal range is off by 2^-25, where the largest weight is 2^7 or more,
    or 2^-8 or more with scales over 1.9 (a product over FP16's range would
    show): 2^-32 or 2^-17 of the sum, times |c - z| <= 15."""
    rows, Hq, D = q.shape
    grp = Hq // pool.H
    out = np.zeros((rows, Hq, D))
    lse = np.full((rows, Hq), -np.inf)
    add = np.zeros(pool.mass.shape)
    tol_o, tol_l, tol_m = np.zeros_like(out), np.zeros_like(lse), np.zeros_like(add)
    for b, n in enumerate(lengths):
        r0, r1 = int(q_start[b]), int(q_start[b + 1])
        m = r1 - r0
        if n == 0 or m == 0:
            continue
        ts = [int(pages[b][t // pool.P]) * pool.P + t % pool.P for t in range(n)]
        t = np.arange(n)
        for h in range(pool.H):
            k = np.stack([pool.value("k", s, h) for s in ts])
            v = np.stack([pool.value("v", s, h) for s in ts])
            at = np.array([pool.slot(s, h) for s in ts])
            for j in range(m):
                pos = n - m + j
                gap = pos - t
                seen = gap >= 0
                if window:
                    seen &= gap < window
                if not seen.any():
                    continue
                for i in range(h * grp, (h + 1) * grp):
                    x = q[r0 + j, i]
                    s = scale * (k @ x)
                    S = (abs(scale) * (np.abs(k) @ np.abs(x)))[seen].max()
                    ds = (32 + 2 * pool.G + 4) * 2.0 ** -23 * S
                    if softcap:
                        s = softcap * np.tanh(s / softcap)
                        ds += 2.0 ** -20 * softcap
                    if slopes is not None:
                        s = s - slopes[i] * gap
                        ds += 2.0 ** -22 * np.abs(slopes[i] * gap[seen]).max()
                    s = np.where(seen, s, -np.inf)
                    top = s.max()
                    ds += 2.0 ** -22 * np.abs(s[seen]).max()
                    e = np.exp(s - top)
                    p = e / e.sum()
                    out[r0 + j, i] = p @ v
                    lse[r0 + j, i] = top + np.log(e.sum())
                    add[at] += p
                    sums = seen.sum() * 2.0 ** -24
                    f = np.expm1(2 * ds) + 2.0 ** -20 + sums
                    tol_o[r0 + j, i] = (f + 2.0 ** -16 + (seen.sum() / 16 + 64) * 2.0 ** -23) * (p @ np.abs(v)) + 1e-30
                    tol_o[r0 + j, i] += 2.0 ** -32 * np.abs(v[seen]).sum(0)
                    if half:
                        tol_o[r0 + j, i] += (2.0 ** -10 + 2.0 ** -22) * (p @ np.abs(v))
                        steep = pool.scales["v"][at].view(np.float16).max() > 1.9
                        tol_o[r0 + j, i] += 15 * seen.sum() * 2.0 ** (-17 if steep else -32)
                    tol_l[r0 + j, i] = ds + sums + 2.0 ** -20 + 2.0 ** -22 * abs(lse[r0 + j, i])
                    tol_m[at] += (f + 2.0 ** -20) * p + 1e-37
    return out, lse, add, tol_o, tol_l, tol_m


# ---------------------------------------------------------------- eviction

def evict(mass, n, budget, recent):
    """Indexes that stay of one head's entries, in order."""
    keep = min(n, budget)
    rec = min(recent, keep)
    old = n - rec
    m = np.where(np.isnan(mass[:old]), -np.inf, mass[:old])
    best = sorted(range(old), key=lambda i: (-m[i], i))[:keep - rec]
    return sorted(best) + list(range(old, n))


# ---------------------------------------------------------------- token choice

def sample(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, log of its share, distance of u from the nearer border of the
    token's interval) of one row, FP64."""
    x = np.where(np.isnan(x), -np.inf, np.asarray(x, np.float64))
    top = x.max()
    if top == -np.inf:
        return -1, -np.inf, 1.0
    if not temperature > 0:
        return int(np.argmax(x)), 0.0, 1.0
    with np.errstate(invalid="ignore"):
        w = np.where(x == top, 1.0, np.exp((x - top) / float(temperature)))
    order = np.lexsort((np.arange(len(x)), -x))
    kept = order[:top_k] if top_k > 0 else order
    if top_p < 1:
        sums = np.cumsum(w[kept])
        ahead = sums - w[kept]
        inside = ahead < float(top_p) * sums[-1]
        inside[0] = True
        kept = kept[inside]
    kept = np.sort(kept[w[kept] >= min(float(min_p), 1.0)])
    kept = kept[w[kept] > 0]
    sums = np.cumsum(w[kept])
    share = np.concatenate([[0.0], sums / sums[-1]])
    i = min(int(np.searchsorted(sums, float(u) * sums[-1], side="right")), len(kept) - 1)
    return int(kept[i]), float(np.log(w[kept[i]] / sums[-1])), float(min(u - share[i], share[i + 1] - u))
