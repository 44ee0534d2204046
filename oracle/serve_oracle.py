"""Plain NumPy forms of a serving step's calls: the 8-bit paged cache, attention over it, the verification of
drafted tokens and low-rank adapters.  Test infrastructure only; shares no code with the HIP path.

The cache's quantizer is evaluated in fp32 operation by operation (it is defined that way, so codes and scales are
compared for equality); everything else in fp64."""
from __future__ import annotations

import numpy as np

BLOCK = 16
LIMIT = np.float32(57344.0)


class Cache:
    """The four arrays of a cache, as stored."""

    def __init__(self, n_pages, n_kv, page, hd, rng=None):
        self.n_pages, self.n_kv, self.page, self.hd = n_pages, n_kv, page, hd
        self.k_codes = np.zeros((n_pages, n_kv, page, hd), np.int8)
        self.v_codes = np.zeros((n_pages, n_kv, page // 8, hd, 8), np.int8)
        self.k_scale = np.zeros((n_pages, n_kv, page // BLOCK), np.float32)
        self.v_scale = np.zeros_like(self.k_scale)
        if rng is not None:  # what other users of the pool left: any codes, NaN scales
            self.k_codes[...] = rng.integers(-128, 128, self.k_codes.shape, dtype=np.int8)
            self.v_codes[...] = rng.integers(-128, 128, self.v_codes.shape, dtype=np.int8)
            self.k_scale[...] = np.nan
            self.v_scale[...] = np.nan

    def arrays(self):
        return self.k_codes, self.k_scale, self.v_codes, self.v_scale

    def _block(self, page, j):
        """(codes [n_kv, 16, hd] of keys, of values) of block j of a page, as views that can be read and written."""
        k = self.k_codes[page, :, BLOCK * j:BLOCK * (j + 1)]
        v = self.v_codes[page, :, 2 * j:2 * j + 2].transpose(0, 1, 3, 2)  # [n_kv, 2, 8, hd]
        return k.reshape(self.n_kv, 2, 8, self.hd), v

    def append(self, table, kv_len, k, v):
        """The new tokens k, v fp32 [n, n_kv, hd] of one sequence as its last keys; returns what is held for them
        (fp32, NaN for a token that stores nothing)."""
        n = len(k)
        held = [np.full(k.shape, np.nan, np.float32) for _ in range(2)]
        first = kv_len - n
        for kb in range(max(first, 0) // BLOCK, -(-kv_len // BLOCK)):
            lo, hi = max(first, BLOCK * kb, 0), min(kv_len, BLOCK * kb + BLOCK)
            if lo >= hi:
                continue
            page, j = int(table[lo // self.page]), BLOCK * kb % self.page // BLOCK
            if not 0 <= page < self.n_pages:
                continue
            begins = lo == BLOCK * kb
            for x, codes, scale, out in ((k, self._block(page, j)[0], self.k_scale, held[0]),
                                         (v, self._block(page, j)[1], self.v_scale, held[1])):
                new = np.clip(np.asarray(x[lo - first:hi - first], np.float32), -LIMIT, LIMIT)
                need = (np.abs(new).max((0, 2)) * np.float32(1.0 / 127.0)).astype(np.float32)  # [n_kv]
                old = scale[page, :, j].copy()
                with np.errstate(invalid="ignore"):
                    s = need if begins else np.where(need <= old, old, np.maximum(need, old * np.float32(1.25)))
                s = s.astype(np.float32)
                with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
                    inv = np.where(s > np.float32(2.0 ** -127), np.float32(1) / s, np.float32(0)).astype(np.float32)
                    ratio = (old / s).astype(np.float32)
                for h in range(self.n_kv):
                    if not begins and s[h] != old[h]:
                        for i in range(lo - BLOCK * kb):
                            c = codes[h, i // 8, i % 8]
                            codes[h, i // 8, i % 8] = np.rint(c.astype(np.float32) * ratio[h]).astype(np.int8)
                    c = np.clip(np.rint(new[:, h] * inv[h]), -127, 127).astype(np.float32)
                    for i in range(lo, hi):
                        codes[h, (i % BLOCK) // 8, i % 8] = c[i - lo].astype(np.int8)
                    out[lo - first:hi - first, h] = c * s[h]
                scale[page, :, j] = s
        return held

    def live(self, table, kv_len):
        """Codes and scales of a sequence's keys, whatever is stored behind them: for comparisons."""
        got = []
        for t in range(kv_len):
            p, o = int(table[t // self.page]), t % self.page
            if 0 <= p < self.n_pages:
                got.append((self.k_codes[p, :, o], self.v_codes[p, :, o // 8, :, o % 8],
                            self.k_scale[p, :, o // BLOCK], self.v_scale[p, :, o // BLOCK]))
        return [np.stack(x) for x in zip(*got)] if got else []

    def get(self, pages, places, head):
        """fp64 keys and values [n, hd] at some slots of a head, and the values' scales [n]."""
        ks = self.k_scale[pages, head, places // BLOCK].astype(np.float64)
        vs = self.v_scale[pages, head, places // BLOCK].astype(np.float64)
        k = self.k_codes[pages, head, places].astype(np.float64) * ks[:, None]
        v = self.v_codes[pages, head, places // 8, :, places % 8].astype(np.float64) * vs[:, None]
        return k, v, vs


def attention(q, cache, table, kv_len, q_len, scale, causal=True, window=0, sinks=0, gate=None, few=True):
    """One sequence: q fp64 [n, n_q, hd], table of page ids.  Returns (out fp64, tol fp64).

    The tolerance of the GPU's evaluation, per element: the output's rounding to bf16, 2^-8 |o|; the fp16
    rounding of p s, 2^-11 of W = sum p |v|, and where p s is below fp16's normal range its steps of 2^-24, half of one
    a key times codes up to 127: for few queries p s is held times 8 with the largest scale s at 2^11 or more, so
    that is 2^-25 / 2^14 = 2^-39 of the largest scale; for prompts with the row's largest p s at 2^11 or more, 2^-36 of
    that (few = None: the larger of the two); and the scores' error d (fp32 sums of hd + 8 terms, M = scale sum |q k|), which changes each
    p by at most a factor e^(2 d) once normalised: (e^(2 d) - 1) W.  The hardware's exp2 (2^-22) and the
    normalising sum (2^-20) sit in the 2^-18 added to the relative part.

    At the ends of the scales' range: few queries lift scales by at most 2^112, so that a step is 2^-140 at least;
    prompts take a scale below 2^-80 of the largest one that any of the rows sees (the key's block may be one of
    zeros) as 2^-80 of that, which moves an output by up to 127 times as much.  The last 2^-133 are a step of the
    smallest bf16 numbers."""
    n_q, hd = q.shape[1], q.shape[2]
    group = n_q // cache.n_kv
    out = np.zeros((q_len, n_q, hd))
    tol = np.full((q_len, n_q, hd), 2.0 ** -133)
    t = np.arange(kv_len)
    ids = np.asarray(table)[t // cache.page] if kv_len else np.zeros(0, int)
    there = (ids >= 0) & (ids < cache.n_pages)
    t, ids = t[there], ids[there]
    pos = kv_len - q_len + np.arange(q_len)[:, None]
    see = np.ones((q_len, len(t)), bool)
    if causal:
        see = t <= pos
        if window:
            see &= (t > pos - window) | (t < sinks)
    some = see.any(1)
    if not some.any():
        return out, tol
    for h in range(cache.n_kv):
        k, v, vs = cache.get(ids, t % cache.page, h)
        for a in range(h * group, (h + 1) * group):
            x = q[some, a]
            s = np.where(see[some], scale * (x @ k.T), -np.inf)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            o, w = p @ v, p @ np.abs(v)
            d = np.where(see[some], scale * (np.abs(x) @ np.abs(k).T), 0).max(1, keepdims=True) * (hd + 8) * 2.0 ** -24
            low = 2.0 ** -36 * (p * vs).max(1, keepdims=True)
            raised = 0 if few else 2.0 ** -80 * vs[see.any(0)].max()
            if few or few is None:
                low = np.maximum(0 if few else low, max(2.0 ** -39 * vs[see.any(0)].max(), 2.0 ** -140))
            e = w * (2.0 ** -11 + 2.0 ** -18 + np.expm1(2 * d)) + len(t) * 127 * low + 127 * raised
            if gate is not None:
                sig = 1 / (1 + np.exp(-gate[some, a]))
                o, e = o * sig, e * sig + np.abs(o * sig) * 2.0 ** -20
            out[some, a] = o
            tol[some, a] = e + (np.abs(o) + e) * 2.0 ** -8 + 2.0 ** -133
    return out, tol


def verify(draft, start, target, q, u, max_draft):
    """Drafts int [D], start int [B + 1], target [D + B, V] and q [D, V] or None (values of fp32 or bf16), u [D + B]:
    (tokens int [B, max_draft + 1], accepted int [B])."""
    B, V = len(start) - 1, target.shape[1]
    tokens = np.full((B, max_draft + 1), -1, np.int64)
    accepted = np.zeros(B, np.int64)
    target = np.asarray(target, np.float64)
    for b in range(B):
        s, n = int(start[b]), min(int(start[b + 1] - start[b]), max_draft)
        row, j = s + b, 0
        while j < n:
            d = int(draft[s + j])
            qd = 1.0 if q is None else float(q[s + j, d]) if 0 <= d < V else 0.0
            if not (0 <= d < V and float(u[row + j]) * qd < target[row + j, d]):
                break
            tokens[b, j] = d
            j += 1
        accepted[b] = j
        p = np.where(target[row + j] > 0, target[row + j], 0.0)
        w = p
        if j < n:
            other = np.zeros(V)
            if q is not None:
                other = np.asarray(q[s + j], np.float64)
            elif 0 <= draft[s + j] < V:
                other[int(draft[s + j])] = 1.0
            with np.errstate(invalid="ignore"):
                w = target[row + j] - other
            w = np.where(w > 0, w, 0.0)
            if not w.sum() > 0:
                w = p
        if w.sum() > 0:
            c = np.cumsum(w)
            hit = np.flatnonzero((c > float(u[row + n]) * c[-1]) & (w > 0))
            tokens[b, j] = hit[0] if len(hit) else np.flatnonzero(w > 0)[-1]
    return tokens, accepted


def lora(x, a, b, ids, base, scales, out_eps):
    """One part: x [T, K], a [adapters, r, K], b [adapters, N, r], base [T, N], all fp64.  Returns (y, tol).

    The tolerance: fp32 sums of K + 20 terms (the matrix cores', four waves' and up to 16 ranges') in h, carried
    through |b|; 3 r + 8 more in the second product, whose pieces hold 24 bits; the sum with base; the output's
    rounding out_eps |y|."""
    x, a, b, base = (np.asarray(t, np.float64) for t in (x, a, b, base))
    y = base.copy()
    tol = np.abs(base) * 2.0 ** -23
    u = 2.0 ** -24
    for t in range(len(x)):
        i = int(ids[t])
        if not 0 <= i < len(a):
            continue
        s = 1.0 if scales is None else float(scales[i])
        h, hm = a[i] @ x[t], np.abs(a[i]) @ np.abs(x[t])
        y[t] += s * (b[i] @ h)
        tol[t] += abs(s) * (np.abs(b[i]) @ (hm * (a.shape[2] + 20) * u + np.abs(h) * (3 * a.shape[1] + 8) * u))
    return y, tol + (np.abs(y) + tol) * out_eps
