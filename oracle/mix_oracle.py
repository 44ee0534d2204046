"""Plain NumPy forms of the token mixers: the 4-bit paged cache, attention over it and the gated
delta rule.  Test infrastructure only; shares no code with the HIP path.

The quantizer is evaluated in fp32 operation by operation (it is defined that way, so codes are
compared for equality); everything else in fp64."""
from __future__ import annotations

import numpy as np

GROUP = 64
LIMIT = np.float32(57344.0)


def k_place(w: int, hd: int) -> int:
    """Place of code word w (dims 8w .. 8w+7) in a stored key row."""
    if hd == 64:
        return w
    return 16 * (w // 16) + 4 * ((w % 8) // 2) + 2 * ((w % 16) // 8) + w % 2


def rotate_f32(x, cos_sin_rows):
    """x fp32 [T, H, hd] rotated by table rows fp32 [T, rot]; each operation rounded."""
    x = np.asarray(x, np.float32)
    rot = cos_sin_rows.shape[1]
    h = rot // 2
    c, s = cos_sin_rows[:, None, :h], cos_sin_rows[:, None, h:]
    y = x.copy()
    y[..., :h] = x[..., :h] * c - x[..., h:rot] * s
    y[..., h:rot] = x[..., h:rot] * c + x[..., :h] * s
    return y


def quantize_f32(x):
    """(codes int [.., hd], scale fp16 [.., hd/64], bias fp16) of fp32 x, as qmm_mix.h defines them."""
    x = np.clip(np.asarray(x, np.float32), -LIMIT, LIMIT)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    lo, hi = g.min(-1), g.max(-1)
    s = ((hi - lo) * np.float32(1.0 / 15.0)).astype(np.float16)
    b = lo.astype(np.float16)
    sf, bf = s.astype(np.float32)[..., None], b.astype(np.float32)[..., None]
    with np.errstate(divide="ignore"):
        inv = np.where(sf > 0, np.float32(1) / sf, np.float32(0)).astype(np.float32)
    c = np.clip(np.rint((g - bf) * inv), 0, 15).astype(np.int64)
    return c.reshape(x.shape), s, b


def dequantize(codes, s, b):
    g = np.asarray(codes, np.float64).reshape(*codes.shape[:-1], codes.shape[-1] // GROUP, GROUP)
    return (g * s.astype(np.float64)[..., None] + b.astype(np.float64)[..., None]).reshape(codes.shape)


class Cache:
    """The four arrays of a cache, as stored."""

    def __init__(self, n_pages, n_kv, page, hd, rng=None):
        self.n_pages, self.n_kv, self.page, self.hd = n_pages, n_kv, page, hd
        shape = (n_pages, n_kv, page)
        self.k_codes = np.zeros(shape + (hd // 8,), np.uint32)
        self.k_meta = np.zeros(shape + (hd // 64,), np.uint32)
        self.v_codes = np.zeros((n_pages, n_kv, page // 8, hd // 4, 8), np.uint16)
        self.v_meta = np.zeros(shape + (hd // 64,), np.uint32)
        if rng is not None:  # what other users of the pool left: any codes, NaN scales
            self.k_codes[...] = rng.integers(0, 1 << 32, self.k_codes.shape, dtype=np.uint32)
            self.v_codes[...] = rng.integers(0, 1 << 16, self.v_codes.shape, dtype=np.uint16)
            self.k_meta[...] = 0x7E007E00
            self.v_meta[...] = 0x7E007E00

    def arrays(self):
        return self.k_codes, self.k_meta, self.v_codes, self.v_meta

    @staticmethod
    def _meta(s, b):
        return s.view(np.uint16).astype(np.uint32) | (b.view(np.uint16).astype(np.uint32) << 16)

    def put(self, slot, head, k, v):
        """One slot's key and value (fp32 [hd]) of a head."""
        p, o = divmod(int(slot), self.page)
        c, s, b = quantize_f32(k)
        for w in range(self.hd // 8):
            word = 0
            for i in range(8):
                word |= int(c[8 * w + i]) << (4 * i)
            self.k_codes[p, head, o, k_place(w, self.hd)] = word
        self.k_meta[p, head, o] = self._meta(s, b)
        c, s, b = quantize_f32(v)
        q = c.reshape(-1, 4)
        self.v_codes[p, head, o // 8, :, o % 8] = q[:, 0] | (q[:, 1] << 4) | (q[:, 2] << 8) | (q[:, 3] << 12)
        self.v_meta[p, head, o] = self._meta(s, b)

    def put_rows(self, slots, k, v):
        """put() of many slots and all heads: k, v fp32 [n, n_kv, hd]."""
        slots = np.asarray(slots)
        p, o = slots // self.page, slots % self.page
        at = [k_place(w, self.hd) for w in range(self.hd // 8)]
        for h in range(self.n_kv):
            c, s, b = quantize_f32(k[:, h])
            c = c.reshape(len(slots), -1, 8).astype(np.uint32)
            words = np.zeros(c.shape[:2], np.uint32)
            for i in range(8):
                words |= c[:, :, i] << np.uint32(4 * i)
            row = np.empty_like(words)
            row[:, at] = words
            self.k_codes[p, h, o], self.k_meta[p, h, o] = row, self._meta(s, b)
            c, s, b = quantize_f32(v[:, h])
            c = c.reshape(len(slots), -1, 4).astype(np.uint16)
            self.v_codes[p, h, o // 8, :, o % 8] = c[:, :, 0] | (c[:, :, 1] << 4) | (c[:, :, 2] << 8) | (c[:, :, 3] << 12)
            self.v_meta[p, h, o] = self._meta(s, b)

    def get(self, slots, head):
        """(codes, scale, bias) of keys and of values of some slots, codes [n, hd]."""
        slots = np.asarray(slots)
        p, o = slots // self.page, slots % self.page
        hd = self.hd
        order = [k_place(w, hd) for w in range(hd // 8)]
        words = self.k_codes[p, head, o][:, order]
        kc = np.stack([(words >> np.uint32(4 * i)) & 15 for i in range(8)], -1).reshape(len(slots), hd)
        units = self.v_codes[p, head, o // 8, :, o % 8]
        vc = np.stack([(units >> np.uint16(4 * i)) & 15 for i in range(4)], -1).reshape(len(slots), hd)

        def halves(meta):
            return ((meta & 0xFFFF).astype(np.uint16).view(np.float16), (meta >> 16).astype(np.uint16).view(np.float16))

        return (kc, *halves(self.k_meta[p, head, o])), (vc, *halves(self.v_meta[p, head, o]))


def attention(q, cache, table, kv_len, q_len, scale, causal=True, window=0, gate=None):
    """One sequence: q fp64 [n, n_q, hd], table of page ids.  Returns (out fp64, tol fp64).

    The tolerance of the GPU's evaluation, per element: the output's rounding to bf16, 2^-8 |o|;
    the fp16 rounding of p s (or of p and of the dequantized value), 2 * 2^-11 of W = sum p (|s c| + |b|);
    and the scores' error d (keys rounded to fp16, 2^-11 of scale sum |q| (|s c| + |b|), and fp32
    sums of at most hd + 8 terms), which changes each p by at most a factor e^(2 d) once
    normalised: (e^(2 d) - 1) W.  The hardware's exp2 (2^-22) and the normalising sum (2^-20) sit in
    the 2^-18 added to the relative part."""
    n_q, hd = q.shape[1], q.shape[2]
    group = n_q // cache.n_kv
    out = np.zeros((q_len, n_q, hd))
    tol = np.zeros((q_len, n_q, hd))
    t = np.arange(kv_len)
    ids = np.asarray(table)[t // cache.page] if kv_len else np.zeros(0, int)
    there = (ids >= 0) & (ids < cache.n_pages)
    slots = np.where(there, ids, 0).astype(np.int64) * cache.page + t % cache.page
    for h in range(cache.n_kv):
        (kc, ks, kb), (vc, vs, vb) = cache.get(slots[there], h)
        k, v = dequantize(kc, ks, kb), dequantize(vc, vs, vb)
        ka = dequantize(kc, ks, np.zeros_like(kb)) + np.repeat(np.abs(kb.astype(np.float64)), GROUP, -1)
        va = dequantize(vc, vs, np.zeros_like(vb)) + np.repeat(np.abs(vb.astype(np.float64)), GROUP, -1)
        for j in range(q_len):
            p0 = kv_len - q_len + j
            see = np.ones(int(there.sum()), bool)
            if causal:
                see = t[there] <= p0
                if window:
                    see &= t[there] > p0 - window
            if not see.any():
                continue
            for a in range(h * group, (h + 1) * group):
                x = q[j, a]
                sc = scale * (k[see] @ x)
                p = np.exp(sc - sc.max())
                p /= p.sum()
                o = p @ v[see]
                w = p @ va[see]
                d = float((scale * (ka[see] @ np.abs(x))).max()) * (2.0 ** -11 + (hd + 8) * 2.0 ** -24)
                e = w * (2 * 2.0 ** -11 + 2.0 ** -18 + np.expm1(2 * d))
                if gate is not None:
                    sig = 1 / (1 + np.exp(-gate[j, a]))
                    o, e = o * sig, e * sig + np.abs(o * sig) * 2.0 ** -20
                out[j, a] = o
                tol[j, a] = e + (np.abs(o) + e) * 2.0 ** -8 + 1e-30
    return out, tol


def attention_spread(q, cache, table, kv_len, q_len, scale, few, causal=True, window=0, gate=None, hide=None,
                     weight=None, bounds=True):
    """One sequence as attention() takes it: (out, sigma, fixed) in fp64.  hide(t) and weight(t) plant mistakes:
    keys that leave, and factors on the weights.

    sigma: root mean square of what independent roundings add, key by key; unlike the bound of
    attention() it shrinks as keys average out.  A rounding to fp16 is off by at most u = 2^-11 of the value,
    u / sqrt(3) in the mean square.  With weights p, o = sum p v:
      few queries:  dO = sum p e1 (s c) + sum p e2 (b - o)             (weight times scale; weight)
      prompts:      dO = sum p e1 (v - o) + sum p e2 v                 (weight; value)
                    + sum p ds (v - o), ds = scale sum_d q_d k_d e_td  (keys, for each key and dim)
                    + scale sum_d e_d q_d sum_t p k_td (v - o)         (scaled queries, for each dim)
    Weights among fp16's subnormals are off by 2^-25 of the largest weight, for few queries (times 8, scales
    lifted to 2^11) by 2^-28 and 2^-39 of the largest scale.  Scores in fp32, hd + 8 roundings of 2^-24 of
    M = scale sum |q| (|s c| + |b|), all of one sign: taken as the mean square of a key's ds.
    fixed: the output's rounding to bf16, 2^-8 |o|, and 2^-18 of W = sum p (|s c| + |b|) for fp32 sums, exp2, the value
    codes' cut (2^-14 of a weight times scale in eight) and the gate's sigmoid."""
    n_q, hd = q.shape[1], q.shape[2]
    group, u2 = n_q // cache.n_kv, 2.0 ** -22 / 3
    out, sigma, fixed = (np.zeros((q_len, n_q, hd)) for _ in range(3))
    t = np.arange(kv_len)
    ids = np.asarray(table)[t // cache.page] if kv_len else np.zeros(0, int)
    there = (ids >= 0) & (ids < cache.n_pages)
    t, slots = t[there], ids[there].astype(np.int64) * cache.page + t[there] % cache.page
    for h in range(cache.n_kv):
        (kc, ks, kb), (vc, vs, vb) = cache.get(slots, h)
        k, v = dequantize(kc, ks, kb), dequantize(vc, vs, vb)
        kbr, vbr = (np.repeat(b.astype(np.float64), GROUP, -1) for b in (kb, vb))
        vsr = np.repeat(vs.astype(np.float64), GROUP, -1)
        for j in range(q_len):
            p0 = kv_len - q_len + j
            see = np.ones(t.shape, bool)
            if causal:
                see = t <= p0
                if window:
                    see &= t > p0 - window
            if hide is not None:
                see &= ~hide(t)
            if not see.any():
                continue
            ki, vi, bi, ci, kbi = k[see], v[see], vbr[see], vc[see] * vsr[see], kbr[see]
            for a in range(h * group, (h + 1) * group):
                x = q[j, a]
                s = scale * (ki @ x)
                p = np.exp(s - s.max()) * (1.0 if weight is None else weight(t[see]))
                p /= p.sum()
                o = p @ vi
                if not bounds:
                    out[j, a] = o if gate is None else o / (1 + np.exp(-gate[j, a]))
                    continue
                w = p @ (ci + np.abs(bi))
                p2, away = p * p, (vi - o) ** 2
                m = scale * ((np.abs(ki - kbi) + np.abs(kbi)) @ np.abs(x)) * (hd + 8) * 2.0 ** -24
                if few:
                    var = u2 * (p2 @ (ci ** 2 + (bi - o) ** 2))
                    var += p.max() ** 2 * (2.0 ** -56 * ((bi - o) ** 2).sum(0) + (2.0 ** -39 * 15 * vsr[see].max()) ** 2 * len(s))
                    ds2 = m * m
                else:
                    var = u2 * (p2 @ (away + vi ** 2)) + p.max() ** 2 * 2.0 ** -50 * away.sum(0)
                    var += u2 * scale ** 2 * ((x[:, None] * ((p[:, None] * ki).T @ (vi - o))) ** 2).sum(0)
                    ds2 = u2 * scale ** 2 * ((ki * x) ** 2).sum(1) + m * m
                sd = np.sqrt(var + (p2 * ds2) @ away)
                f = 2.0 ** -18 * w
                if gate is not None:
                    sig = 1 / (1 + np.exp(-gate[j, a]))
                    o, sd, f = o * sig, sd * sig, f * sig
                out[j, a], sigma[j, a] = o, sd
                fixed[j, a] = f + 2.0 ** -8 * (np.abs(o) + 8 * sd) + 1e-30
    return out, sigma, fixed


def gdn(q, k, v, g, beta, state, scale, l2norm):
    """One sequence in fp64: q, k [n, Hk, Dk], v [n, Hv, Dv], state [Hv, Dv, Dk].  Returns (y, state)."""
    s = np.array(state, np.float64)
    n, hv = v.shape[0], v.shape[1]
    rep = hv // q.shape[1]
    q, k = np.asarray(q, np.float64), np.asarray(k, np.float64)
    if l2norm:
        q = q / np.sqrt((q * q).sum(-1, keepdims=True) + 1e-6)
        k = k / np.sqrt((k * k).sum(-1, keepdims=True) + 1e-6)
    q, k = np.repeat(q * scale, rep, 1), np.repeat(k, rep, 1)
    y = np.zeros(v.shape)
    for t in range(n):
        s *= np.exp(np.asarray(g[t], np.float64))[:, None, None]
        d = np.asarray(beta[t], np.float64)[:, None] * (v[t] - np.einsum("hvk,hk->hv", s, k[t]))
        s += d[:, :, None] * k[t][:, None, :]
        y[t] = np.einsum("hvk,hk->hv", s, q[t])
    return y, s
