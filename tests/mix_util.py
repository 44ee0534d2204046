"""Inputs of attention in which every key's place shows, and the check that goes with them."""
import numpy as np
import torch

from oracle import mix_oracle as mix
from tests.gpu_util import bf16_bits_to_f64, say


def bf16_bits(x):
    """fp32 array -> (bits uint16, the values they stand for)."""
    bits = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    return bits, bf16_bits_to_f64(bits)


def needles(rng, n_q, n_kv, hd, page, kv_len, seqs, q_len, window=0):
    """`seqs` sequences of q_len queries on one table of kv_len keys (and some behind them).

    Each (query, head) row has a key that carries most of its weight: the last or the first one that it sees in two
    heads of the first sequence, else one of all those that it sees, spread so that no part of the keys can be
    lost unseen; and a key just outside of them (behind, or in front of a window) that would take most of its weight.
    Returns (cache, table [max_pages], queries' bits and values [seqs, q_len, n_q, hd])."""
    group, extra = n_q // n_kv, 40
    pages = -(-(kv_len + extra) // page)
    c = mix.Cache(pages + 2, n_kv, page, hd, rng)
    table = rng.permutation(pages + 2)[:pages].astype(np.int32)
    bits, q = bf16_bits(rng.standard_normal((seqs, q_len, n_q, hd)))
    k = 0.4 * rng.standard_normal((kv_len + extra, n_kv, hd))
    v = rng.standard_normal((kv_len + extra, n_kv, hd))
    rows = seqs * q_len * group
    for h in range(n_kv):
        for i in range(rows):
            # neighbouring rows of a head are of different sequences, so that all of them reach everywhere
            b, j, a = i % seqs, i // seqs % q_len, i // seqs // q_len
            x = q[b, j, h * group + a]
            p = kv_len - q_len + j
            lo = max(0, p - window + 1) if window else 0
            y = x * (np.log(p - lo + 1) + 3) / (hd ** -0.5 * (x * x).sum())
            at = lo + int((i + rng.uniform()) / rows * (p - lo + 1))
            k[p if b == 0 and a == 0 else lo if b == 0 and a == 1 else at, h] += y
            if i % 2 == 0:
                k[p + 1, h] += y
            elif lo > 0:
                k[lo - 1, h] += y
    t = np.arange(kv_len + extra)
    c.put_rows(table[t // page] * page + t % page, k.astype(np.float32), v.astype(np.float32))
    return c, table, bits, q


def attention_check(got, out, sigma, fixed, what, quiet=False):
    """got against attention_spread's values: each element within the fixed part and 8 sigma, and each row's error
    within twice the expected norm.  Raises AssertionError."""
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    err = np.abs(got - out)
    worst = float((err / (fixed + 8 * sigma + 1e-300)).max())
    rows = float((np.sqrt((err ** 2).sum(-1)) / np.sqrt((sigma ** 2 + fixed ** 2 / 3).sum(-1) + 1e-300)).max())
    assert worst <= 1, f"{what}: an element is off by {worst:.3g} of what it may be"
    assert rows <= 2, f"{what}: a row is off by {rows:.3g} of the expected norm"
    if not quiet:
        say(f"  {what}: worst element {worst:.3g}, worst row {rows:.3g} of 2")
