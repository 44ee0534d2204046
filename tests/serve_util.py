"""Inputs and device forms that the tests of a serving step's calls share."""
import numpy as np
import torch

import gemm_affine_u4_amd as qmm
from oracle import serve_oracle as srv
from tests.gpu_util import bf16_bits_to_f64, dev


def bf16(x):
    """fp32 array -> (bits uint16, the values they stand for)."""
    bits = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    return bits, bf16_bits_to_f64(bits)


def gpu_cache(c):
    return qmm.KV8Cache(*[dev(a.copy()) for a in c.arrays()])


def ints(*a):
    return dev(np.array(a, np.int32))


def angles(rot, n=97, base=1e4):
    a = np.arange(n)[:, None] * base ** (-2.0 * np.arange(rot // 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def tables(rng, kv_lens, page, spare=2):
    """(page table, pages of the pool): the sequences' pages in any order, one entry more than the longest needs."""
    need = [-(-n // page) for n in kv_lens]
    width, pages = max(max(need), 1) + 1, sum(need) + spare
    order = rng.permutation(pages)
    table, used = np.full((len(kv_lens), width), -1, np.int32), 0
    for b, m in enumerate(need):
        table[b, :m] = order[used:used + m]
        used += m
    return table, pages


def filled(rng, kv_lens, n_kv, hd, page, spare=2, scale_k=1.0, scale_v=1.0):
    """A pool whose unused slots hold rubbish and NaN scales, and the sequences' page tables."""
    table, pages = tables(rng, kv_lens, page, spare)
    c = srv.Cache(pages, n_kv, page, hd, rng)
    for b, n in enumerate(kv_lens):
        k = (scale_k * (rng.standard_normal((n, n_kv, hd)) + 0.5)).astype(np.float32)
        v = (scale_v * rng.standard_normal((n, n_kv, hd))).astype(np.float32)
        if n:
            c.append(table[b], n, k, v)
    return c, table


def few_rows(rows):
    """The form that attention of so many rows per KV head takes: of few queries, prompts', or (None) either."""
    return True if rows <= 16 else None if rows <= 256 else False


def whole_adapters(rng, T, K, rank, rows, n_ad):
    """Adapters whose h = A x are whole numbers of 24 bits times a power of two, and whose B passes one of them on to each
    output: every product and sum is exact in fp32, so that y shows all bits that h is carried with.
    Returns x, a, b (of fp32, exact in bf16), ids and y in fp64."""
    ids = rng.integers(0, n_ad, T).astype(np.int32)
    at = np.sort(rng.choice(K, 3, replace=False))  # the three inputs that count
    x = np.zeros((T, K), np.float32)
    x[:, at] = rng.choice([-1.0, 1.0], (T, 1)) * 2.0 ** rng.integers(-20, 20, (T, 1)) * np.array([65536.0, 256.0, 1.0])
    a = np.zeros((n_ad, rank, K), np.float32)
    a[:, :, at[0]] = rng.integers(128, 256, (n_ad, rank))
    a[:, :, at[1:]] = rng.integers(0, 256, (n_ad, rank, 2))
    b = np.zeros((n_ad, rows, rank), np.float32)
    b[:, np.arange(rows), np.arange(rows) % rank] = 2.0 ** rng.integers(-6, 6, (n_ad, rows))
    h = np.einsum("tk,trk->tr", x[:, at].astype(np.float64), a[ids][:, :, at])
    return x, a, b, ids, np.einsum("tr,tnr->tn", h, b[ids])
