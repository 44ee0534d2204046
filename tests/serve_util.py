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
