"""GPU: attention over the paged 8-bit cache where scales are at the ends of their range, and what is stored for keys that
no query sees.  Calls of more than 256 rows per KV head are those of prompts."""
import numpy as np
import pytest
import torch

import gemm_affine_u4_amd as qmm
from oracle import serve_oracle as srv
from tests.gpu_util import Guarded, assert_within, bf16_bits_to_f64, dev
from tests.serve_util import bf16, filled, gpu_cache, ints, tables
from tests.test_serve_cache import check_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("bad", [np.nan, np.inf, 1e30])
def test_prompts_do_not_depend_on_scales_that_no_row_sees(hd, bad):
    """Beside a long prompt, sequences whose few rows leave most of a block's columns without a row: blocks behind their
    windows have any scale, and the outputs keep their bits."""
    rng = np.random.default_rng([60, hd])
    n_q, n_kv, page = 8, 2, 16
    q_lens = [70] + rng.integers(1, 10, 40).tolist()
    kv = [300] + rng.integers(140, 400, 40).tolist()
    starts = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    qb, _ = bf16(rng.standard_normal((int(starts[-1]), n_q, hd)))
    for window, sinks in ((60, 0), (47, 5), (70, 30)):
        c, table = filled(rng, kv, n_kv, hd, page)
        scales = [s.copy() for s in (c.k_scale, c.v_scale)]
        for b, (n, m) in enumerate(zip(q_lens, kv)):
            hidden = range(-(-sinks // 16), (m - n - window + 1) // 16)
            for t in hidden if b % 2 else hidden[-1:]:  # all of them, or the one beside the window
                c.k_scale[table[b, t]] = c.v_scale[table[b, t]] = bad
        got = []
        for _ in range(2):
            out = torch.empty(int(starts[-1]), n_q, hd, dtype=torch.bfloat16, device="cuda")
            need = qmm.qmm_kv8_attn_workspace_bytes(out.shape[0], len(kv), max(q_lens), n_q, n_kv, hd,
                                                    table.shape[1] * page, window, sinks)
            qmm.qmm_kv8_attn(dev(qb), gpu_cache(c), dev(table), ints(*kv), out,
                             torch.empty(need, dtype=torch.uint8, device="cuda"), q_start=dev(starts), max_q=max(q_lens),
                             window=window, sinks=sinks)
            torch.cuda.synchronize()
            got.append(out.view(torch.int16).cpu().numpy())
            assert np.all(np.isfinite(out.float().cpu().numpy()))
            c.k_scale, c.v_scale = scales  # as they were appended
        assert np.array_equal(*got), f"window {window}: {np.count_nonzero(got[0] != got[1])} outputs differ"


# values of these magnitudes have scales from 2^-86 down to 2^-126.5, below the smallest normal number
@pytest.mark.parametrize("scale_v", [1e-24, 1e-28, 1e-31, 1e-34, 1.2e-36, 3.5e-37])
@pytest.mark.parametrize("hd,n_q,n_kv", [(128, 5, 1), (64, 10, 2), (256, 5, 1)])
def test_values_of_the_smallest_magnitudes(hd, n_q, n_kv, scale_v):
    """Single tokens, prompts whose keys are one split's, and prompts in splits."""
    rng = np.random.default_rng([61, hd, int(1e40 * scale_v) % 9973])
    for q_lens, lens in (([1, 1], [150, 40]), ([66], [100]), ([66, 4], [1700, 2300]), ([1], [3000])):
        check_attention(rng, q_lens, lens, n_q, n_kv, hd, 32, scale_v=scale_v, gated=hd == 64)


def mixed(rng, lens, n_kv, hd, page, factor):
    """Caches whose block i of 16 keys holds values factor(i) times as large."""
    table, pages = tables(rng, lens, page)
    c = srv.Cache(pages, n_kv, page, hd, rng)
    for b, n in enumerate(lens):
        f = np.array([factor(i) for i in range(-(-n // 16))])[np.arange(n) // 16, None, None]
        c.append(table[b], n, rng.standard_normal((n, n_kv, hd)).astype(np.float32),
                 (f * rng.standard_normal((n, n_kv, hd))).astype(np.float32))
    return c, table


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("name", ["fall", "rise", "one", "last", "turns", "zeros"])
def test_prompts_over_blocks_of_very_different_scales(hd, name):
    """Values of 1e-36 to 1e4 and of zeros in one sequence, in orders that move a row's maximum late, early and often."""
    rng = np.random.default_rng([62, hd])
    steps = 10.0 ** np.linspace(4, -36, 24)
    factor = {"fall": lambda i: steps[min(i // 3, 23)], "rise": lambda i: steps[23 - min(i // 3, 23)],
              "one": lambda i: 1e4 if i == 40 else 1e-36, "last": lambda i: 1.0 if i >= 69 else 3e-37,
              "turns": lambda i: (1.0, 1e-36, 0.0, 1e-20)[i // 5 % 4], "zeros": lambda i: 1e-33 if i == 70 else 0.0}[name]
    for lens, q_lens in (([1150], [66]), ([1150, 60], [70, 33])):
        c, table = mixed(rng, lens, 2, hd, 16, factor)
        for window, sinks in ((0, 0), (700, 40)):
            check_attention(rng, q_lens, lens, 8, 2, hd, 16, c=c, table=table.copy(), window=window, sinks=sinks,
                            what=name)


@pytest.mark.parametrize("name", ["rise", "last", "turns"])
def test_prompts_over_such_blocks_in_one_split(name):
    """The same where sequences are many, so that a block walks all of a sequence's keys."""
    rng = np.random.default_rng([63])
    factor = {"rise": lambda i: 10.0 ** (-36 + i / 4), "last": lambda i: 1.0 if i >= 150 else 3e-37,
              "turns": lambda i: (1.0, 1e-36, 0.0, 1e-20)[i // 70 % 4]}[name]
    lens = [2500] + [40] * 20
    c, table = mixed(rng, lens, 4, 128, 32, factor)
    check_attention(rng, [66] + [33] * 20, lens, 16, 4, 128, 32, c=c, table=table, check={0, 3})


@pytest.mark.parametrize("q_lens,lens", [([66], [1500]), ([70, 9], [300, 400])])
@pytest.mark.parametrize("low,high", [(1.0, 1e24), (1e20, 1e28), (1e-30, 1e28)])
def test_prompts_over_values_far_above_what_append_stores(q_lens, lens, low, high):
    """Scales that a caller's own cache may hold; they grow on the way."""
    rng = np.random.default_rng([64])
    c, table = mixed(rng, lens, 1, 128, 16, lambda i: 1.0)
    for b, n in enumerate(lens):
        for i in range(-(-n // 16)):
            c.v_scale[table[b, i]] *= np.float32(low if i < n // 32 else high)
    check_attention(rng, q_lens, lens, 4, 1, 128, 16, c=c, table=table)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("tail,others", [(0, 0), (1, 64), (40, 64)])
def test_prompts_behind_a_long_run_of_zero_values(hd, tail, others):
    """600000 keys whose values are zeros, then ordinary ones: their weights count as much as any.  Beside many other
    sequences a block walks all of these keys."""
    rng = np.random.default_rng([65, hd, tail])
    page, q_len, group, n_zero = 4096, 52, 5, 146 * 4096
    c = srv.Cache(2, 1, page, hd)
    k = rng.standard_normal((2 * page, 1, hd)).astype(np.float32)
    v = rng.standard_normal((2 * page, 1, hd)).astype(np.float32)
    v[:page] = 0
    c.append([0, 1], 2 * page, k, v)
    n = n_zero + q_len + tail
    table = np.array([[0] * 146 + [1]] * (1 + others), np.int32)
    T = q_len + others
    qb, qv = bf16(0.1 * rng.standard_normal((T, group, hd)))  # weights of about the same size
    out = Guarded((T, group, hd), False)
    need = qmm.qmm_kv8_attn_workspace_bytes(T, 1 + others, q_len, group, 1, hd, 147 * page)
    qmm.qmm_kv8_attn(dev(qb), gpu_cache(c), dev(table), ints(n, *[1] * others), out.t,
                     torch.empty(need, dtype=torch.uint8, device="cuda"),
                     q_start=ints(0, *range(q_len, T + 1)), max_q=q_len)
    torch.cuda.synchronize()
    got = bf16_bits_to_f64(out.values())
    kz, _, _ = c.get(np.zeros(page, int), np.arange(page), 0)
    ko, vo, _ = c.get(np.ones(q_len + tail, int), np.arange(q_len + tail), 0)
    for j in range(q_len):
        m = tail + j + 1
        for a in range(group):
            x = qv[j, a] * hd ** -0.5
            p, w = 146 * np.exp(kz @ x).sum(), np.exp(ko[:m] @ x)
            o, mag = w @ vo[:m] / (p + w.sum()), w @ np.abs(vo[:m]) / (p + w.sum())
            # the weights' fp16 and the output's bf16; sums of 600000 weights, all positive, in fp32 in an order that adds
            # 8 at a time: 600000 / 8 roundings of 2^-24 of the sum at most
            assert np.all(np.abs(got[j, a] - o) <= mag * (2.0 ** -11 + 75000 * 2.0 ** -24) + np.abs(o) * 2.0 ** -8 + 1e-12), (j, a)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("q_len", [1, 3, 70])
def test_a_single_visible_key_whatever_its_score(hd, q_len):
    """A row that sees one key has its value, whether the score is far below or above 0."""
    rng = np.random.default_rng([66, hd, q_len])
    n = 90
    table, pages = tables(rng, [n], 16)
    c = srv.Cache(pages, 1, 16, hd, rng)
    k = rng.uniform(1e3, 2e3, (n, 1, hd)).astype(np.float32)
    v = rng.standard_normal((n, 1, hd)).astype(np.float32)
    c.append(table[0], n, k, v)
    t = np.arange(n - q_len, n)
    want = c.get(table[0, t // 16], t % 16, 0)[1]
    for size, loud in ((1e24, 1), (1e29, 1), (-1e24, 1), (-1e29, 1), (1e-3, 1e30), (-1e-3, 1e30)):
        qb, _ = bf16(size * rng.uniform(0.5, 1, (q_len, 4, hd)))
        out = Guarded((q_len, 4, hd), False)
        need = qmm.qmm_kv8_attn_workspace_bytes(q_len, 1, q_len, 4, 1, hd, table.shape[1] * 16, 1)
        g = gpu_cache(c)
        g.tensors[1].mul_(loud)  # key scales that a caller's own cache may hold
        qmm.qmm_kv8_attn(dev(qb), g, dev(table), ints(n), out.t, torch.empty(need, dtype=torch.uint8, device="cuda"),
                         q_start=ints(0, q_len), max_q=q_len, window=1)
        torch.cuda.synchronize()
        # one weight of fp16 (2^-11), the sum's exponential (2^-18) and the output's rounding
        assert_within(bf16_bits_to_f64(out.values()), np.broadcast_to(want[:, None], (q_len, 4, hd)),
                      np.abs(want[:, None]) * (2.0 ** -8 + 2.0 ** -10) + 1e-30, f"{q_len} queries of {size}")


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("q_len", [1, 3, 70])
@pytest.mark.parametrize("size", [1e8, 1e9, 1e12, 1e20, 1e28])
def test_rows_whose_largest_score_stands_alone(hd, q_len, size):
    """Keys are multiples of one direction, so that scores are far apart and the nearest one is the answer, above and
    below 0, whatever comes before it."""
    rng = np.random.default_rng([67, hd, q_len])
    n = 700
    table, pages = tables(rng, [n], 32)
    c = srv.Cache(pages, 1, 32, hd, rng)
    steps = rng.permutation(np.arange(1, 126))[np.arange(n) % 125].astype(np.float32)  # whole codes, all different in 125
    k = np.tile(steps[:, None, None], (1, 1, hd))
    c.append(table[0], n, k, rng.standard_normal((n, 1, hd)).astype(np.float32))
    c.k_codes[:] = 0
    for i in range(n):
        c.k_codes[table[0, i // 32], 0, i % 32] = steps[i]
    c.k_scale[:] = 1.0
    first = n - q_len
    for sign in (1.0, -1.0):
        qb, _ = bf16(np.full((q_len, 4, hd), sign * size))
        out = Guarded((q_len, 4, hd), False)
        need = qmm.qmm_kv8_attn_workspace_bytes(q_len, 1, q_len, 4, 1, hd, table.shape[1] * 32, 125)
        qmm.qmm_kv8_attn(dev(qb), gpu_cache(c), dev(table), ints(n), out.t,
                         torch.empty(need, dtype=torch.uint8, device="cuda"), q_start=ints(0, q_len), max_q=q_len, window=125)
        torch.cuda.synchronize()
        t = np.arange(n)
        best = []
        for j in range(q_len):
            see = np.flatnonzero((t <= first + j) & (t > first + j - 125))
            best.append(see[np.argmax(sign * steps[see])])
        best = np.array(best)
        want = c.get(table[0, best // 32], best % 32, 0)[1]
        assert_within(bf16_bits_to_f64(out.values()), np.broadcast_to(want[:, None], (q_len, 4, hd)),
                      np.abs(want[:, None]) * (2.0 ** -8 + 2.0 ** -10) + 1e-30, f"{q_len} queries of {sign * size}")
