"""GPU tests of the token mixers (qmm_mix.h) at the ends of their ranges: scores whose size leaves fp32
few bits below the point, rows that see nothing in split calls, and the like."""
import numpy as np
import pytest
import torch

import gemm_affine_u4_amd as qmm
from oracle import mix_oracle as mix
from tests.gpu_util import Guarded, assert_within, bf16_bits_to_f64, dev
from tests.test_mix_parity import bf16, gpu_cache

pytestmark = pytest.mark.gpu


def attend(c, table, q_bits, q_lens, kv_lens, scale=None):
    """qmm_kv4_attn over an oracle's cache, NaN in its workspace: (out in fp64, rows' starts)."""
    starts = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    T, n_q, hd = q_bits.shape
    out = Guarded((T, n_q, hd), False)
    need = qmm.qmm_kv4_attn_workspace_bytes(T, len(kv_lens), max(q_lens), n_q, c.n_kv, hd, table.shape[1] * c.page)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    qmm.qmm_kv4_attn(dev(q_bits), gpu_cache(c), dev(table), dev(np.array(kv_lens, np.int32)), out.t, ws,
                     q_start=dev(starts), max_q=max(q_lens), scale=scale)
    torch.cuda.synchronize()
    return bf16_bits_to_f64(out.values()), starts


@pytest.mark.parametrize("hd,group,page", [(128, 5, 32), (64, 3, 16), (256, 6, 64)])
@pytest.mark.parametrize("power", [0, 12, 60])
@pytest.mark.parametrize("kv_lens", [[200, 77], [4000]])
def test_weights_of_large_scores(hd, group, page, power, kv_lens):
    """Scores near 2^22 (and 2^34, 2^82) whose differences are exact: a key is (15, c, 0, ..) with scale 1 and
    bias 0, a query (2^18, 1, 0, ..) times 2^power, so a score is (15 2^18 + c) 2^power, 22 bits.  c is the same
    for 32 neighbouring keys, so that waves and splits have maxima of their own.

    The weights are then limited by fp16 alone: 2^-11 each of the weight times scale, of the weight with the
    bias and of the weight in the sum, so 2 2^-11 of W = sum p (|s c| + |b|), 2^-18 W for all that is
    fp32, and the output's rounding to bf16."""
    rng = np.random.default_rng([60, hd, power, len(kv_lens)])
    width = max(-(-n // page) for n in kv_lens)
    c = mix.Cache(len(kv_lens) * width, 1, page, hd, rng)
    table = rng.permutation(len(kv_lens) * width).astype(np.int32).reshape(len(kv_lens), width)
    steps = []
    for b, n in enumerate(kv_lens):
        t = np.arange(n)
        cs = rng.integers(0, 16, n // 32 + 1)[t // 32]
        k = np.zeros((n, 1, hd), np.float32)
        k[:, 0, 0], k[:, 0, 1] = 15, cs
        v = rng.standard_normal((n, 1, hd)) + rng.standard_normal((n // 32 + 1, 1, hd))[t // 32]
        c.put_rows(table[b, t // page] * page + t % page, k, v.astype(np.float32))
        steps.append(cs)
    q = np.zeros((2 * len(kv_lens), group, hd))
    q[:, :, 0], q[:, :, 1] = 2.0 ** 18 * 2.0 ** power, 2.0 ** power
    scale = np.float32(0.3)
    got, starts = attend(c, table, bf16(q)[0], [2] * len(kv_lens), kv_lens, float(scale))
    for b, n in enumerate(kv_lens):
        t = np.arange(n)
        _, (vc, vs, vb) = c.get(table[b, t // page] * page + t % page, 0)
        v = mix.dequantize(vc, vs, vb)
        va = mix.dequantize(vc, vs, np.zeros_like(vb)) + np.repeat(np.abs(vb.astype(np.float64)), 64, -1)
        for j in range(2):
            m = n - 1 + j
            s = float(scale) * (steps[b][:m] - steps[b][:m].max()) * 2.0 ** power
            p = np.exp(s) / np.exp(s).sum()
            o, w = p @ v[:m], p @ va[:m]
            e = w * (2 * 2.0 ** -11 + 2.0 ** -18)
            for a in range(group):
                assert_within(got[starts[b] + j, a], o, e + (np.abs(o) + e) * 2.0 ** -8, f"sequence {b} query {j} head {a}")


@pytest.mark.parametrize("hd,n_q,n_kv", [(128, 5, 1), (64, 6, 2), (256, 4, 1)])
def test_rows_of_large_queries_that_see_nothing(hd, n_q, n_kv):
    """Split calls whose rows see no key give zeros, whatever the queries' size."""
    rng = np.random.default_rng([61, hd])
    page, n = 32, 6000
    pages = -(-n // page)
    c = mix.Cache(4, n_kv, page, hd, rng)
    table = np.full((2, pages), -1, np.int32)
    table[1, ::2] = c.n_pages + 7
    q = bf16(2.0 ** 40 * rng.standard_normal((3, n_q, hd)))[0]
    got, _ = attend(c, table, q, [1, 2], [n, n - 40])
    assert np.all(got == 0), got


@pytest.mark.parametrize("size", [1.0, 2.0 ** 40])
def test_absent_pages_beside_present_ones_in_a_split_call(size):
    """One page is there among many splits that see nothing: its keys alone make the output."""
    rng = np.random.default_rng(62)
    page, n, hd, n_q = 32, 6000, 128, 5
    pages = -(-n // page)
    c = mix.Cache(4, 1, page, hd, rng)
    row = rng.standard_normal((1, 1, hd)).astype(np.float32)  # one value in all of its keys
    c.put_rows(2 * page + np.arange(page), rng.standard_normal((page, 1, hd)).astype(np.float32), np.repeat(row, page, 0))
    (_, (vc, vs, vb)) = c.get([2 * page], 0)
    v = mix.dequantize(vc, vs, vb)[0]
    va = np.abs(mix.dequantize(vc, vs, np.zeros_like(vb))[0]) + np.abs(np.repeat(vb[0].astype(np.float64), 64))
    e = va * (2 * 2.0 ** -11 + 2.0 ** -18)
    for at in (0, 77, pages - 2):
        table = np.full((1, pages), -1, np.int32)
        table[0, at] = 2
        got, _ = attend(c, table, bf16(size * rng.standard_normal((1, n_q, hd)))[0], [1], [n])
        for a in range(n_q):
            assert_within(got[0, a], v, e + (np.abs(v) + e) * 2.0 ** -8, f"page {at} head {a}")


@pytest.mark.parametrize("hd,page", [(128, 32), (64, 16), (256, 64)])
@pytest.mark.parametrize("size,gap", [(1.0, 8.0), (1e-2, 8.0), (1e-3, 8.0), (1e-4, 8.0), (1e-5, 6.0), (1e4, 8.0)])
def test_small_values_behind_dominant_keys(hd, page, size, gap):
    """Values of any size under weights of any size: a key's part is rounded relative to itself.

    256 sequences on one table, so that none is split and a wave walks a quarter of the keys; the first tile of
    each wave has a key that stands `gap` above all others.  Weights times 8 stay normal in fp16.
    Then, as above, the error is at most 2 2^-11 W, W = sum p (|s c| + |b|), 2^-18 W for fp32, and bf16's; scores
    differ by what their fp32 sums of hd + 8 terms round, d, which changes a weight by e^(2 d)."""
    rng = np.random.default_rng([63, hd, int(gap), int(np.log2(size)) + 100])
    n, B, n_kv = 8000, 256, 8
    pages = -(-n // page)
    c = mix.Cache(pages, n_kv, page, hd, rng)
    table = rng.permutation(pages).astype(np.int32)[None]
    t = np.arange(n)
    slots = table[0, t // page] * page + t % page
    bits, q = bf16(rng.standard_normal((1, n_kv, hd)))
    scale = hd ** -0.5
    k = 0.02 * rng.standard_normal((n, n_kv, hd))
    k[5:128:32] = q[0] * gap / (scale * (q[0] ** 2).sum(-1, keepdims=True))
    c.put_rows(slots, k.astype(np.float32), (size * rng.standard_normal((n, n_kv, hd))).astype(np.float32))
    got, _ = attend(c, np.repeat(table, B, 0), np.repeat(bits, B, 0), [1] * B, [n] * B)
    assert np.array_equal(got, np.broadcast_to(got[:1], got.shape))
    for h in range(n_kv):
        (kc, ks, kb), (vc, vs, vb) = c.get(slots, h)
        kd, v = mix.dequantize(kc, ks, kb), mix.dequantize(vc, vs, vb)
        ka = mix.dequantize(kc, ks, np.zeros_like(kb)) + np.repeat(np.abs(kb.astype(np.float64)), 64, -1)
        va = mix.dequantize(vc, vs, np.zeros_like(vb)) + np.repeat(np.abs(vb.astype(np.float64)), 64, -1)
        s = scale * (kd @ q[0, h])
        p = np.exp(s - s.max())
        assert 8 * p.min() > 2.0 ** -14
        p /= p.sum()
        o, w = p @ v, p @ va
        d = float((scale * (ka @ np.abs(q[0, h]))).max()) * (hd + 8) * 2.0 ** -24
        e = w * (2 * 2.0 ** -11 + 2.0 ** -18 + np.expm1(2 * d))
        assert_within(got[0, h], o, e + (np.abs(o) + e) * 2.0 ** -8, f"head {h}")


def test_a_prompt_of_many_blocks():
    """More queries than 65535 blocks of 16 rows hold; rows are checked here and there, as single tokens are."""
    rng = np.random.default_rng(65)
    n_q, n_kv, hd, page, n = 40, 8, 64, 64, 26300
    c = mix.Cache(5, n_kv, page, hd)
    c.put_rows(np.arange(5 * page), *(rng.standard_normal((5 * page, n_kv, hd)).astype(np.float32) for _ in range(2)))
    table = rng.integers(0, 5, (1, -(-n // page))).astype(np.int32)
    bits, q = bf16(rng.standard_normal((n, n_q, hd)))
    got, _ = attend(c, table, bits, [n], [n])
    for j in (0, 1, 24, 25, 26, 51, 13107, 26213, 26214, n - 1):
        ref, tol = mix.attention(q[j:j + 1], c, table[0], j + 1, 1, hd ** -0.5)
        assert_within(got[j:j + 1], ref, tol, f"query {j}")


@pytest.mark.parametrize("max_len", [1, 16, 100])
def test_gdn_of_no_tokens_copies_its_states(max_len):
    rng = np.random.default_rng(64)
    hk, hv, d, n_slots = 2, 4, 128, 4
    s_in = dev(rng.standard_normal((n_slots, hv, d, d)).astype(np.float32))
    s_out = torch.full_like(s_in, 7.0)
    empty = {h: torch.empty(0, h, d, dtype=torch.bfloat16, device="cuda") for h in (hk, hv)}
    flat = torch.empty(0, hv, device="cuda")
    ws = torch.empty(qmm.qmm_gdn_workspace_bytes(0, 3, max_len, hk, hv, d, d), dtype=torch.uint8, device="cuda")
    args = empty[hk], empty[hk], empty[hv], flat, flat, s_in, torch.empty_like(empty[hv]), ws
    start, slots = torch.zeros(4, dtype=torch.int32, device="cuda"), dev(np.array([2, n_slots, 0], np.int32))
    qmm.qmm_gdn(*args, state_out=s_out, seq_start=start, state_slots=slots, max_len=max_len)
    qmm.qmm_gdn(*args, seq_start=start, state_slots=slots, max_len=max_len)  # in place: nothing to do
    torch.cuda.synchronize()
    assert torch.equal(s_out[2], s_in[2]) and torch.equal(s_out[0], s_in[0])
    assert torch.all(s_out[1] == 7) and torch.all(s_out[3] == 7)
