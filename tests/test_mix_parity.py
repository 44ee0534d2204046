"""GPU parity of the token mixers (qmm_mix.h) against the plain NumPy forms in oracle/mix_oracle.py."""
import numpy as np
import pytest
import torch

import gemm_affine_u4_amd as qmm
from oracle import mix_oracle as mix
from tests.gpu_util import Guarded, assert_within, bf16_bits_to_f64, dev, say

pytestmark = pytest.mark.gpu


def bf16(x):
    """fp32 array -> (bits uint16, the values they stand for)."""
    bits = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    return bits, bf16_bits_to_f64(bits)


def gpu_cache(c):
    return qmm.KV4Cache(*[dev(a.copy()) for a in c.arrays()])


def host(t, dtype):
    return t.cpu().numpy().view(dtype)


def angles(rot, n=97, base=1e4):
    a = np.arange(n)[:, None] * base ** (-2.0 * np.arange(rot // 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


# ---- appending -----------------------------------------------------------------------------

@pytest.mark.parametrize("T,n_q,n_kv,hd,rot,page,f32", [
    (1, 5, 1, 128, 128, 16, False), (3, 40, 8, 128, 128, 32, False), (37, 6, 2, 256, 64, 16, True),
    (5, 14, 2, 64, 64, 64, False), (9, 3, 3, 64, 20, 16, True), (4, 4, 1, 128, 6, 128, False),
    (130, 2, 1, 256, 256, 32, False), (2, 7, 7, 128, 16, 4096, True), (700, 24, 4, 128, 128, 32, False)])
def test_append(T, n_q, n_kv, hd, rot, page, f32):
    rng = np.random.default_rng([T, n_q, n_kv, hd, rot])
    pages = -(-T // page) + 2
    c = mix.Cache(pages, n_kv, page, hd, rng)
    g = gpu_cache(c)
    k = rng.standard_normal((T, n_kv, hd)).astype(np.float32) * 3
    v = rng.standard_normal((T, n_kv, hd)).astype(np.float32)
    q = rng.standard_normal((T, n_q, hd)).astype(np.float32)
    v[0, 0, :64] = 0.25                      # a constant group
    k[T // 2, 0, hd - 1] = 1e5               # beyond the clamp (rotated or not)
    v[T - 1, n_kv - 1] *= 1e-6               # below fp16's normal scales
    if not f32:
        k, v, q = (bf16(x)[1].astype(np.float32) for x in (k, v, q))
    up = (lambda x: dev(x)) if f32 else (lambda x: dev(bf16(x)[0]).view(torch.bfloat16))
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    if T > 2:
        slots[1], slots[T - 1] = -1, pages * page  # padded rows
    pos = rng.integers(0, 97, T).astype(np.int32)
    if T > 3:
        pos[2], pos[3] = -5, 1000
    table = angles(rot)
    outs = [Guarded((T, h, hd), False) for h in (n_q, n_kv, n_kv)]
    qmm.qmm_kv4_append(g, up(k), up(v), dev(slots), positions=dev(pos), cos_sin=dev(table), q=up(q), q_out=outs[0].t,
                       k_held=outs[1].t, v_held=outs[2].t)
    torch.cuda.synchronize()
    rows = table[np.clip(pos, 0, 96)]
    kr, qr = mix.rotate_f32(k, rows), mix.rotate_f32(q, rows)
    for t in range(T):
        if 0 <= slots[t] < pages * page:
            for h in range(n_kv):
                c.put(slots[t], h, kr[t, h], v[t, h])
    for name, a, b, dt in zip(("k_codes", "k_meta", "v_codes", "v_meta"), c.arrays(), g.tensors,
                              (np.uint32, np.uint32, np.uint16, np.uint32)):
        assert np.array_equal(a, host(b, dt)), name
    for x, o in ((qr, outs[0]), (mix.dequantize(*mix.quantize_f32(kr)), outs[1]),
                 (mix.dequantize(*mix.quantize_f32(v)), outs[2])):
        assert np.array_equal(bf16(x)[0], o.values())


def test_append_without_rotation_or_outputs():
    rng = np.random.default_rng(5)
    c = mix.Cache(2, 2, 16, 128, rng)
    g = gpu_cache(c)
    k, v = (bf16(rng.standard_normal((3, 2, 128)))[1].astype(np.float32) for _ in range(2))
    slots = np.array([7, 31, 16], np.int32)
    qmm.qmm_kv4_append(g, dev(bf16(k)[0]).view(torch.bfloat16), dev(bf16(v)[0]).view(torch.bfloat16), dev(slots))
    torch.cuda.synchronize()
    for t in range(3):
        for h in range(2):
            c.put(slots[t], h, k[t, h], v[t, h])
    for a, b, dt in zip(c.arrays(), g.tensors, (np.uint32, np.uint32, np.uint16, np.uint32)):
        assert np.array_equal(a, host(b, dt))
    qmm.qmm_kv4_append(g, torch.empty(0, 2, 128, dtype=torch.bfloat16, device="cuda"),
                       torch.empty(0, 2, 128, dtype=torch.bfloat16, device="cuda"), dev(np.zeros(0, np.int32)))


# ---- attention -----------------------------------------------------------------------------

def filled(rng, q_lens, kv_lens, n_kv, hd, page, spare=2, scale_v=1.0):
    """A pool whose unused slots hold rubbish and NaN scales, and the sequences' page tables."""
    need = [-(-n // page) for n in kv_lens]
    width = max(max(need), 1) + 1
    pages = sum(need) + spare
    order = rng.permutation(pages)
    c = mix.Cache(pages, n_kv, page, hd, rng)
    table = np.full((len(kv_lens), width), -1, np.int32)
    used = 0
    for b, n in enumerate(kv_lens):
        table[b, :need[b]] = order[used:used + need[b]]
        used += need[b]
        # keys and values of the sequence's slots, packed at once through the same put()
        for t in range(n):
            slot = int(table[b, t // page]) * page + t % page
            for h in range(n_kv):
                c.put(slot, h, rng.standard_normal(hd).astype(np.float32) + 0.5,
                      scale_v * rng.standard_normal(hd).astype(np.float32))
    return c, table


def check_attention(rng, q_lens, kv_lens, n_q, n_kv, hd, page, window=0, causal=True, gated=False, pad=3, drop=None,
                    use_start=True, max_q=None, what="", q_scale=1.0, scale_v=1.0):
    c, table = filled(rng, q_lens, kv_lens, n_kv, hd, page, scale_v=scale_v)
    if drop is not None:
        table[drop] = c.n_pages + 5  # no such page
    starts = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    T = int(starts[-1]) + (pad if use_start else 0)
    qb, qv = bf16(q_scale * rng.standard_normal((T, n_q, hd)))
    gb, gv = bf16(2 * rng.standard_normal((T, n_q, hd)))
    out = Guarded((T, n_q, hd), False)
    out.t.fill_(0x1234)
    max_q = max(max(q_lens), 1) if max_q is None else max_q
    need = qmm.qmm_kv4_attn_workspace_bytes(T, len(kv_lens), max_q, n_q, n_kv, hd, table.shape[1] * page)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN everywhere
    g = gpu_cache(c)
    qmm.qmm_kv4_attn(dev(qb), g, dev(table), dev(np.array(kv_lens, np.int32)), out.t, ws,
                     q_start=dev(starts) if use_start else None, max_q=max_q, causal=causal, window=window,
                     gate=dev(gb) if gated else None)
    torch.cuda.synchronize()
    got_bits = out.values()
    got = bf16_bits_to_f64(got_bits)
    assert np.all(got_bits[starts[-1]:] == 0x1234), "rows behind the last sequence"
    for b, (n, kv) in enumerate(zip(q_lens, kv_lens)):
        m = min(n, max_q)
        assert np.all(got_bits[starts[b] + m:starts[b + 1]] == 0x1234), "rows past max_q"
        if n == 0:
            continue
        ref, tol = mix.attention(qv[starts[b]:starts[b + 1]], c, table[b], kv, n, hd ** -0.5, causal, window,
                                 gv[starts[b]:starts[b + 1]] if gated else None)
        assert_within(got[starts[b]:starts[b] + m], ref[:m], tol[:m], f"{what} sequence {b} q {n} kv {kv}")
    return out


@pytest.mark.parametrize("hd,n_q,n_kv", [(64, 14, 2), (128, 5, 1), (256, 6, 1), (128, 16, 1), (128, 40, 2), (64, 3, 3)])
@pytest.mark.parametrize("page", [16, 32, 128])
def test_attention_of_single_tokens(hd, n_q, n_kv, page):
    rng = np.random.default_rng([hd, n_q, page])
    check_attention(rng, [1] * 7, [1, 15, 16, 33, 0, 131, 290], n_q, n_kv, hd, page, use_start=False)


@pytest.mark.parametrize("hd,n_q,n_kv,page", [(128, 10, 2, 16), (256, 4, 1, 64), (64, 7, 1, 32)])
@pytest.mark.parametrize("gated", [False, True])
def test_attention_of_a_few_tokens_each(hd, n_q, n_kv, page, gated):
    rng = np.random.default_rng([hd, page, gated])
    check_attention(rng, [3, 0, 5, 1, 4], [3, 9, 70, 200, 2], n_q, n_kv, hd, page, gated=gated)


@pytest.mark.parametrize("hd,n_q,n_kv,page", [(128, 10, 2, 16), (256, 6, 1, 64), (64, 7, 1, 32), (128, 8, 8, 32)])
@pytest.mark.parametrize("window", [0, 1, 40])
def test_attention_of_prompts(hd, n_q, n_kv, page, window):
    rng = np.random.default_rng([hd, page, window])
    check_attention(rng, [67, 1, 129, 30], [67, 200, 140, 25], n_q, n_kv, hd, page, window=window, gated=window == 40)


def test_attention_without_a_mask():
    rng = np.random.default_rng(11)
    check_attention(rng, [1, 1], [75, 300], 4, 2, 128, 32, causal=False)
    check_attention(rng, [70, 3, 33], [75, 1, 40], 4, 1, 128, 32, causal=False)


def test_absent_pages_and_empty_rows():
    rng = np.random.default_rng(12)
    check_attention(rng, [1, 1, 1], [64, 64, 64], 4, 1, 128, 16, drop=(0, 1))
    check_attention(rng, [1, 1], [32, 64], 4, 1, 256, 32, drop=(0, 0))   # nothing left of sequence 0
    check_attention(rng, [80, 40], [90, 64], 6, 2, 128, 16, drop=(0, 2))
    check_attention(rng, [40, 70], [16, 10], 6, 2, 64, 32)               # more queries than keys
    check_attention(rng, [90, 1], [96, 1], 4, 1, 128, 32, drop=(0, 0), window=20)


def test_rows_past_max_q_are_left():
    rng = np.random.default_rng(13)
    check_attention(rng, [5, 2], [50, 60], 4, 2, 128, 32, max_q=3)
    check_attention(rng, [70, 20], [80, 60], 4, 1, 128, 32, max_q=41)


@pytest.mark.parametrize("q_scale,scale_v", [(30.0, 1.0), (1e-3, 1e-2), (1.0, 100.0)])
def test_attention_magnitudes(q_scale, scale_v):
    """Peaked and flat softmaxes, small and large values."""
    rng = np.random.default_rng(14)
    check_attention(rng, [1, 1], [150, 40], 5, 1, 128, 32, q_scale=q_scale, scale_v=scale_v)
    check_attention(rng, [66], [100], 5, 1, 128, 32, q_scale=q_scale, scale_v=scale_v)


def attn_setup(rng, q_lens, kv_lens, n_q, n_kv, hd, page):
    c, table = filled(rng, q_lens, kv_lens, n_kv, hd, page)
    starts = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    q = dev(bf16(rng.standard_normal((int(starts[-1]), n_q, hd)))[0])
    need = qmm.qmm_kv4_attn_workspace_bytes(q.shape[0], len(kv_lens), max(q_lens), n_q, n_kv, hd, table.shape[1] * page)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    args = (gpu_cache(c), dev(table), dev(np.array(kv_lens, np.int32)))
    return q, args, dev(starts), ws


@pytest.mark.parametrize("q_lens", [[1, 1, 1], [70, 5, 33]])
def test_attention_in_a_graph_and_on_another_stream(q_lens):
    rng = np.random.default_rng(15)
    q, (c, table, lens), starts, ws = attn_setup(rng, q_lens, [400, 90, 33], 10, 2, 128, 16)
    out = torch.zeros_like(q)

    def call(o, w):
        qmm.qmm_kv4_attn(q, c, table, lens, o, w, q_start=starts, max_q=max(q_lens))

    call(out, ws)
    torch.cuda.synchronize()
    want = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        call(out, ws)
    side.synchronize()
    assert torch.equal(out, want)
    # two graphs with a workspace each, replayed in turn with eager work between
    graphs, outs = [], []
    for _ in range(2):
        o, w = torch.zeros_like(q), torch.empty_like(ws)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            call(o, w)
        graphs.append((gr, o, w))
    for _ in range(3):
        for gr, o, w in graphs:
            o.zero_()
            w.fill_(255)
            gr.replay()
            call(out, ws)
            torch.cuda.synchronize()
            assert torch.equal(o, want) and torch.equal(out, want)
    # lengths are read on the device: a replay follows them
    lens.copy_(torch.tensor([300, 80, 33], dtype=torch.int32))
    for gr, o, w in graphs:
        gr.replay()
    call(out, ws)
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1], out) and torch.equal(graphs[1][1], out) and not torch.equal(out, want)


def test_a_long_context_is_split_and_joined_the_same_every_time():
    """One sequence of many keys on one head: value rows are copied from 64 distinct ones, so the
    plain form groups equal keys: softmax weights times their counts."""
    rng = np.random.default_rng(16)
    hd, page, n = 128, 64, 40000
    base = mix.Cache(1, 1, page, hd)
    for t in range(page):
        base.put(t, 0, rng.standard_normal(hd).astype(np.float32), rng.standard_normal(hd).astype(np.float32))
    pages = -(-n // page)
    g = qmm.KV4Cache(*[dev(np.ascontiguousarray(np.repeat(a, pages, 0))) for a in base.arrays()])
    qb, qv = bf16(rng.standard_normal((1, 5, hd)))
    table = dev(rng.permutation(pages).astype(np.int32)[None])
    ws = torch.empty(qmm.qmm_kv4_attn_workspace_bytes(1, 1, 1, 5, 1, hd, pages * page), dtype=torch.uint8, device="cuda")
    outs = []
    for _ in range(3):
        o = Guarded((1, 5, hd), False)
        qmm.qmm_kv4_attn(dev(qb), g, table, dev(np.array([n], np.int32)), o.t, ws)
        torch.cuda.synchronize()
        outs.append(o.values())
    assert np.array_equal(outs[0], outs[1]) and np.array_equal(outs[0], outs[2])
    (kc, ks, kb), (vc, vs, vb) = base.get(np.arange(page), 0)
    k, v = mix.dequantize(kc, ks, kb), mix.dequantize(vc, vs, vb)
    counts = np.bincount(np.arange(n) % page, minlength=page)
    # the whole period's tolerance is that of one period: weights of equal keys add up
    _, tol = mix.attention(qv, base, [0], page, 1, hd ** -0.5)
    for a in range(5):
        s = k @ qv[0, a] * hd ** -0.5
        w = counts * np.exp(s - s.max())
        ref = (w / w.sum()) @ v
        assert_within(bf16_bits_to_f64(outs[0])[0, a], ref, 1.01 * tol[0, a], f"head {a}")


def check_long(rng, q_lens, kv_lens, n_q, n_kv, hd, page, causal=True, window=0, check=()):
    """Long contexts whose tables name a few whole pages again and again."""
    c = mix.Cache(5, n_kv, page, hd)
    for slot in range(5 * page):
        for h in range(n_kv):
            c.put(slot, h, rng.standard_normal(hd).astype(np.float32), rng.standard_normal(hd).astype(np.float32))
    table = rng.integers(0, 5, (len(kv_lens), -(-max(kv_lens) // page))).astype(np.int32)
    starts = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    T, max_q = int(starts[-1]), max(q_lens)
    qb, qv = bf16(rng.standard_normal((T, n_q, hd)))
    out = Guarded((T, n_q, hd), False)
    need = qmm.qmm_kv4_attn_workspace_bytes(T, len(kv_lens), max_q, n_q, n_kv, hd, table.shape[1] * page)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    qmm.qmm_kv4_attn(dev(qb), gpu_cache(c), dev(table), dev(np.array(kv_lens, np.int32)), out.t, ws, q_start=dev(starts),
                     max_q=max_q, causal=causal, window=window)
    torch.cuda.synchronize()
    got = bf16_bits_to_f64(out.values())
    for b, (n, kv) in enumerate(zip(q_lens, kv_lens)):
        if kv == max(kv_lens) or b % 16 == 0 or b in check:
            sl = slice(starts[b], starts[b + 1])
            ref, tol = mix.attention(qv[sl], c, table[b], kv, n, hd ** -0.5, causal, window, None)
            assert_within(got[sl], ref, tol, f"sequence {b} q {n} kv {kv}")


@pytest.mark.parametrize("hd,page", [(128, 16), (64, 32), (256, 16)])
def test_long_contexts_of_single_tokens(hd, page):
    """More sequences than the GPU has room for, one of them with hundreds of steps for each wave."""
    rng = np.random.default_rng([41, hd])
    lens = rng.integers(0, 70, 300).tolist()
    lens[123] = 13003
    check_long(rng, [1] * 300, lens, 16, 8, hd, page)


@pytest.mark.parametrize("B", [2, 9, 63, 64, 65])
def test_long_contexts_in_any_order(B):
    """Ragged lengths, equal and empty ones among them, in batches that are put in order or not."""
    rng = np.random.default_rng([50, B])
    lens = rng.integers(1, 2600, B).tolist()
    lens[B // 2], lens[-1], lens[0] = 0, lens[0], 2700
    check_long(rng, [1] * B, lens, 4, 2, 128, 32, check=range(B))
    if B < 10:
        check_long(rng, [67 + b % 3 for b in range(B)], [n + 70 for n in lens], 4, 2, 128, 32, check=range(B))


@pytest.mark.parametrize("hd,page", [(128, 16), (64, 64), (256, 16)])
def test_long_contexts_of_prompts(hd, page):
    rng = np.random.default_rng([42, hd])
    check_long(rng, [70], [4900], 3, 1, hd, page)                    # split over the keys and joined
    check_long(rng, [90, 3], [3300, 2700], 2, 1, hd, page, window=1500)
    lens = rng.integers(33, 90, 34).tolist()
    lens[30] = 3471
    check_long(rng, [33] * 34, lens, 16, 8, hd, page)                # one block walks all of them
    check_long(rng, [66] * 34, [n + 33 for n in lens], 16, 8, hd, page)


@pytest.mark.parametrize("hd,rows", [(64, 128), (64, 129), (128, 128), (128, 129), (256, 64), (256, 65)])
def test_attention_where_the_kernels_meet(hd, rows):
    """The most rows per KV head that the few-query kernel takes, and one more."""
    rng = np.random.default_rng([44, hd, rows])
    check_attention(rng, [rows, 5], [rows + 140, 70], 1, 1, hd, 16, gated=True)
    check_attention(rng, [rows], [rows - 9], 2, 2, hd, 32, window=50)


def test_a_cache_past_32_bit_offsets():
    """The last pages of a pool whose code arrays are larger than 4 GiB each."""
    rng = np.random.default_rng(47)
    n_q, n_kv, hd, page, n = 16, 8, 256, 64, 100
    pages = (1 << 32) // (n_kv * page * hd // 2) + 3
    shapes = qmm.kv4_cache_shapes(pages, n_kv, page, hd)
    g = qmm.KV4Cache(*[torch.zeros(s, dtype=t, device="cuda")
                       for s, t in zip(shapes.values(), (torch.int32, torch.int32, torch.int16, torch.int32))])
    c = mix.Cache(2, n_kv, page, hd)
    q, k, v = (rng.standard_normal((n, h, hd)).astype(np.float32) for h in (n_q, n_kv, n_kv))
    small = np.array([[1, 0]], np.int32)
    table = np.array([[pages - 1, pages - 2]], np.int32)
    pos = np.arange(n)
    qmm.qmm_kv4_append(g, dev(k), dev(v), dev((table[0, pos // page] * page + pos % page).astype(np.int32)))
    for t in range(n):
        for h in range(n_kv):
            c.put(int(small[0, t // page]) * page + t % page, h, k[t, h], v[t, h])
    qb, qv = bf16(q)
    for first in (n - 1, 0):  # one token, then the whole prompt
        m = n - first
        out = Guarded((m, n_q, hd), False)
        ws = torch.empty(qmm.qmm_kv4_attn_workspace_bytes(m, 1, m, n_q, n_kv, hd, 2 * page), dtype=torch.uint8, device="cuda")
        qmm.qmm_kv4_attn(dev(qb[first:]), g, dev(table), dev(np.array([n], np.int32)), out.t, ws,
                         q_start=dev(np.array([0, m], np.int32)), max_q=m)
        torch.cuda.synchronize()
        ref, tol = mix.attention(qv[first:], c, small[0], n, m, hd ** -0.5)
        assert_within(bf16_bits_to_f64(out.values()), ref, tol, f"{m} queries")


def test_append_then_attend_step_by_step():
    """A sequence's prompt and three single tokens after it through append and attention."""
    rng = np.random.default_rng(17)
    n_q, n_kv, hd, page, n0 = 6, 2, 128, 16, 37
    c = mix.Cache(6, n_kv, page, hd, rng)
    g = gpu_cache(c)
    table = np.array([[4, 1, 3, 0]], np.int32)
    cs = angles(hd)
    done = 0
    for n in (n0, 1, 1, 1):
        q, k, v = (rng.standard_normal((n, h, hd)).astype(np.float32) for h in (n_q, n_kv, n_kv))
        pos = np.arange(done, done + n).astype(np.int32)
        slots = (table[0, pos // page] * page + pos % page).astype(np.int32)
        q_rot = torch.empty(n, n_q, hd, dtype=torch.bfloat16, device="cuda")
        qmm.qmm_kv4_append(g, dev(k), dev(v), dev(slots), positions=dev(pos), cos_sin=dev(cs), q=dev(q), q_out=q_rot)
        done += n
        out = Guarded((n, n_q, hd), False)
        ws = torch.empty(qmm.qmm_kv4_attn_workspace_bytes(n, 1, n, n_q, n_kv, hd, 4 * page), dtype=torch.uint8,
                         device="cuda")
        qmm.qmm_kv4_attn(q_rot, g, dev(table), dev(np.array([done], np.int32)), out.t, ws,
                         q_start=dev(np.array([0, n], np.int32)), max_q=n)
        torch.cuda.synchronize()
        kr = mix.rotate_f32(k, cs[pos])
        for t in range(n):
            for h in range(n_kv):
                c.put(slots[t], h, kr[t, h], v[t, h])
        qv = bf16(mix.rotate_f32(q, cs[pos]))[1]
        ref, tol = mix.attention(qv, c, table[0], done, n, hd ** -0.5)
        assert_within(bf16_bits_to_f64(out.values()), ref, tol, f"after {done} tokens")


# ---- the gated delta rule ------------------------------------------------------------------

def gdn_tol(n, dk, s0, v, s1, qnorm, scale):
    """Elementwise bounds of state and output.  With unit keys and beta <= 1 a step does not
    enlarge an earlier error (the update is a projection), so n steps of dot products and sums of
    at most dk + 16 roundings, each at most 2^-24 of M = |row of S|_2 + |v|, add up to
    (n + 1) (dk + 16) 2^-24 M; an output adds one more product with q."""
    m = max(np.sqrt((np.asarray(s0, np.float64) ** 2).sum(-1)).max(initial=0.0), np.sqrt((s1 ** 2).sum(-1)).max()) + np.abs(v).max(
        initial=0.0)
    u = (dk + 16) * 2.0 ** -24 * m
    return (n + 1) * u, (n + 2) * u * np.sqrt(dk) * qnorm * scale


def check_gdn(rng, lens, hk, hv, dk, dv, l2norm=True, f32=False, in_place=False, no_slot=None, pad=2, max_len=None,
              use_start=True, decay=0.2, what=""):
    B = len(lens)
    starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(starts[-1]) + (pad if use_start else 0)
    q, k = (rng.standard_normal((T, hk, dk)) + 0.4 for _ in range(2))
    if not l2norm:
        q, k = (x / np.sqrt((x * x).sum(-1, keepdims=True)) * 0.98 for x in (q, k))
    (qb, qv), (kb, kv), (vb, vv) = bf16(q), bf16(k), bf16(rng.standard_normal((T, hv, dv)))
    g = (-decay * rng.exponential(size=(T, hv))).astype(np.float32)
    beta = rng.uniform(0, 1, (T, hv)).astype(np.float32)
    n_slots = B + 2
    slots = rng.permutation(n_slots)[:B].astype(np.int32)
    if no_slot is not None:
        slots[no_slot] = n_slots
    s0 = rng.standard_normal((n_slots, hv, dv, dk)).astype(np.float32)
    s_in, y = dev(s0), Guarded((T, hv, dv), f32)
    s_out = Guarded((n_slots, hv, dv, dk), True)
    s_out.t.fill_(7.0)
    y.t.fill_(3)
    max_len = max(max(lens), 1) if max_len is None else max_len
    need = qmm.qmm_gdn_workspace_bytes(T, B, max_len, hk, hv, dk, dv)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    qmm.qmm_gdn(dev(qb), dev(kb), dev(vb), dev(g), dev(beta), s_in, y.t, ws, state_out=s_in if in_place else s_out.t,
                seq_start=dev(starts) if use_start else None, state_slots=dev(slots), max_len=max_len, l2norm=l2norm)
    torch.cuda.synchronize()
    got_y = y.values() if f32 else bf16_bits_to_f64(y.values())
    s_out.check_guards()
    got_s = (s_in if in_place else s_out.t).cpu().numpy()
    scale = dk ** -0.5
    stale = 3.0 if f32 else bf16_bits_to_f64(np.array([3], np.uint16))[0]
    assert np.all(got_y[starts[-1]:] == stale), "rows behind the last sequence"
    touched = np.zeros(n_slots, bool)
    for b in range(B):
        sl, n = slice(starts[b], starts[b] + min(lens[b], max_len)), min(lens[b], max_len)
        assert np.all(got_y[starts[b] + n:starts[b + 1]] == stale)
        kept = slots[b] < n_slots
        before = s0[slots[b]] if kept else np.zeros_like(s0[0])
        ry, rs = mix.gdn(qv[sl], kv[sl], vv[sl], g[sl], beta[sl], before, scale, l2norm)
        ts, ty = gdn_tol(n, dk, before, vv[sl], rs, 1.0, scale)
        if n:
            assert_within(got_y[sl], ry, ty + np.abs(ry) * (2.0 ** -24 if f32 else 2.0 ** -8), f"{what} y {b} len {n}")
        if kept:
            touched[slots[b]] = True
            assert_within(got_s[slots[b]], rs, ts, f"{what} state {b} len {n}")
            # roundings of either sign: their norm grows with the root of their number
            rel = np.linalg.norm(got_s[slots[b]] - rs) / max(np.linalg.norm(rs), 1e-30)
            assert rel <= np.sqrt((n + 1) * (dk + 16)) * 2.0 ** -24, rel
    left = s0 if in_place else np.full_like(s0, 7.0)
    assert np.array_equal(got_s[~touched], left[~touched]), "slots of no sequence"


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (128, 64), (64, 64)])
@pytest.mark.parametrize("hk,hv,B", [(2, 4, 5), (1, 1, 1), (16, 32, 40)])
def test_gdn_single_tokens(dk, dv, hk, hv, B):
    rng = np.random.default_rng([dk, dv, hv])
    check_gdn(rng, [1] * B, hk, hv, dk, dv, use_start=False)
    check_gdn(rng, [1] * B, hk, hv, dk, dv, in_place=True, f32=True)


def test_gdn_few_tokens_ragged():
    rng = np.random.default_rng(21)
    check_gdn(rng, [3, 0, 16, 1], 2, 6, 128, 128)
    check_gdn(rng, [0, 7, 2], 1, 2, 64, 128, in_place=True, no_slot=1)
    check_gdn(rng, [5, 2], 2, 2, 128, 64, l2norm=False, f32=True)
    check_gdn(rng, [9, 4], 2, 4, 128, 128, max_len=6)


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (128, 64), (64, 64)])
@pytest.mark.parametrize("lens", [[64], [65], [17, 200, 0, 63], [1, 129]])
def test_gdn_prompts(dk, dv, lens):
    rng = np.random.default_rng([dk, dv, len(lens), lens[0]])
    check_gdn(rng, lens, 2, 4, dk, dv, f32=True)
    check_gdn(rng, lens, 1, 3, dk, dv, in_place=True, no_slot=0 if len(lens) > 1 else None)


@pytest.mark.parametrize("dk,dv,f32", [(128, 128, False), (128, 128, True), (64, 128, False), (128, 64, True)])
def test_gdn_prompts_of_many_heads(dk, dv, f32):
    """More heads than the GPU takes at 16 columns a block."""
    rng = np.random.default_rng([dk, dv, 43])
    check_gdn(rng, [70, 0, 129, 33], 8, 24, dk, dv, f32=f32, no_slot=3)


def test_gdn_prompt_corners():
    rng = np.random.default_rng(23)
    check_gdn(rng, [150], 2, 2, 128, 128, l2norm=False, f32=True)
    check_gdn(rng, [100], 1, 2, 128, 128, decay=0.0, f32=True)      # nothing fades
    check_gdn(rng, [100], 1, 2, 128, 128, decay=30.0, f32=True)     # everything fades at once
    check_gdn(rng, [90, 120], 2, 4, 128, 128, max_len=70)
    # the same key over and over: each write replaces the last one
    T = 80
    kb, kv = bf16(np.broadcast_to(rng.standard_normal((1, 1, 128)), (T, 1, 128)))
    vb, vv = bf16(rng.standard_normal((T, 1, 128)))
    g, beta = np.zeros((T, 1), np.float32), np.ones((T, 1), np.float32)
    state, y = torch.zeros(1, 1, 128, 128, device="cuda"), torch.zeros(T, 1, 128, device="cuda")
    ws = torch.empty(qmm.qmm_gdn_workspace_bytes(T, 1, T, 1, 1, 128, 128), dtype=torch.uint8, device="cuda")
    qmm.qmm_gdn(dev(kb), dev(kb), dev(vb), dev(g), dev(beta), state, y, ws,
                seq_start=dev(np.array([0, T], np.int32)), max_len=T, l2norm=True)
    torch.cuda.synchronize()
    ry, rs = mix.gdn(kv, kv, vv, g, beta, np.zeros((1, 128, 128)), 128 ** -0.5, True)
    ts, ty = gdn_tol(T, 128, np.zeros((1, 128, 128)), vv, rs, 1.0, 128 ** -0.5)
    assert_within(state.cpu().numpy()[0], rs, ts, "state")
    assert_within(y.cpu().numpy(), ry, ty, "y")


@pytest.mark.parametrize("n", [12, 150])
@pytest.mark.parametrize("low", [-1e4, -1e9, float(np.finfo(np.float32).min), -np.inf])
def test_gdn_forgets_at_the_lowest_decays(n, low):
    """A log decay of any size below fp32's range ends what came before and nothing else."""
    rng = np.random.default_rng(46)
    hk, hv, d = 1, 2, 128
    (qb, qv), (kb, kv), (vb, vv) = (bf16(rng.standard_normal((n, h, d))) for h in (hk, hk, hv))
    g = (-0.1 * rng.exponential(size=(n, hv))).astype(np.float32)
    cut = n - 5
    g[cut], g[3] = low, low
    beta = rng.uniform(0, 1, (n, hv)).astype(np.float32)
    s0 = rng.standard_normal((1, hv, d, d)).astype(np.float32)
    state, y = dev(s0), torch.zeros(n, hv, d, device="cuda")
    ws = torch.empty(qmm.qmm_gdn_workspace_bytes(n, 1, n, hk, hv, d, d), dtype=torch.uint8, device="cuda")
    qmm.qmm_gdn(dev(qb), dev(kb), dev(vb), dev(g), dev(beta), state, y, ws, seq_start=dev(np.array([0, n], np.int32)),
                max_len=n, l2norm=True)
    torch.cuda.synchronize()
    ry, rs = mix.gdn(qv, kv, vv, np.maximum(g, -1e3), beta, s0[0], d ** -0.5, True)
    ts, ty = gdn_tol(n, d, s0[0], vv, rs, 1.0, d ** -0.5)
    assert_within(y.cpu().numpy(), ry, ty + np.abs(ry) * 2.0 ** -24, "y")
    assert_within(state[0].cpu().numpy(), rs, ts, "state")
    _, alone = mix.gdn(qv[cut:], kv[cut:], vv[cut:], np.maximum(g[cut:], -1e3), beta[cut:], np.zeros_like(s0[0]), d ** -0.5, True)
    assert_within(state[0].cpu().numpy(), alone, ts, "state of the last tokens alone")


@pytest.mark.parametrize("hk,hv", [(1, 2), (16, 48)])
def test_gdn_gives_the_same_bits_every_time(hk, hv):
    rng = np.random.default_rng([48, hv])
    lens, d = [500, 1, 333, 90], 128
    T, B = sum(lens), len(lens)
    q, k, v = (dev(bf16(rng.standard_normal((T, h, d)))[0]) for h in (hk, hk, hv))
    g = dev(-0.1 * rng.exponential(size=(T, hv)).astype(np.float32))
    beta = dev(rng.uniform(0, 1, (T, hv)).astype(np.float32))
    s_in = dev(rng.standard_normal((B, hv, d, d)).astype(np.float32))
    starts = dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
    ws = torch.empty(qmm.qmm_gdn_workspace_bytes(T, B, max(lens), hk, hv, d, d), dtype=torch.uint8, device="cuda")
    first = None
    for i in range(8):
        s_out, y = torch.empty_like(s_in), torch.empty(T, hv, d, device="cuda")
        ws.fill_(255 - i)
        qmm.qmm_gdn(q, k, v, g, beta, s_in, y, ws, state_out=s_out, seq_start=starts, max_len=max(lens), l2norm=True)
        torch.cuda.synchronize()
        if first is None:
            first = s_out, y
        assert torch.equal(s_out, first[0]) and torch.equal(y, first[1]), i


def test_attention_gives_the_same_bits_every_time():
    rng = np.random.default_rng(49)
    for q_lens, kv_lens, hd in (([1] * 9, [700, 3, 64, 65, 300, 31, 1, 128, 257], 128), ([200, 77], [260, 700], 128),
                                ([90, 130], [300, 131], 256)):
        q, (c, table, lens), starts, ws = attn_setup(rng, q_lens, kv_lens, 8, 2, hd, 16)
        first = None
        for i in range(6):
            out = torch.empty_like(q)
            ws.fill_(255 - i)
            qmm.qmm_kv4_attn(q, c, table, lens, out, ws, q_start=starts, max_q=max(q_lens))
            torch.cuda.synchronize()
            first = out if first is None else first
            assert torch.equal(out, first), (q_lens, i)


def test_gdn_prompt_then_tokens_through_one_state():
    """A sequence cut into calls of both kernels, its state in place, against one pass over all of it."""
    rng = np.random.default_rng(45)
    hk, hv, d, cuts = 2, 4, 128, [100, 1, 1, 7, 70, 1]
    T = sum(cuts)
    (qb, qv), (kb, kv), (vb, vv) = (bf16(rng.standard_normal((T, h, d))) for h in (hk, hk, hv))
    g = (-0.1 * rng.exponential(size=(T, hv))).astype(np.float32)
    beta = rng.uniform(0, 1, (T, hv)).astype(np.float32)
    s0 = rng.standard_normal((1, hv, d, d)).astype(np.float32)
    state, y = dev(s0), torch.zeros(T, hv, d, device="cuda")
    at = 0
    for n in cuts:
        sl = slice(at, at + n)
        ws = torch.empty(qmm.qmm_gdn_workspace_bytes(n, 1, n, hk, hv, d, d), dtype=torch.uint8, device="cuda")
        qmm.qmm_gdn(dev(qb[sl]), dev(kb[sl]), dev(vb[sl]), dev(g[sl]), dev(beta[sl]), state, y[sl], ws,
                    seq_start=dev(np.array([0, n], np.int32)), max_len=n, l2norm=True)
        at += n
    torch.cuda.synchronize()
    ry, rs = mix.gdn(qv, kv, vv, g, beta, s0[0], d ** -0.5, True)
    ts, ty = gdn_tol(T, d, s0[0], vv, rs, 1.0, d ** -0.5)
    assert_within(y.cpu().numpy(), ry, ty + np.abs(ry) * 2.0 ** -24, "y")
    assert_within(state[0].cpu().numpy(), rs, ts, "state")


@pytest.mark.parametrize("lens", [[1, 1, 1], [100, 30]])
def test_gdn_in_a_graph_and_on_another_stream(lens):
    rng = np.random.default_rng(24)
    T, B, hk, hv, d = sum(lens), len(lens), 2, 4, 128
    q, k, v = (dev(bf16(rng.standard_normal((T, h, d)))[0]) for h in (hk, hk, hv))
    g = dev(-0.1 * rng.exponential(size=(T, hv)).astype(np.float32))
    beta = dev(rng.uniform(0, 1, (T, hv)).astype(np.float32))
    starts = dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
    s_in = dev(rng.standard_normal((B, hv, d, d)).astype(np.float32))
    need = qmm.qmm_gdn_workspace_bytes(T, B, max(lens), hk, hv, d, d)

    def call(s_out, y, ws):
        qmm.qmm_gdn(q, k, v, g, beta, s_in, y, ws, state_out=s_out, seq_start=starts, max_len=max(lens), l2norm=True)

    def fresh():
        return torch.zeros_like(s_in), torch.zeros(T, hv, d, device="cuda"), torch.empty(need, dtype=torch.uint8, device="cuda")

    want = fresh()
    call(*want)
    torch.cuda.synchronize()
    other = fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(*other)
    side.synchronize()
    assert torch.equal(other[0], want[0]) and torch.equal(other[1], want[1])
    graphs = []
    for _ in range(2):
        bufs, gr = fresh(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            call(*bufs)
        graphs.append((gr, bufs))
    for _ in range(3):
        for gr, bufs in graphs:
            for t in bufs:
                t.zero_()
            gr.replay()
            call(*other)
            torch.cuda.synchronize()
            assert torch.equal(bufs[0], want[0]) and torch.equal(bufs[1], want[1]) and torch.equal(other[1], want[1])
