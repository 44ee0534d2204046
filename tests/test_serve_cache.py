"""GPU parity of the paged 8-bit cache and of attention over it (qmm_serve.h) with oracle/serve_oracle.py."""
import numpy as np
import pytest
import torch

import gemm_affine_u4_amd as qmm
from oracle import mix_oracle as mix
from oracle import serve_oracle as srv
from tests.gpu_util import Guarded, assert_within, bf16_bits_to_f64, dev, say
from tests.serve_util import angles, bf16, few_rows, filled, gpu_cache, ints, tables

pytestmark = pytest.mark.gpu


def same_cache(c, g, table, kv_lens):
    """The live keys of every sequence, codes and scales, bit for bit."""
    back = srv.Cache(c.n_pages, c.n_kv, c.page, c.hd)
    back.k_codes, back.k_scale, back.v_codes, back.v_scale = (t.cpu().numpy() for t in g.tensors)
    for b, n in enumerate(kv_lens):
        for name, x, y in zip(("k", "v", "k_scale", "v_scale"), c.live(table[b], n), back.live(table[b], n)):
            assert np.array_equal(x, y), (b, name)
    return back


def up(x, f32):
    return dev(x) if f32 else dev(bf16(x)[0]).view(torch.bfloat16)


# ---- appending -----------------------------------------------------------------------------

@pytest.mark.parametrize("new,old,n_q,n_kv,hd,rot,page,f32", [
    ([1], [0], 5, 1, 128, 128, 16, False), ([1, 1, 1], [15, 16, 17], 40, 8, 128, 128, 32, False),
    ([37, 1, 0, 20], [0, 5, 9, 43], 6, 2, 256, 64, 16, True), ([5, 16], [30, 16], 14, 2, 64, 64, 64, False),
    ([9, 3], [8, 1], 3, 3, 64, 20, 16, True), ([4, 40], [1, 0], 4, 1, 128, 6, 128, False),
    ([130, 2, 15, 17], [7, 14, 1, 15], 2, 1, 256, 256, 32, False), ([2], [4000], 7, 7, 128, 16, 4096, True),
    ([700], [33], 24, 4, 128, 128, 32, False), ([1] * 70, list(range(70)), 2, 2, 64, 32, 32, False)])
def test_append(new, old, n_q, n_kv, hd, rot, page, f32):
    rng = np.random.default_rng([len(new), new[0], n_q, n_kv, hd, rot])
    lens = [n + m for n, m in zip(new, old)]
    table, pages = tables(rng, lens, page)
    c = srv.Cache(pages, n_kv, page, hd, rng)
    for b, m in enumerate(old):
        if m:
            c.append(table[b], m, rng.standard_normal((m, n_kv, hd)).astype(np.float32),
                     0.3 * rng.standard_normal((m, n_kv, hd)).astype(np.float32))
    g = gpu_cache(c)
    T, pad = sum(new), 2
    k, v, q = (rng.standard_normal((T + pad, h, hd)).astype(np.float32) for h in (n_kv, n_kv, n_q))
    k *= rng.choice([0.2, 1.0, 3.0], (T + pad, 1, 1)).astype(np.float32)  # scales that stay, and that grow
    v[0, 0] = 0.0
    k[T // 2, 0, hd - 1] = 1e5                # beyond the clamp
    v[T - 1, n_kv - 1] *= 1e-30
    if not f32:
        k, v, q = (bf16(x)[1].astype(np.float32) for x in (k, v, q))
    pos = rng.integers(0, 97, T + pad).astype(np.int32)
    if T > 3:
        pos[2], pos[3] = -5, 1000
    cs = angles(rot)
    outs = [Guarded((T + pad, h, hd), False) for h in (n_q, n_kv, n_kv)]
    for o in outs:
        o.t.fill_(0x1234)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    qmm.qmm_kv8_append(g, up(k, f32), up(v, f32), dev(table), dev(np.array(lens, np.int32)), q_start=dev(starts),
                       max_q=max(new), positions=dev(pos), cos_sin=dev(cs), q=up(q, f32), q_out=outs[0].t,
                       k_held=outs[1].t, v_held=outs[2].t)
    torch.cuda.synchronize()
    rows = cs[np.clip(pos, 0, 96)]
    kr, qr = mix.rotate_f32(k, rows), mix.rotate_f32(q, rows)
    got = [o.values() for o in outs]
    assert np.array_equal(got[0][:T], bf16(qr)[0][:T])
    for b, n in enumerate(new):
        if n:
            sl = slice(starts[b], starts[b + 1])
            held = c.append(table[b], lens[b], kr[sl], v[sl])
            for x, o in zip(held, got[1:]):
                assert np.array_equal(bf16(x)[0], o[sl])
    for o in got:
        assert np.all(o[T:] == 0x1234), "rows behind the last sequence"
    same_cache(c, g, table, lens)


def test_append_nothing_stored_and_nothing_optional():
    """Absent pages, more tokens than keys, tokens past max_q, lengths past the table; no rotation, no outputs."""
    rng = np.random.default_rng(5)
    n_kv, hd, page = 2, 128, 16
    new, lens, max_q = [20, 5, 30, 3, 18], [40, 3, 35, 0, 200], 25
    table, pages = tables(rng, [40, 3, 35, 0, 48], page)
    table[0, 2] = pages + 4                        # keys 32 .. 39: no page
    width = table.shape[1] * page                  # sequence 4: its length is clamped to this
    table[4, -1] = -7
    c = srv.Cache(pages, n_kv, page, hd, rng)
    c.append(table[0], 20, *(rng.standard_normal((20, n_kv, hd)).astype(np.float32) for _ in range(2)))
    c.append(table[2], 5, *(rng.standard_normal((5, n_kv, hd)).astype(np.float32) for _ in range(2)))
    c.append(table[4], width - 18, *(rng.standard_normal((width - 18, n_kv, hd)).astype(np.float32) for _ in range(2)))
    before = [a.copy() for a in c.arrays()]
    g = gpu_cache(c)
    T = sum(new)
    k, v = (bf16(rng.standard_normal((T, n_kv, hd)))[1].astype(np.float32) for _ in range(2))
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    held = Guarded((T, n_kv, hd), False)
    held.t.fill_(0x1234)
    qmm.qmm_kv8_append(g, up(k, False), up(v, False), dev(table), dev(np.array(lens, np.int32)), q_start=dev(starts),
                       max_q=max_q, v_held=held.t)
    torch.cuda.synchronize()
    got = held.values()
    ends = [40, 3, 30, 0, width]                   # sequence 2: 25 of its 30 tokens
    for b in range(5):
        n = min(new[b], max_q)
        kv = min(lens[b], width) - (new[b] - n)
        want = c.append(table[b], kv, k[starts[b]:starts[b] + n], v[starts[b]:starts[b] + n])[1]
        want = np.concatenate([want, np.full((new[b] - n, n_kv, hd), np.nan, np.float32)])
        bits = np.where(np.isnan(want), 0x1234, bf16(want)[0])
        assert np.array_equal(got[starts[b]:starts[b + 1]], bits), b
    back = same_cache(c, g, table, ends)
    used = {int(p) for b in range(5) for p in table[b, :-(-ends[b] // page)] if 0 <= p < pages}
    for x, y in zip(before, back.arrays()):        # pages that nothing was stored in
        for p in set(range(pages)) - used:
            assert np.array_equal(x[p], y[p], equal_nan=x.dtype == np.float32)
    none = torch.empty(0, n_kv, hd, dtype=torch.bfloat16, device="cuda")
    qmm.qmm_kv8_append(g, none, none, dev(table[:1]), ints(0), q_start=ints(0, 0))


def test_append_positions_default_to_places():
    rng = np.random.default_rng(6)
    c = srv.Cache(3, 1, 16, 64)
    g, h = gpu_cache(c), gpu_cache(c)
    k, v = (dev(rng.standard_normal((40, 1, 64)).astype(np.float32)) for _ in range(2))
    cs, table = dev(angles(64)), ints(2, 0, 1).view(1, 3)
    qmm.qmm_kv8_append(g, k, v, table, ints(40), q_start=ints(0, 40), max_q=40, cos_sin=cs)
    qmm.qmm_kv8_append(h, k, v, table, ints(40), q_start=ints(0, 40), max_q=40, cos_sin=cs,
                       positions=dev(np.arange(40, dtype=np.int32)))
    torch.cuda.synchronize()
    for x, y in zip(g.tensors, h.tensors):
        assert torch.equal(x, y)


def test_append_of_the_smallest_values():
    """Blocks whose scale has no finite reciprocal hold zeros; just above that, and beside larger ones, they do not."""
    rng = np.random.default_rng(8)
    n, n_kv, hd, page = 33, 5, 128, 16
    k, v = (rng.standard_normal((n, n_kv, hd)).astype(np.float32) for _ in range(2))
    for h, s in enumerate((1e-40, 1e-37, 1e-35, 1.0, 0.0)):
        k[:, h] *= np.float32(s)
        v[:, h] *= np.float32(s)
    table, pages = tables(rng, [n], page)
    c = srv.Cache(pages, n_kv, page, hd, rng)
    g = gpu_cache(c)
    qmm.qmm_kv8_append(g, dev(k), dev(v), dev(table), ints(n), q_start=ints(0, n), max_q=n)
    torch.cuda.synchronize()
    c.append(table[0], n, k, v)
    same_cache(c, g, table, [n])


def test_append_with_a_max_q_far_above_the_tokens():
    rng = np.random.default_rng(9)
    n_kv, hd, page, B = 8, 64, 16, 60
    table, pages = tables(rng, [3] * B, page)
    c = srv.Cache(pages, n_kv, page, hd, rng)
    g = gpu_cache(c)
    k, v = (rng.standard_normal((3 * B, n_kv, hd)).astype(np.float32) for _ in range(2))
    qmm.qmm_kv8_append(g, dev(k), dev(v), dev(table), dev(np.full(B, 3, np.int32)),
                       q_start=dev(np.arange(B + 1, dtype=np.int32) * 3), max_q=1 << 22)
    torch.cuda.synchronize()
    for b in range(B):
        c.append(table[b], 3, k[3 * b:3 * b + 3], v[3 * b:3 * b + 3])
    same_cache(c, g, table, [3] * B)


def test_append_token_by_token_then_take_back():
    """Blocks that fill token by token, drafts taken back by a shorter length and written over."""
    rng = np.random.default_rng(7)
    n_kv, hd, page = 2, 128, 32
    table, pages = tables(rng, [100, 100], page)
    c = srv.Cache(pages, n_kv, page, hd, rng)
    g = gpu_cache(c)
    lens = np.array([0, 0])
    for step, new in enumerate([(3, 1)] + [(1, 2)] * 9 + [(6, 1)] * 5):
        if step % 3 == 2:
            lens = np.maximum(lens - [2, 0], 0)   # two drafts of sequence 0 were not kept
        T = sum(new)
        k, v = (bf16(rng.standard_normal((T, n_kv, hd)) * (1 + 0.2 * step))[1].astype(np.float32) for _ in range(2))
        lens = lens + new
        starts = np.array([0, new[0], T], np.int32)
        qmm.qmm_kv8_append(g, up(k, False), up(v, False), dev(table), dev(lens.astype(np.int32)), q_start=dev(starts),
                           max_q=max(new))
        torch.cuda.synchronize()
        for b in range(2):
            c.append(table[b], int(lens[b]), k[starts[b]:starts[b + 1]], v[starts[b]:starts[b + 1]])
        same_cache(c, g, table, lens.tolist())


# ---- attention -----------------------------------------------------------------------------

def check_attention(rng, q_lens, kv_lens, n_q, n_kv, hd, page, window=0, sinks=0, causal=True, gated=False, pad=3,
                    drop=None, use_start=True, max_q=None, what="", q_scale=1.0, scale_k=1.0, scale_v=1.0, c=None,
                    table=None, check=None):
    if c is None:
        c, table = filled(rng, kv_lens, n_kv, hd, page, scale_k=scale_k, scale_v=scale_v)
    if drop is not None:
        table[drop] = c.n_pages + 5  # no such page
    starts = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    T = int(starts[-1]) + (pad if use_start else 0)
    qb, qv = bf16(q_scale * rng.standard_normal((T, n_q, hd)))
    gb, gv = bf16(2 * rng.standard_normal((T, n_q, hd)))
    out = Guarded((T, n_q, hd), False)
    out.t.fill_(0x1234)
    max_q = max(max(q_lens), 1) if max_q is None else max_q
    need = qmm.qmm_kv8_attn_workspace_bytes(T, len(kv_lens), max_q, n_q, n_kv, hd, table.shape[1] * page, window, sinks)
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN everywhere
    qmm.qmm_kv8_attn(dev(qb), gpu_cache(c), dev(table), dev(np.array(kv_lens, np.int32)), out.t, ws[:need],
                     q_start=dev(starts) if use_start else None, max_q=max_q, causal=causal, window=window, sinks=sinks,
                     gate=dev(gb) if gated else None)
    torch.cuda.synchronize()
    assert bool((ws[need:] == 0xFF).all()), "write behind the workspace"
    got_bits = out.values()
    got = bf16_bits_to_f64(got_bits)
    assert np.all(got_bits[starts[-1]:] == 0x1234), "rows behind the last sequence"
    for b, (n, kv) in enumerate(zip(q_lens, kv_lens)):
        m = min(n, max_q)
        assert np.all(got_bits[starts[b] + m:starts[b + 1]] == 0x1234), "rows past max_q"
        if n == 0 or (check is not None and b not in check):
            continue
        ref, tol = srv.attention(qv[starts[b]:starts[b + 1]], c, table[b], kv, n, hd ** -0.5, causal, window, sinks,
                                 gv[starts[b]:starts[b + 1]] if gated else None,
                                 few=few_rows(max_q * n_q // n_kv))
        assert_within(got[starts[b]:starts[b] + m], ref[:m], tol[:m], f"{what} sequence {b} q {n} kv {kv}")
    return got_bits


@pytest.mark.parametrize("hd,n_q,n_kv", [(64, 14, 2), (128, 5, 1), (256, 6, 1), (128, 16, 1), (128, 40, 2), (64, 3, 3),
                                         (256, 40, 2)])
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


@pytest.mark.parametrize("hd,n_q,n_kv,page", [(128, 10, 2, 16), (256, 6, 1, 32), (64, 7, 1, 128)])
@pytest.mark.parametrize("window,sinks", [(1, 1), (33, 4), (64, 64), (100, 17), (20, 1000), (500, 3), (31, 33), (1 << 62, 1 << 62)])
def test_attention_with_sinks(hd, n_q, n_kv, page, window, sinks):
    """Windows and first keys that meet, overlap, end inside tiles and pages, or cover everything."""
    rng = np.random.default_rng([hd, window % 1009, sinks % 1009])
    check_attention(rng, [1, 1, 1, 1], [5, 64, 171, 700], n_q, n_kv, hd, page, window=window, sinks=sinks)
    check_attention(rng, [4, 6, 2], [9, 230, 641], n_q, n_kv, hd, page, window=window, sinks=sinks, gated=True)
    check_attention(rng, [80, 33, 150], [80, 600, 420], n_q, n_kv, hd, page, window=window, sinks=sinks)


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
    check_attention(rng, [90, 1], [400, 333], 4, 1, 128, 16, drop=(0, 0), window=20, sinks=18)
    check_attention(rng, [3, 1], [400, 333], 4, 1, 128, 16, drop=(1, 0), window=20, sinks=5)


def test_rows_past_max_q_are_left():
    rng = np.random.default_rng(13)
    check_attention(rng, [5, 2], [50, 60], 4, 2, 128, 32, max_q=3)
    check_attention(rng, [70, 20], [80, 60], 4, 1, 128, 32, max_q=41)


@pytest.mark.parametrize("q_scale,scale_k,scale_v", [(30.0, 1.0, 1.0), (1e-3, 1.0, 1e-2), (1.0, 1.0, 100.0),
                                                     (1e-12, 1e4, 1e-20), (1e6, 1e-5, 1e4)])
def test_attention_magnitudes(q_scale, scale_k, scale_v):
    """Peaked and flat softmaxes, small and large keys and values."""
    rng = np.random.default_rng(14)
    for q_lens, lens in (([1, 1], [150, 40]), ([66], [100])):
        check_attention(rng, q_lens, lens, 5, 1, 128, 32, q_scale=q_scale, scale_k=scale_k, scale_v=scale_v)


def test_blocks_of_very_different_scales():
    """Blocks whose values or keys are 2^40 apart, and blocks of zeros, in every order."""
    rng = np.random.default_rng(18)
    for order in (1, -1):
        table, pages = tables(rng, [128, 90], 16)
        c = srv.Cache(pages, 2, 16, 128, rng)
        for b, n in enumerate((128, 90)):
            f = 2.0 ** (-5.0 * (np.arange(n) // 16))[::order, None, None]
            f[32:48] = 0
            c.append(table[b], n, rng.standard_normal((n, 2, 128)).astype(np.float32),
                     (f * rng.standard_normal((n, 2, 128))).astype(np.float32))
        for q in ([1, 1], [70, 40]):
            check_attention(rng, q, [128, 90], 6, 2, 128, 16, c=c, table=table.copy())


def attn_setup(rng, q_lens, kv_lens, n_q, n_kv, hd, page, window, sinks):
    c, table = filled(rng, kv_lens, n_kv, hd, page)
    starts = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    q = dev(bf16(rng.standard_normal((int(starts[-1]), n_q, hd)))[0])
    need = qmm.qmm_kv8_attn_workspace_bytes(q.shape[0], len(kv_lens), max(q_lens), n_q, n_kv, hd, table.shape[1] * page,
                                            window, sinks)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    return q, (gpu_cache(c), dev(table), dev(np.array(kv_lens, np.int32))), dev(starts), ws


@pytest.mark.parametrize("q_lens,window,sinks", [([1, 1, 1], 0, 0), ([2, 1, 3], 200, 5), ([70, 5, 33], 0, 0)])
def test_attention_in_a_graph_and_on_another_stream(q_lens, window, sinks):
    rng = np.random.default_rng(15)
    q, (c, table, lens), starts, ws = attn_setup(rng, q_lens, [1400, 90, 33], 10, 2, 128, 16, window, sinks)
    out = torch.zeros_like(q)

    def call(o, w):
        qmm.qmm_kv8_attn(q, c, table, lens, o, w, q_start=starts, max_q=max(q_lens), window=window, sinks=sinks)

    call(out, ws)
    torch.cuda.synchronize()
    want = out.clone()
    out.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(out, ws)
    side.synchronize()
    assert torch.equal(out, want)
    graphs = []
    for _ in range(2):  # two graphs with a workspace each, replayed in turn with eager work between
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
    lens.copy_(torch.tensor([1300, 80, 33], dtype=torch.int32))  # lengths are read on the device: a replay follows them
    for gr, o, w in graphs:
        gr.replay()
    call(out, ws)
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1], out) and torch.equal(graphs[1][1], out) and not torch.equal(out, want)


def repeated(rng, n_kv, hd, page, kv_lens):
    """A few whole pages, and tables that name them again and again."""
    c = srv.Cache(5, n_kv, page, hd)
    x = rng.standard_normal((2, 5 * page, n_kv, hd)).astype(np.float32)
    c.append(np.arange(5), 5 * page, x[0], x[1])
    return c, rng.integers(0, 5, (len(kv_lens), -(-max(kv_lens) // page))).astype(np.int32)


def check_long(rng, q_lens, kv_lens, n_q, n_kv, hd, page, check=(), **kw):
    c, table = repeated(rng, n_kv, hd, page, kv_lens)
    check = {b for b, kv in enumerate(kv_lens) if kv == max(kv_lens) or b % 16 == 0 or b in check}
    return check_attention(rng, q_lens, kv_lens, n_q, n_kv, hd, page, c=c, table=table, check=check, **kw)


@pytest.mark.parametrize("hd,page", [(128, 16), (64, 32), (256, 16)])
def test_long_contexts_of_single_tokens(hd, page):
    """More sequences than the GPU has room for, one of them with hundreds of steps for each wave."""
    rng = np.random.default_rng([41, hd])
    lens = rng.integers(0, 70, 300).tolist()
    lens[123] = 13003
    check_long(rng, [1] * 300, lens, 16, 8, hd, page)


@pytest.mark.parametrize("B", [1, 2, 9, 63, 64, 65])
def test_long_contexts_in_any_order(B):
    """Ragged lengths, equal and empty ones among them, in batches that are put in order or not."""
    rng = np.random.default_rng([50, B])
    lens = rng.integers(1, 2600, B).tolist()
    lens[B // 2], lens[-1], lens[0] = 0, lens[0], 2700
    check_long(rng, [1] * B, lens, 4, 2, 128, 32, check=range(B))
    check_long(rng, [1 + b % 3 for b in range(B)], [n + 3 for n in lens], 4, 2, 256, 16, check=range(B), window=700,
               sinks=9)
    if B < 10:
        check_long(rng, [67 + b % 3 for b in range(B)], [n + 70 for n in lens], 4, 2, 128, 32, check=range(B))


@pytest.mark.parametrize("hd,page", [(128, 16), (64, 64), (256, 16)])
def test_long_contexts_of_prompts(hd, page):
    rng = np.random.default_rng([42, hd])
    check_long(rng, [70], [4900], 3, 1, hd, page)
    check_long(rng, [90, 3], [3300, 2700], 2, 1, hd, page, window=1500, sinks=70)
    lens = rng.integers(33, 90, 34).tolist()
    lens[30] = 3471
    check_long(rng, [33] * 34, lens, 16, 8, hd, page)
    check_long(rng, [66] * 34, [n + 33 for n in lens], 16, 8, hd, page)


@pytest.mark.parametrize("n", [1, 6, 70])
def test_a_very_long_context(n):
    """Hundreds of thousands of keys on pages that repeat; with a window only its part is walked."""
    rng = np.random.default_rng([43, n])
    check_long(rng, [n], [200003], 5, 1, 128, 64)
    check_long(rng, [n], [200003], 5, 1, 128, 64, window=50000, sinks=40)


@pytest.mark.parametrize("hd,rows", [(64, 128), (64, 129), (128, 128), (128, 129), (256, 64), (256, 65), (128, 16),
                                     (128, 17), (128, 33), (64, 65), (64, 256), (128, 257), (256, 255), (128, 96),
                                     (128, 97), (256, 17)])
def test_attention_where_the_kernels_meet(hd, rows):
    rng = np.random.default_rng([44, hd, rows])
    check_attention(rng, [rows, 5], [rows + 140, 70], 1, 1, hd, 16, gated=True)
    check_attention(rng, [rows, 3], [rows + 77, 130], 40, 40, hd, 32)
    check_attention(rng, [rows], [rows - 9], 2, 2, hd, 32, window=50)


def test_every_key_counts():
    """Each key's value is its own number and queries are 0, so that the output is the mean over the visible keys:
    a key lost or counted twice anywhere shows."""
    rng = np.random.default_rng(45)
    hd, page, n = 128, 16, 1500
    table, pages = tables(rng, [n], page)
    c = srv.Cache(pages, 1, page, hd, rng)
    v = rng.choice([-127.0, 127.0], (n, 1, hd)).astype(np.float32)
    c.append(table[0], n, rng.standard_normal((n, 1, hd)).astype(np.float32), v)
    for q_len in (1, 3, 140):
        for window, sinks in ((0, 0), (70, 0), (70, 7), (1000, 100)):
            q = torch.zeros(q_len, 2, hd, dtype=torch.bfloat16, device="cuda")
            out = Guarded((q_len, 2, hd), False)
            ws = torch.empty(qmm.qmm_kv8_attn_workspace_bytes(q_len, 1, q_len, 2, 1, hd, table.shape[1] * page, window,
                                                              sinks), dtype=torch.uint8, device="cuda")
            qmm.qmm_kv8_attn(q, gpu_cache(c), dev(table), ints(n), out.t, ws, q_start=ints(0, q_len), max_q=q_len,
                             window=window, sinks=sinks)
            torch.cuda.synchronize()
            got = bf16_bits_to_f64(out.values())
            for j in range(q_len):
                t = np.arange(n)
                see = (t <= n - q_len + j) & ((t > n - q_len + j - window) | (t < sinks) if window else True)
                want = v[see, 0].astype(np.float64).mean(0)
                # sums of whole numbers below 2^24 are exact, weights 1 and scales 1: the division and the bf16 rounding
                assert np.all(np.abs(got[j] - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -20)), (q_len, window, sinks, j)


def test_a_cache_past_32_bit_offsets():
    """The last pages of a pool whose code arrays are larger than 4 GiB each."""
    rng = np.random.default_rng(47)
    n_q, n_kv, hd, page, n = 16, 8, 256, 64, 100
    pages = (1 << 32) // (n_kv * page * hd) + 3
    g = qmm.KV8Cache(*[torch.zeros(s, dtype=torch.int8 if "codes" in k else torch.float32, device="cuda")
                       for k, s in qmm.kv8_cache_shapes(pages, n_kv, page, hd).items()])
    c = srv.Cache(2, n_kv, page, hd)
    k, v = (rng.standard_normal((n, n_kv, hd)).astype(np.float32) for _ in range(2))
    table = np.array([[pages - 1, pages - 2]], np.int32)
    qmm.qmm_kv8_append(g, dev(k), dev(v), dev(table), ints(n), q_start=ints(0, n), max_q=n)
    c.append([1, 0], n, k, v)
    torch.cuda.synchronize()
    for x, y in zip(c.arrays(), g.tensors):
        y = y[-2:].cpu().numpy()
        assert np.array_equal(x[1], y[1]) and np.array_equal(x[0, :, :2], y[0, :, :2])  # 36 keys of the second page
    qb, qv = bf16(rng.standard_normal((n, n_q, hd)))
    for first in (n - 1, 0):  # one token, then the whole prompt
        m = n - first
        out = Guarded((m, n_q, hd), False)
        ws = torch.empty(qmm.qmm_kv8_attn_workspace_bytes(m, 1, m, n_q, n_kv, hd, 2 * page), dtype=torch.uint8,
                         device="cuda")
        qmm.qmm_kv8_attn(dev(qb[first:]), g, dev(table), ints(n), out.t, ws, q_start=ints(0, m), max_q=m)
        torch.cuda.synchronize()
        ref, tol = srv.attention(qv[first:], c, [1, 0], n, m, hd ** -0.5, few=few_rows(m * n_q // n_kv))
        assert_within(bf16_bits_to_f64(out.values()), ref, tol, f"{m} queries")


@pytest.mark.parametrize("q_len", [1, 4, 40])
@pytest.mark.parametrize("hd,bad", [(128, np.nan), (128, 1e30), (256, np.nan), (64, np.inf)])
def test_blocks_behind_the_window_may_have_any_scale(q_len, hd, bad):
    """A server may have given pages away that no row sees any more, while the table still names them."""
    rng = np.random.default_rng([49, q_len, hd])
    for kv, window, sinks in ((300, 60, 0), (300, 47, 5), (97, 33, 16)):
        c, table = filled(rng, [kv], 2, hd, 16)
        want = check_attention(rng, [q_len], [kv], 8, 2, hd, 16, window=window, sinks=sinks, c=c, table=table)
        for t in range(-(-sinks // 16), (kv - q_len - window + 1) // 16):
            c.k_scale[table[0, t]] = c.v_scale[table[0, t]] = bad
        out = bf16_bits_to_f64(check_given_away(rng, q_len, kv, hd, window, sinks, c, table))
        assert np.all(np.isfinite(out))


def check_given_away(rng, q_len, kv, hd, window, sinks, c, table):
    """Outputs with those blocks' scales as they are and with ones: the same bits."""
    qb, _ = bf16(rng.standard_normal((q_len, 8, hd)))
    got = []
    for clean in (False, True):
        if clean:
            for s in (c.k_scale, c.v_scale):
                s[~(np.abs(s) < 1e20)] = 1.0
        out = torch.empty(q_len, 8, hd, dtype=torch.bfloat16, device="cuda")
        need = qmm.qmm_kv8_attn_workspace_bytes(q_len, 1, q_len, 8, 2, hd, table.shape[1] * 16, window, sinks)
        qmm.qmm_kv8_attn(dev(qb), gpu_cache(c), dev(table), ints(kv), out, torch.empty(need, dtype=torch.uint8, device="cuda"),
                         q_start=ints(0, q_len), max_q=q_len, window=window, sinks=sinks)
        torch.cuda.synchronize()
        got.append(out.view(torch.int16).cpu().numpy().view(np.uint16))
    assert np.array_equal(got[0], got[1])
    return got[0]


def test_two_sequences_share_their_first_pages():
    rng = np.random.default_rng(48)
    c, table = filled(rng, [64], 2, 128, 16, spare=6)
    free = [p for p in range(c.n_pages) if p not in table[0]]
    both = np.array([list(table[0, :4]) + [free[0]], list(table[0, :4]) + [free[1]]], np.int32)
    g = gpu_cache(c)
    k, v = (rng.standard_normal((4, 2, 128)).astype(np.float32) for _ in range(2))
    qmm.qmm_kv8_append(g, dev(k), dev(v), dev(both), ints(67, 65), q_start=ints(0, 3, 4), max_q=3)
    c.append(both[0], 67, k[:3], v[:3])
    c.append(both[1], 65, k[3:], v[3:])
    same_cache(c, g, both, [67, 65])
    check_attention(rng, [3, 1], [67, 65], 4, 2, 128, 16, c=c, table=both)


def test_calls_repeat_bit_for_bit():
    for q_lens in ([1, 1, 1], [3, 4, 1], [70, 40, 9]):
        got = [check_long(np.random.default_rng(49), q_lens, [5000, 300, 77], 8, 2, 128, 32, check=()) for _ in range(3)]
        assert np.array_equal(got[0], got[1]) and np.array_equal(got[0], got[2])
    say("  the same bits")
