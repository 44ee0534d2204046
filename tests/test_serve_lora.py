"""GPU parity of low-rank adapters beside a projection (qmm_serve.h) with oracle/serve_oracle.py."""
import numpy as np
import pytest
import torch

import gemm_affine_u4_amd as qmm
import synth
from oracle import serve_oracle as srv
from tests.gpu_util import Guarded, assert_within, bf16_bits_to_f64, dev, dev_weight
from tests.serve_util import bf16, whole_adapters

pytestmark = pytest.mark.gpu


def values(x, f32):
    return np.asarray(x, np.float32).astype(np.float64) if f32 else bf16(x)[1]


def up(x, f32):
    return dev(np.asarray(x, np.float32)) if f32 else dev(bf16(x)[0])


def check(rng, ids, n_ad, rank, K, rows, base32, out32, scales=True, in_place=False, rows_checked=24):
    ids = np.asarray(ids, np.int32)
    T, parts, total = len(ids), len(rows), sum(rows)
    x = bf16(rng.standard_normal((T, K)))
    a = bf16(rng.standard_normal((n_ad, parts * rank, K)) / np.sqrt(K))
    b = bf16(rng.standard_normal((n_ad, total, rank)))
    s = rng.uniform(-2, 2, n_ad).astype(np.float32) if scales else None
    base = [values(rng.standard_normal((T, n)), base32) for n in rows]
    outs = [Guarded((T, n), out32) for n in rows]
    for o in outs:
        o.poison()
    if in_place:
        for o, v in zip(outs, base):
            o.t.copy_(up(v, out32))
    need = qmm.qmm_lora_workspace_bytes(T, K, rank, parts)
    ws = torch.full((need + 1024,), 0xFF, dtype=torch.uint8, device="cuda")
    y = [o.t for o in outs]
    qmm.qmm_lora(dev(x[0]), dev(a[0]), dev(b[0]), dev(ids), y if parts > 1 else y[0], ws[:need],
                 base=None if in_place else [up(v, base32) for v in base] if parts > 1 else up(base[0], base32),
                 scales=None if s is None else dev(s))
    torch.cuda.synchronize()
    assert bool((ws[need:] == 0xFF).all()), "write behind the workspace"
    at = np.unique(np.concatenate([[0, T - 1], rng.integers(0, T, rows_checked)])) if T > rows_checked else np.arange(T)
    row = 0
    for p, n in enumerate(rows):
        got = outs[p].values()
        got = got if out32 else bf16_bits_to_f64(got)
        ref, tol = srv.lora(x[1][at], a[1][:, p * rank:(p + 1) * rank], b[1][:, row:row + n], ids[at], base[p][at], s,
                            2.0 ** -24 if out32 else 2.0 ** -8)
        assert_within(got[at], ref, tol, f"part {p}")
        none = (ids < 0) | (ids >= n_ad)
        want = base[p][none] if out32 else bf16(base[p][none])[1]
        assert np.array_equal(got[none], want), "tokens without an adapter"
        assert np.all(np.isfinite(got))
        row += n
    return outs


@pytest.mark.parametrize("rank", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("rows", [[512], [320, 64, 64], [33], [100, 7, 250], [272, 16]])
@pytest.mark.parametrize("T", [1, 20])
def test_a_batch(rank, rows, T):
    rng = np.random.default_rng([rank, rows[0], T])
    check(rng, rng.integers(-1, 6, T) if T > 1 else [3], 6, rank, 512, rows, False, False)
    check(rng, rng.integers(-1, 7, T), 6, rank, 192, rows, True, True, scales=False)


@pytest.mark.parametrize("base32,out32", [(False, False), (True, False), (True, True), (False, True)])
def test_types(base32, out32):
    rng = np.random.default_rng([base32, out32])
    check(rng, [0, 1, -1, 1, 99], 2, 16, 1024, [256, 128], base32, out32)
    check(rng, rng.integers(-1, 2, 300), 2, 16, 256, [256, 40], base32, out32)


@pytest.mark.parametrize("f32", [False, True])
def test_in_place(f32):
    rng = np.random.default_rng(5)
    check(rng, [2, -1, 0, 0, 2], 3, 16, 320, [160, 48], f32, f32, in_place=True)
    check(rng, rng.integers(-1, 3, 270), 3, 32, 320, [161], f32, f32, in_place=True)


@pytest.mark.parametrize("rank,rows", [(8, [512]), (16, [300, 60, 60]), (64, [1000]), (128, [128, 128])])
@pytest.mark.parametrize("T", [256, 257, 1000])
def test_prompts(rank, rows, T):
    """Requests that stand side by side, and tokens whose adapters follow no order."""
    rng = np.random.default_rng([rank, T])
    runs = np.repeat([4, -1, 0, 2, 9, 1], rng.multinomial(T, np.ones(6) / 6))
    check(rng, runs, 5, rank, 640, rows, True, True)
    check(rng, rng.integers(0, 40, T), 40, rank, 128, rows, False, False)


@pytest.mark.parametrize("rank,T", [(16, 2048), (16, 2049), (64, 2500), (8, 2111)])
def test_thousands_of_tokens_of_mixed_adapters(rank, T):
    rng = np.random.default_rng([31, rank, T])
    runs = rng.integers(1, 90, T)
    ids = np.repeat(rng.integers(-1, 41, T), runs)[:T]
    check(rng, ids, 40, rank, 256, [272, 40], True, False, rows_checked=80)
    check(rng, rng.integers(-1, 41, T), 40, rank, 192, [96], False, True, rows_checked=80)


def test_long_inputs_and_every_tile_full_of_adapters():
    rng = np.random.default_rng(6)
    check(rng, np.arange(64), 64, 16, 13824, [96], True, True, rows_checked=8)
    check(rng, np.arange(300) % 64, 64, 8, 64, [64], True, True)   # 64 distinct ones in a tile of 64
    check(rng, [-1] * 40, 3, 8, 64, [64], True, False)             # none at all
    check(rng, [7] * 17, 8, 32, 65536, [16], True, True, rows_checked=3)


def test_a_row_does_not_depend_on_the_others():
    """The same tokens in another order, and among other requests, bit for bit within a launch shape."""
    rng = np.random.default_rng(7)
    T, K, r, n = 60, 512, 16, 320
    x = dev(bf16(rng.standard_normal((T, K)))[0])
    a, b = dev(bf16(rng.standard_normal((9, r, K)))[0]), dev(bf16(rng.standard_normal((9, n, r)))[0])
    base = dev(rng.standard_normal((T, n)).astype(np.float32))
    ids = dev(rng.integers(-1, 9, T).astype(np.int32))
    ws = torch.empty(qmm.qmm_lora_workspace_bytes(T, K, r), dtype=torch.uint8, device="cuda")

    def run(order):
        y = torch.empty_like(base)
        qmm.qmm_lora(x[order].contiguous(), a, b, ids[order].contiguous(), y, ws, base=base[order].contiguous())
        back = torch.empty_like(y)
        back[order] = y
        return back

    want = run(torch.arange(T, device="cuda"))
    for _ in range(3):
        assert torch.equal(run(torch.randperm(T, device="cuda")), want)


def test_past_32_bit_offsets():
    """Outputs and weights of more than 4 GiB: the last tokens and the last adapter."""
    rng = np.random.default_rng(8)
    T, n, r, K = 70000, 16384, 8, 64
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    xv = bf16(rng.standard_normal((3, K)))
    x[-3:] = dev(xv[0]).view(torch.bfloat16)
    n_ad = (1 << 32) // (n * r * 2) + 2
    b = torch.zeros(n_ad, n, r, dtype=torch.bfloat16, device="cuda")
    bv = bf16(rng.standard_normal((n, r)))
    b[-1] = dev(bv[0]).view(torch.bfloat16)
    av = bf16(rng.standard_normal((r, K)))
    a = torch.zeros(n_ad, r, K, dtype=torch.bfloat16, device="cuda")
    a[-1] = dev(av[0]).view(torch.bfloat16)
    y = torch.ones(T, n, dtype=torch.float32, device="cuda")
    ids = torch.full((T,), n_ad - 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(qmm.qmm_lora_workspace_bytes(T, K, r), dtype=torch.uint8, device="cuda")
    qmm.qmm_lora(x, a, b, ids, y, ws)
    torch.cuda.synchronize()
    assert bool((y[:-3] == 1).all())
    ref, tol = srv.lora(xv[1], av[1][None], bv[1][None], [0] * 3, np.ones((3, n)), None, 2.0 ** -24)
    assert_within(y[-3:].cpu().numpy(), ref, tol, "the last tokens")


@pytest.mark.parametrize("T", [5, 400])
def test_in_a_graph_and_on_another_stream(T):
    rng = np.random.default_rng(9)
    K, r, n = 512, 16, 200
    x = dev(bf16(rng.standard_normal((T, K)))[0])
    a, b = dev(bf16(rng.standard_normal((9, r, K)))[0]), dev(bf16(rng.standard_normal((9, n, r)))[0])
    base = dev(rng.standard_normal((T, n)).astype(np.float32))
    ids = dev(rng.integers(-1, 9, T).astype(np.int32))
    need = qmm.qmm_lora_workspace_bytes(T, K, r)
    y, ws = torch.empty_like(base), torch.empty(need, dtype=torch.uint8, device="cuda")
    qmm.qmm_lora(x, a, b, ids, y, ws, base=base)
    torch.cuda.synchronize()
    want = y.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y.zero_()
    qmm_stream = side
    side.wait_stream(torch.cuda.current_stream())
    qmm.qmm_lora(x, a, b, ids, y, ws, base=base, stream=qmm_stream)
    side.synchronize()
    assert torch.equal(y, want)
    graphs = []
    for _ in range(2):
        o, w = torch.empty_like(base), torch.empty(need, dtype=torch.uint8, device="cuda")
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            qmm.qmm_lora(x, a, b, ids, o, w, base=base)
        graphs.append((gr, o, w))
    for _ in range(3):
        for gr, o, w in graphs:
            o.fill_(7.0)
            w.fill_(255)
            gr.replay()
            qmm.qmm_lora(x, a, b, ids, y, ws, base=base)
            torch.cuda.synchronize()
            assert torch.equal(o, want) and torch.equal(y, want)


@pytest.mark.parametrize("rank", [8, 32, 128])
@pytest.mark.parametrize("T,K", [(1, 64), (20, 2048), (300, 2048), (3000, 512)])
def test_all_bits_of_h(T, K, rank):
    """h is taken on with 24 bits: outputs of exact products and sums are right to half a step of fp32."""
    rng = np.random.default_rng([33, T, rank])
    rows = 272
    x, a, b, ids, want = whole_adapters(rng, T, K, rank, rows, 5)
    y = Guarded((T, rows), True)
    y.t.zero_()
    ws = torch.empty(qmm.qmm_lora_workspace_bytes(T, K, rank), dtype=torch.uint8, device="cuda")
    qmm.qmm_lora(dev(bf16(x)[0]), dev(bf16(a)[0]), dev(bf16(b)[0]), dev(ids), y.t, ws)
    torch.cuda.synchronize()
    assert_within(y.values(), want, np.abs(want) * 2.0 ** -24, "whole numbers")


def test_beside_the_quantized_projection():
    """qmm_linear in fp32, then the adapters, rounded once to bf16."""
    rng = np.random.default_rng(10)
    K, N, T, r = 512, 192, 6, 8
    w = synth.gen_weight(synth.CFG_TEST, 9, synth.PROJ_QKV, N, K)
    xb, xv = bf16(rng.standard_normal((T, K)))
    p = torch.empty(T, N, dtype=torch.float32, device="cuda")
    qmm.qmm_linear(dev(xb), *dev_weight(w), p)
    a, b = bf16(rng.standard_normal((2, r, K)) / 20), bf16(rng.standard_normal((2, N, r)))
    ids = np.array([0, 1, 1, -1, 0, 5], np.int32)
    out = Guarded((T, N), False)
    ws = torch.empty(qmm.qmm_lora_workspace_bytes(T, K, r), dtype=torch.uint8, device="cuda")
    qmm.qmm_lora(dev(xb), dev(a[0]), dev(b[0]), dev(ids), out.t, ws, base=p)
    torch.cuda.synchronize()
    ref, tol = srv.lora(xv, a[1], b[1], ids, p.cpu().numpy(), None, 2.0 ** -8)
    assert_within(bf16_bits_to_f64(out.values()), ref, tol, "linear + adapters")
