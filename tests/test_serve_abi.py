"""A serving step's boundary without a GPU: the header's entry points are exported, bad arguments are refused before
anything is enqueued, and the oracle's own pins."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import gemm_affine_u4_amd as qmm
from oracle import serve_oracle as srv
from tests.serve_util import bf16, whole_adapters

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
S = qmm.STATUS
MB = 1 << 20
A = 1 << 32  # fake device addresses, never dereferenced
B0 = A + 256 * MB


def test_header_functions_are_exported():
    text = open(os.path.join(ROOT, "include", "qmm_serve.h")).read()
    names = sorted(set(re.findall(r"^(?:int|size_t)\s+(qmm_\w+)\s*\(", text, re.M)))
    assert names == ["qmm_kv8_append", "qmm_kv8_attn", "qmm_kv8_attn_workspace_bytes", "qmm_lora",
                     "qmm_lora_workspace_bytes", "qmm_spec_verify", "qmm_spec_verify_workspace_bytes"]
    out = subprocess.run(["nm", "-D", "--defined-only", qmm.LIB_PATH], capture_output=True, text=True).stdout
    assert set(names) <= set(re.findall(r" T (qmm_\w+)$", out, re.M))
    assert set(names) <= set(qmm.__all__)


class Kv8Struct(ctypes.Structure):
    """qmm_kv8_cache of the C ABI."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_codes", "k_scale", "v_codes", "v_scale")] + [
        (n, ctypes.c_int64) for n in ("n_pages", "page_size", "n_kv_heads", "head_dim")]


def cache(**kw):
    f = dict(k_codes=A, k_scale=A + 64 * MB, v_codes=A + 128 * MB, v_scale=A + 192 * MB, n_pages=8, page_size=32,
             n_kv_heads=2, head_dim=128)
    f.update(kw)
    return Kv8Struct(*[f[n] for n, _ in Kv8Struct._fields_])


def append(c=None, **kw):
    f = dict(k=B0, v=B0 + MB, T=4, dt=0, q_start=B0 + 2 * MB, kv_lens=B0 + 2 * MB + 4096, table=B0 + 2 * MB + 8192, B=2,
             max_pages=4, max_q=3, positions=B0 + 3 * MB, cos_sin=B0 + 4 * MB, max_pos=64, rot=128, q=B0 + 5 * MB, n_q=4,
             q_out=B0 + 6 * MB, k_held=B0 + 7 * MB, v_held=B0 + 8 * MB)
    f.update(kw)
    c = cache() if c is None else c
    return qmm.load_library().qmm_kv8_append(ctypes.addressof(c) if c else None, *f.values(), None)


def attn(c=None, **kw):
    f = dict(q=B0, T=3, q_start=B0 + MB, kv_lens=B0 + 2 * MB, table=B0 + 3 * MB, B=2, max_pages=4, max_q=2,
             cache=None, n_q=4, scale=0.1, causal=1, window=9, sinks=2, gate=B0 + 4 * MB, ws=B0 + 8 * MB,
             ws_bytes=64 * MB, out=B0 + 5 * MB)
    f.update(kw)
    c = cache() if c is None else c
    f["cache"] = ctypes.addressof(c) if c else None
    return qmm.load_library().qmm_kv8_attn(*f.values(), None)


def verify(**kw):
    f = dict(draft=B0, D=7, start=B0 + MB, B=3, max_draft=4, p=B0 + 2 * MB, q=B0 + 4 * MB, V=1000, dt=1, u=B0 + 6 * MB,
             tokens=B0 + 7 * MB, accepted=B0 + 8 * MB, ws=B0 + 9 * MB, ws_bytes=MB)
    f.update(kw)
    return qmm.load_library().qmm_spec_verify(*f.values(), None)


def lora(**kw):
    f = dict(x=B0, T=5, K=512, a=B0 + MB, b=B0 + 2 * MB, n=3, rank=16, ids=B0 + 3 * MB, scales=B0 + 3 * MB + 4096,
             parts=2, rows=(64, 32), base=(B0 + 4 * MB, B0 + 5 * MB), base_dt=1, y=(B0 + 6 * MB, B0 + 7 * MB), dt=0,
             ws=B0 + 8 * MB, ws_bytes=16 * MB)
    f.update(kw)
    if f["rows"] is not None:
        f["rows"] = (ctypes.c_int64 * 3)(*f["rows"])
    for name in ("base", "y"):
        if f[name] is not None:
            f[name] = (ctypes.c_void_p * 3)(*f[name])
    return qmm.load_library().qmm_lora(*f.values(), None)


@pytest.mark.parametrize("bad, want", [
    (dict(k_codes=None), "NULL"), (dict(v_scale=None), "NULL"), (dict(head_dim=96), "SHAPE"),
    (dict(head_dim=512), "SHAPE"), (dict(page_size=8), "SHAPE"), (dict(page_size=48), "SHAPE"),
    (dict(page_size=8192), "SHAPE"), (dict(n_pages=0), "SHAPE"), (dict(n_pages=1 << 27), "SHAPE"),
    (dict(n_kv_heads=0), "SHAPE"), (dict(k_codes=A + 8), "ALIGN"), (dict(v_scale=A + 192 * MB + 4), "ALIGN")])
def test_bad_caches(bad, want):
    assert append(cache(**bad)) == S["QMM_ERR_" + want]
    assert attn(cache(**bad)) == S["QMM_ERR_" + want]


@pytest.mark.parametrize("bad, want", [
    (dict(k=None), "NULL"), (dict(kv_lens=None), "NULL"), (dict(table=None), "NULL"), (dict(q_out=None), "NULL"),
    (dict(cos_sin=None, q=None), "NULL"), (dict(cos_sin=None, positions=None), "NULL"),
    (dict(dt=2), "ENUM"), (dict(T=-1), "SHAPE"), (dict(T=(1 << 24) + 1), "SHAPE"), (dict(rot=3), "SHAPE"),
    (dict(rot=130), "SHAPE"), (dict(rot=0), "SHAPE"), (dict(max_pos=0), "SHAPE"), (dict(n_q=0), "SHAPE"),
    (dict(B=0), "SHAPE"), (dict(B=65536), "SHAPE"), (dict(max_q=0), "SHAPE"), (dict(max_pages=0), "SHAPE"),
    (dict(B=65535, max_q=1 << 24), "SHAPE"), (dict(q_start=None), "SHAPE"), (dict(max_pages=1 << 26), "SHAPE"),
    (dict(k=B0 + 2), "ALIGN"), (dict(table=B0 + 2 * MB + 2), "ALIGN"), (dict(v_held=B0 + 8 * MB + 8), "ALIGN"),
    (dict(q_out=B0 + 5 * MB), "ALIAS"), (dict(k_held=B0 + 8 * MB + 256), "ALIAS"), (dict(k=A + 16), "ALIAS"),
    (dict(kv_lens=A + 64 * MB), "ALIAS")])
def test_append_refuses(bad, want):
    assert append(**bad) == S["QMM_ERR_" + want]


def test_append_of_more_blocks_than_a_launch_has_threads_for_is_refused():
    """A wave for each block of 16 keys that a sequence may meet, four waves of 64 in a workgroup, below 2^32 threads."""
    for B, max_q in ((8191, 131058), (1, (1 << 24)), (65535, 16 * 1021 + 2), (65532, 16 * 1022 + 2)):
        threads = (B * ((max_q + 14) // 16 + 1) + 3) // 4 * 256
        assert append(T=0, B=B, max_q=max_q, max_pages=1) == (S["QMM_ERR_SHAPE"] if threads >= 1 << 32 else 0), (B, max_q)


@pytest.mark.parametrize("bad, want", [
    (dict(q=None), "NULL"), (dict(kv_lens=None), "NULL"), (dict(table=None), "NULL"), (dict(ws=None), "NULL"),
    (dict(out=None), "NULL"), (dict(causal=2), "ENUM"), (dict(window=-1), "SHAPE"), (dict(causal=0, sinks=0), "SHAPE"),
    (dict(sinks=-1), "SHAPE"), (dict(window=0), "SHAPE"),  # sinks without a window
    (dict(n_q=3), "SHAPE"), (dict(n_q=0), "SHAPE"), (dict(scale=0.0), "SHAPE"), (dict(scale=float("nan")), "SHAPE"),
    (dict(scale=float("inf")), "SHAPE"), (dict(B=0), "SHAPE"), (dict(max_q=0), "SHAPE"), (dict(max_pages=0), "SHAPE"),
    (dict(max_pages=1 << 26), "SHAPE"), (dict(q_start=None), "SHAPE"), (dict(ws_bytes=0), "SHAPE"),
    (dict(T=-1), "SHAPE"), (dict(max_q=1 << 24), "SHAPE"),
    (dict(q=B0 + 2), "ALIGN"), (dict(ws=B0 + 8 * MB + 16), "ALIGN"), (dict(gate=B0 + 4 * MB + 2), "ALIGN"),
    (dict(out=B0), "ALIAS"), (dict(ws=A), "ALIAS"), (dict(out=A + 128 * MB), "ALIAS"), (dict(out=B0 + 3 * MB), "ALIAS")])
def test_attention_refuses(bad, want):
    assert attn(**bad) == S["QMM_ERR_" + want]


@pytest.mark.parametrize("bad, want", [
    (dict(draft=None), "NULL"), (dict(start=None), "NULL"), (dict(p=None), "NULL"), (dict(u=None), "NULL"),
    (dict(tokens=None), "NULL"), (dict(accepted=None), "NULL"), (dict(ws=None), "NULL"), (dict(dt=2), "ENUM"),
    (dict(B=0), "SHAPE"), (dict(B=65536), "SHAPE"), (dict(V=0), "SHAPE"), (dict(V=(1 << 24) + 1), "SHAPE"),
    (dict(D=-1), "SHAPE"), (dict(max_draft=-1), "SHAPE"), (dict(max_draft=65536), "SHAPE"), (dict(ws_bytes=8), "SHAPE"),
    (dict(p=B0 + 2 * MB + 2), "ALIGN"), (dict(tokens=B0 + 7 * MB + 1), "ALIGN"), (dict(ws=B0 + 9 * MB + 8), "ALIGN"),
    (dict(tokens=B0 + 8 * MB - 8), "ALIAS"), (dict(accepted=B0), "ALIAS"), (dict(ws=B0 + 2 * MB), "ALIAS")])
def test_verify_refuses(bad, want):
    assert verify(**bad) == S["QMM_ERR_" + want]


@pytest.mark.parametrize("bad, want", [
    (dict(x=None), "NULL"), (dict(a=None), "NULL"), (dict(b=None), "NULL"), (dict(ids=None), "NULL"),
    (dict(rows=None), "NULL"), (dict(y=None), "NULL"), (dict(ws=None), "NULL"), (dict(y=(B0 + 6 * MB, None)), "NULL"),
    (dict(base=(None, B0 + 5 * MB)), "NULL"), (dict(dt=3), "ENUM"), (dict(base_dt=-1), "ENUM"),
    (dict(K=96), "SHAPE"), (dict(K=0), "SHAPE"), (dict(rank=24), "SHAPE"), (dict(rank=256), "SHAPE"),
    (dict(parts=0), "SHAPE"), (dict(parts=4), "SHAPE"), (dict(n=0), "SHAPE"), (dict(n=65536), "SHAPE"),
    (dict(T=-1), "SHAPE"), (dict(rows=(64, 0)), "SHAPE"), (dict(ws_bytes=64), "SHAPE"),
    (dict(T=1 << 24, K=64, rank=8, rows=(1 << 22, 64), ws_bytes=1 << 50), "SHAPE"),
    (dict(x=B0 + 8), "ALIGN"), (dict(b=B0 + 2 * MB + 2), "ALIGN"), (dict(ids=B0 + 3 * MB + 2), "ALIGN"),
    (dict(base=(B0 + 4 * MB + 2, B0 + 5 * MB)), "ALIGN"), (dict(y=(B0 + 6 * MB + 1, B0 + 7 * MB)), "ALIGN"),
    (dict(y=(B0 + 4 * MB, B0 + 7 * MB)), "ALIAS"),  # in place needs one dtype
    (dict(y=(B0 + 6 * MB, B0 + 6 * MB)), "ALIAS"), (dict(y=(B0, B0 + 7 * MB)), "ALIAS"), (dict(ws=B0), "ALIAS"),
    (dict(base_dt=0, y=(B0 + 5 * MB, B0 + 4 * MB)), "ALIAS")])  # the other part's base
def test_lora_refuses(bad, want):
    assert lora(**bad) == S["QMM_ERR_" + want]


def test_workspace_bytes():
    f = qmm.qmm_kv8_attn_workspace_bytes
    assert f(1, 1, 1, 8, 2, 128, 64) > 0
    for bad in ((1, 0, 1, 8, 2, 128, 64), (1, 1, 1, 7, 2, 128, 64), (1, 1, 1, 8, 2, 100, 64), (1, 1, 1, 8, 2, 128, 0),
                (1, 1, 1, 8, 2, 128, 1 << 31), (1, 1, 1, 8, 2, 128, 64, -1, 0), (1, 1, 1, 8, 2, 128, 64, 0, 4)):
        assert f(*bad) == 0
    assert qmm.qmm_spec_verify_workspace_bytes(1, 1) > 0
    assert qmm.qmm_spec_verify_workspace_bytes(0, 1) == 0 and qmm.qmm_spec_verify_workspace_bytes(1, 0) == 0
    assert qmm.qmm_lora_workspace_bytes(0, 64, 8) > 0 and qmm.qmm_lora_workspace_bytes(4, 64, 12) == 0
    assert qmm.qmm_lora_workspace_bytes(4, 100, 8) == 0 and qmm.qmm_lora_workspace_bytes(4, 64, 8, 4) == 0


@pytest.mark.parametrize("B,max_q,max_kv,window", [(1, 1, 131072, 0), (4, 3, 20000, 4000), (1, 90, 9000, 0),
                                                   (64, 1, 64, 0)])
def test_workspace_bytes_of_no_tokens(B, max_q, max_kv, window):
    """A step without tokens is one of valid sizes: some bytes, and a call with as many enqueues nothing."""
    need = qmm.qmm_kv8_attn_workspace_bytes(0, B, max_q, 4, 2, 128, max_kv, window, 0)
    assert 0 < need <= qmm.qmm_kv8_attn_workspace_bytes(1, B, max_q, 4, 2, 128, max_kv, window, 0)
    assert attn(T=0, B=B, max_q=max_q, max_pages=max_kv // 32, window=window, sinks=0, ws_bytes=need) == 0


def test_python_side_refuses_host_tensors():
    shapes = qmm.kv8_cache_shapes(2, 1, 32, 64)
    t = [torch.zeros(s, dtype=torch.int8 if "codes" in n else torch.float32) for n, s in shapes.items()]
    with pytest.raises(ValueError, match="device tensor"):
        qmm.KV8Cache(*t)
    with pytest.raises(ValueError, match="v_codes"):
        qmm.KV8Cache(t[0], t[1], t[0], t[3])
    with pytest.raises(ValueError, match="k_scale"):
        qmm.KV8Cache(t[0], t[1].double(), t[2], t[3])


# ---- the oracle's own pins -----------------------------------------------------------------

def test_append_oracle_bounds():
    """A block that fills token by token: what is held stays within 2.5 steps, a block written at once within half."""
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((40, 2, 64)) * np.linspace(0.2, 3, 40)[:, None, None]).astype(np.float32)
    for parts, steps in (([40], 0.5), ([1] * 40, 2.5), ([5, 20, 15], 2.5)):
        c = srv.Cache(3, 2, 16, 64, rng)
        done = 0
        for n in parts:
            held = c.append([2, 0, 1], done + n, x[done:done + n], x[done:done + n] * 0.5)
            done += n
        assert np.all(np.isfinite(held[0]))
        t = np.arange(40)
        for h in range(2):
            k, v, vs = c.get(np.array([2, 0, 1])[t // 16], t % 16, h)
            ks = c.k_scale[np.array([2, 0, 1])[t // 16], h, 0]
            assert np.all(np.abs(k - x[:, h]) <= (steps + 1e-5) * ks[:, None])
            assert np.all(np.abs(v - 0.5 * x[:, h]) <= (steps + 1e-5) * vs[:, None])


def test_append_oracle_corners():
    c = srv.Cache(1, 1, 16, 64)
    x = np.zeros((3, 1, 64), np.float32)
    x[1, 0, 0], x[2, 0, 1] = 1e9, -3.0
    k, _ = c.append([0], 3, x, x)
    assert k[1, 0, 0] == np.float32(57344) and np.all(k[0] == 0)  # clamped
    k, _ = c.append([0], 3, x[:1] * 0, x[:1])                       # one token anew, in the same place
    assert np.all(k == 0) and c.k_scale[0, 0, 0] == np.float32(57344) * np.float32(1 / 127)
    k, _ = c.append([0], 1, x[:1], x[:1])                           # begins the block: all zeros
    assert c.k_scale[0, 0, 0] == 0 and np.all(k == 0)
    k, _ = c.append([0], 2, x[2:], x[2:])                           # a zero scale grows
    assert c.k_scale[0, 0, 0] == np.float32(3) * np.float32(1 / 127) and np.isclose(k[0, 0, 1], -3)
    k, _ = c.append([-1], 2, x[:2], x[:2])                          # no page
    assert np.all(np.isnan(k))
    k, _ = c.append([0], 2, x, x)                                   # more tokens than keys
    assert np.all(np.isnan(k[0])) and np.all(np.isfinite(k[1:]))


def test_attention_oracle_against_definition():
    rng = np.random.default_rng(2)
    c = srv.Cache(4, 1, 16, 64, rng)
    x = rng.standard_normal((34, 1, 64)).astype(np.float32)
    c.append([1, 2, 3], 34, x, x[::-1].copy())
    q = rng.standard_normal((3, 2, 64))
    t = np.arange(34)
    k, v, _ = c.get(np.array([1, 2, 3])[t // 16], t % 16, 0)
    assert np.abs(k - x[:, 0]).max() < 0.02
    out, _ = srv.attention(q, c, [1, 2, 3], 34, 3, 0.125)
    win, _ = srv.attention(q, c, [1, 2, 3], 34, 3, 0.125, window=5, sinks=2)
    for j in range(3):
        for a in range(2):
            w = np.exp(0.125 * (k @ q[j, a])) * (t <= 31 + j)
            assert np.allclose(out[j, a], (w[:, None] * v).sum(0) / w.sum(), rtol=1e-12)
            w = w * ((t > 26 + j) | (t < 2))
            assert np.allclose(win[j, a], (w[:, None] * v).sum(0) / w.sum(), rtol=1e-12)
    out, _ = srv.attention(q, c, [1], 1, 3, 0.125)
    assert np.all(out[:2] == 0) and np.allclose(out[2], v[0])


def test_verify_oracle_keeps_the_target_distribution():
    """Kept draft or new token at the first place, over many numbers: the target's frequencies."""
    rng = np.random.default_rng(3)
    V, N = 5, 40000
    p, q = rng.dirichlet(np.ones(V)), rng.dirichlet(np.ones(V))
    draft = rng.choice(V, N, p=q)
    start = np.arange(N + 1)
    target = np.tile(p, (2 * N, 1))
    for probs in (np.tile(q, (N, 1)), None):
        tokens, acc = srv.verify(draft, start, target, probs, rng.random(2 * N), 1)
        if probs is None:  # looked-up drafts: the same for any of them
            draft = np.full(N, int(p.argmax()))
            tokens, acc = srv.verify(draft, start, target, probs, rng.random(2 * N), 1)
        got = np.bincount(tokens[:, 0], minlength=V) / N
        assert np.abs(got - p).max() < 5 * np.sqrt(0.25 / N)
        assert np.all((tokens[:, 1] >= 0) == (acc == 1))


def test_verify_oracle_corners():
    target = np.array([[0, 0.5, 0.5, 0], [0, 0, 0, 1.0], [0.25, 0.25, 0.25, 0.25]])
    t, a = srv.verify(np.array([1, 3]), np.array([0, 2]), target, None, np.array([0.4, 0.99, 0.5]), 2)
    assert t.tolist() == [[1, 3, 2]] and a[0] == 2
    t, a = srv.verify(np.array([1, 3]), np.array([0, 2]), target, None, np.array([0.5, 0.0, 0.999]), 2)
    assert t.tolist() == [[2, -1, -1]] and a[0] == 0   # 1 is refused, and has no weight left
    t, a = srv.verify(np.array([9, 3]), np.array([0, 2]), target, None, np.array([0.0, 0.0, 0.0]), 2)
    assert t.tolist() == [[1, -1, -1]]                # no such token; zeros in front are passed over
    q = target[:2]
    t, a = srv.verify(np.array([0, 3]), np.array([0, 2]), target, q, np.array([0.0, 0.0, 0.9]), 2)
    assert t.tolist() == [[2, -1, -1]]                # nothing left of p - q: p itself
    t, a = srv.verify(np.array([0]), np.array([0, 1]), np.zeros((2, 4)), None, np.array([0.3, 0.3]), 1)
    assert t.tolist() == [[-1, -1]]


def test_lora_oracle():
    rng = np.random.default_rng(4)
    x, a, b = rng.standard_normal((3, 8)), rng.standard_normal((2, 4, 8)), rng.standard_normal((2, 5, 4))
    base = rng.standard_normal((3, 5))
    y, _ = srv.lora(x, a, b, [1, -1, 0], base, [2.0, 0.5], 0)
    assert np.allclose(y[0], base[0] + 0.5 * b[1] @ a[1] @ x[0]) and np.all(y[1] == base[1])
    assert np.allclose(y[2], base[2] + 2 * b[0] @ a[0] @ x[2])


def test_adapters_that_show_all_bits_of_h():
    """Of the inputs that the GPU's adapters are held against: three bf16 pieces of h give the outputs, two do not, and the
    oracle's bound for any inputs would not have told them apart."""
    x, a, b, ids, want = whole_adapters(np.random.default_rng(5), 40, 64, 8, 24, 3)
    for t in (x, a, b):
        assert np.array_equal(bf16(t)[1], t)
    ref, tol = srv.lora(x, a, b, ids, np.zeros(want.shape), None, 2.0 ** -24)
    assert np.array_equal(ref, want)
    for pieces in (3, 2):
        h, left = np.zeros((40, 8)), np.einsum("tk,trk->tr", x.astype(np.float64), a[ids])
        for _ in range(pieces):
            p = bf16(left)[1]
            h, left = h + p, left - p
        y = np.einsum("tr,tnr->tn", h, b[ids])
        off = np.abs(y - want) > np.abs(want) * 2.0 ** -24
        assert not off.any() if pieces == 3 else off.mean() > 0.9
        assert np.all(np.abs(y - want) <= tol)
