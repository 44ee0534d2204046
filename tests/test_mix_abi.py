"""The token mixers' boundary without a GPU: the header's entry points are exported, bad
arguments are refused before anything is enqueued, and the oracle's own pins."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import gemm_affine_u4_amd as qmm
from oracle import mix_oracle as mix

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
S = qmm.STATUS
MB = 1 << 20
A = 1 << 32  # fake device addresses, never dereferenced


def test_header_functions_are_exported():
    text = open(os.path.join(ROOT, "include", "qmm_mix.h")).read()
    names = sorted(set(re.findall(r"^(?:int|size_t)\s+(qmm_\w+)\s*\(", text, re.M)))
    assert names == ["qmm_gdn", "qmm_gdn_workspace_bytes", "qmm_kv4_append", "qmm_kv4_attn",
                     "qmm_kv4_attn_workspace_bytes"]
    out = subprocess.run(["nm", "-D", "--defined-only", qmm.LIB_PATH], capture_output=True, text=True).stdout
    assert set(names) <= set(re.findall(r" T (qmm_\w+)$", out, re.M))


class Kv4Struct(ctypes.Structure):
    """qmm_kv4_cache of the C ABI."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_codes", "k_meta", "v_codes", "v_meta")] + [
        (n, ctypes.c_int64) for n in ("n_pages", "page_size", "n_kv_heads", "head_dim")]


def cache(**kw):
    f = dict(k_codes=A, k_meta=A + 64 * MB, v_codes=A + 128 * MB, v_meta=A + 192 * MB, n_pages=8, page_size=32,
             n_kv_heads=2, head_dim=128)
    f.update(kw)
    return Kv4Struct(*[f[n] for n, _ in Kv4Struct._fields_])


B0 = A + 256 * MB


def append(c=None, **kw):
    f = dict(k=B0, v=B0 + MB, T=4, dt=0, slots=B0 + 2 * MB, positions=B0 + 3 * MB, cos_sin=B0 + 4 * MB, max_pos=64,
             rot=128, q=B0 + 5 * MB, n_q=4, q_out=B0 + 6 * MB, k_held=B0 + 7 * MB, v_held=B0 + 8 * MB)
    f.update(kw)
    c = cache() if c is None else c
    return qmm.load_library().qmm_kv4_append(ctypes.addressof(c) if c else None, *f.values(), None)


def attn(c=None, **kw):
    f = dict(q=B0, T=3, q_start=B0 + MB, kv_lens=B0 + 2 * MB, table=B0 + 3 * MB, B=2, max_pages=4, max_q=2,
             cache=None, n_q=4, scale=0.1, causal=1, window=0, gate=B0 + 4 * MB, ws=B0 + 8 * MB, ws_bytes=64 * MB,
             out=B0 + 5 * MB)
    f.update(kw)
    c = cache() if c is None else c
    f["cache"] = ctypes.addressof(c) if c else None
    return qmm.load_library().qmm_kv4_attn(*f.values(), None)


def gdn(**kw):
    f = dict(q=B0, k=B0 + MB, v=B0 + 2 * MB, g=B0 + 3 * MB, beta=B0 + 4 * MB, T=5, seq_start=B0 + 5 * MB, B=2,
             max_len=4, Hk=2, Hv=4, Dk=128, Dv=128, scale=0.1, l2=1, s_in=B0 + 8 * MB, s_out=B0 + 16 * MB,
             slots=B0 + 6 * MB, n_slots=3, ws=B0 + 64 * MB, ws_bytes=64 * MB, y=B0 + 7 * MB, od=0)
    f.update(kw)
    return qmm.load_library().qmm_gdn(*f.values(), None)


@pytest.mark.parametrize("bad, want", [
    (dict(k_codes=None), "NULL"), (dict(v_meta=None), "NULL"), (dict(head_dim=96), "SHAPE"),
    (dict(head_dim=512), "SHAPE"), (dict(page_size=8), "SHAPE"), (dict(page_size=48), "SHAPE"),
    (dict(page_size=8192), "SHAPE"), (dict(n_pages=0), "SHAPE"), (dict(n_pages=1 << 27), "SHAPE"),
    (dict(n_kv_heads=0), "SHAPE"), (dict(k_codes=A + 8), "ALIGN"), (dict(v_codes=A + 128 * MB + 2), "ALIGN")])
def test_bad_caches(bad, want):
    assert append(cache(**bad)) == S["QMM_ERR_" + want]
    assert attn(cache(**bad)) == S["QMM_ERR_" + want]


@pytest.mark.parametrize("bad, want", [
    (dict(k=None), "NULL"), (dict(slots=None), "NULL"), (dict(positions=None), "NULL"), (dict(q_out=None), "NULL"),
    (dict(cos_sin=None), "NULL"),  # q without a rotation
    (dict(dt=2), "ENUM"), (dict(T=-1), "SHAPE"), (dict(T=(1 << 24) + 1), "SHAPE"), (dict(rot=3), "SHAPE"),
    (dict(rot=130), "SHAPE"), (dict(rot=0), "SHAPE"), (dict(max_pos=0), "SHAPE"), (dict(n_q=0), "SHAPE"),
    (dict(k=B0 + 2), "ALIGN"), (dict(slots=B0 + 2 * MB + 2), "ALIGN"), (dict(v_held=B0 + 8 * MB + 8), "ALIGN"),
    (dict(q_out=B0 + 5 * MB), "ALIAS"), (dict(k_held=B0 + 8 * MB + 256), "ALIAS"), (dict(k=A + 16), "ALIAS")])
def test_append_refuses(bad, want):
    assert append(**bad) == S["QMM_ERR_" + want]


def test_append_of_nothing_is_accepted_without_a_launch():
    assert append(T=0) == S["QMM_OK"]
    assert qmm.load_library().qmm_kv4_append(None, *([None] * 2), 1, 0, None, None, None, 0, 0, None, 0, None, None,
                                             None, None) == S["QMM_ERR_NULL"]


@pytest.mark.parametrize("bad, want", [
    (dict(q=None), "NULL"), (dict(kv_lens=None), "NULL"), (dict(table=None), "NULL"), (dict(ws=None), "NULL"),
    (dict(out=None), "NULL"), (dict(causal=2), "ENUM"), (dict(T=-1), "SHAPE"), (dict(B=0), "SHAPE"),
    (dict(B=65536), "SHAPE"), (dict(max_q=0), "SHAPE"), (dict(max_pages=0), "SHAPE"), (dict(max_pages=1 << 27), "SHAPE"),
    (dict(n_q=3), "SHAPE"), (dict(n_q=1), "SHAPE"), (dict(scale=0.0), "SHAPE"), (dict(scale=-1.0), "SHAPE"),
    (dict(scale=float("nan")), "SHAPE"), (dict(scale=float("inf")), "SHAPE"), (dict(window=-1), "SHAPE"),
    (dict(window=4, causal=0), "SHAPE"), (dict(q_start=None), "SHAPE"),  # T != B
    (dict(max_q=1 << 24), "SHAPE"), (dict(ws_bytes=255), "SHAPE"), (dict(out=B0 + 5 * MB + 8), "ALIGN"),
    (dict(ws=B0 + 8 * MB + 16), "ALIGN"), (dict(out=B0), "ALIAS"), (dict(out=A), "ALIAS"), (dict(ws=B0), "ALIAS")])
def test_attn_refuses(bad, want):
    assert attn(**bad) == S["QMM_ERR_" + want]


def test_attn_of_nothing_is_accepted_without_a_launch():
    assert attn(T=0) == S["QMM_OK"]


@pytest.mark.parametrize("bad, want", [
    (dict(q=None), "NULL"), (dict(beta=None), "NULL"), (dict(s_in=None), "NULL"), (dict(s_out=None), "NULL"),
    (dict(ws=None), "NULL"), (dict(y=None), "NULL"), (dict(od=2), "ENUM"), (dict(l2=2), "ENUM"), (dict(T=-1), "SHAPE"),
    (dict(B=0), "SHAPE"), (dict(max_len=0), "SHAPE"), (dict(Hv=3), "SHAPE"), (dict(Hk=0), "SHAPE"),
    (dict(Dk=96), "SHAPE"), (dict(Dv=32), "SHAPE"), (dict(seq_start=None), "SHAPE"), (dict(n_slots=0), "SHAPE"),
    (dict(slots=None, n_slots=1), "SHAPE"), (dict(scale=float("nan")), "SHAPE"), (dict(ws_bytes=16), "SHAPE"),
    (dict(q=B0 + 2), "ALIGN"), (dict(s_in=B0 + 8 * MB + 4), "ALIGN"), (dict(y=B0), "ALIAS"),
    (dict(s_out=B0 + 8 * MB + 64), "ALIAS"), (dict(y=B0 + 16 * MB), "ALIAS")])
def test_gdn_refuses(bad, want):
    assert gdn(**bad) == S["QMM_ERR_" + want]


def test_workspace_sizes():
    for bad in ((-1, 1, 1, 4, 2, 128, 64), (1, 0, 1, 4, 2, 128, 64), (1, 1, 1, 5, 2, 128, 64), (1, 1, 1, 4, 2, 96, 64),
                (1, 1, 1, 4, 2, 128, 0)):
        assert qmm.qmm_kv4_attn_workspace_bytes(*bad) == 0
    assert qmm.qmm_kv4_attn_workspace_bytes(1, 1, 1, 4, 2, 128, 64) > 0
    for bad in ((-1, 1, 1, 2, 4, 128, 128), (1, 1, 0, 2, 4, 128, 128), (1, 1, 1, 3, 4, 128, 128),
                (1, 1, 1, 2, 4, 80, 128)):
        assert qmm.qmm_gdn_workspace_bytes(*bad) == 0
    assert qmm.qmm_gdn_workspace_bytes(1, 1, 1, 2, 4, 128, 128) > 0


def test_binding_checks_shapes():
    sh = qmm.kv4_cache_shapes(2, 2, 32, 128)
    t = [torch.zeros(sh["k_codes"], dtype=torch.int32), torch.zeros(sh["k_meta"], dtype=torch.int32),
         torch.zeros(sh["v_codes"], dtype=torch.int16), torch.zeros(sh["v_meta"], dtype=torch.int32)]
    with pytest.raises(ValueError, match="device tensor"):
        qmm.KV4Cache(*t)
    with pytest.raises(ValueError, match="k_meta"):
        qmm.KV4Cache(t[0], t[1][:1], t[2], t[3])
    with pytest.raises(ValueError, match="v_codes"):
        qmm.KV4Cache(t[0], t[1], t[2].to(torch.int32), t[3])


# ---- the oracle's pins ---------------------------------------------------------------------

@pytest.mark.parametrize("hd", [64, 128, 256])
def test_key_places_are_a_permutation_that_keeps_groups_in_a_lane_half(hd):
    place = [mix.k_place(w, hd) for w in range(hd // 8)]
    assert sorted(place) == list(range(hd // 8))
    if hd > 64:  # 16 bytes of a lane: two words of one group, then two of the next
        for p in range(0, hd // 8, 4):
            ws = [place.index(p + i) for i in range(4)]
            assert ws[1] == ws[0] + 1 and ws[3] == ws[2] + 1 and ws[2] == ws[0] + 8
            assert ws[0] // 8 == ws[1] // 8


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_cache_round_trip(hd):
    rng = np.random.default_rng(1)
    c = mix.Cache(3, 2, 16, hd)
    rows = rng.standard_normal((48, 2, 2, hd)).astype(np.float32)
    for slot in range(48):
        for h in range(2):
            c.put(slot, h, rows[slot, h, 0], rows[slot, h, 1])
    for h in range(2):
        for got, i in zip(c.get(np.arange(48), h), (0, 1)):
            codes, s, b = mix.quantize_f32(rows[:, h, i])
            assert np.array_equal(got[0], codes) and np.array_equal(got[1], s) and np.array_equal(got[2], b)
            # half a step, the bias' fp16 rounding, and the end of the range that the scale's rounding may miss
            x = rows[:, h, i].astype(np.float64)
            tol = np.repeat(s.astype(np.float64) * (0.5 + 15 * 2.0 ** -11) + np.abs(b.astype(np.float64)) * 2.0 ** -11,
                            64, -1) + 1e-6
            assert np.all(np.abs(mix.dequantize(*got) - x) <= tol)


def test_quantizer_corners():
    x = np.zeros((6, 64), np.float32)
    x[1] = 3.5                       # constant: scale 0
    x[2, 5] = 1e30                   # clamped
    x[3] = np.linspace(0, 15, 64)
    x[4] = -1e30
    x[5] = np.linspace(0, 1e-7, 64)  # below fp16's smallest scale
    c, s, b = mix.quantize_f32(x)
    v = mix.dequantize(c, s, b)
    assert np.all(v[0] == 0) and np.all(v[1] == 3.5) and np.all(v[4] == -57344)
    assert np.all(np.isfinite(v)) and v[2, 5] >= 57000 and np.abs(v).max() < 65504
    assert np.array_equal(c[3], np.rint(x[3]))


def test_attention_oracle_against_definition():
    rng = np.random.default_rng(2)
    c = mix.Cache(4, 1, 16, 64, rng)
    for slot in range(16, 50):
        c.put(slot, 0, rng.standard_normal(64).astype(np.float32), rng.standard_normal(64).astype(np.float32))
    q = rng.standard_normal((3, 2, 64))
    out, _ = mix.attention(q, c, [1, 2, 3], 34, 3, 0.125)
    (kc, ks, kb), (vc, vs, vb) = c.get(np.arange(16, 50), 0)
    k, v = mix.dequantize(kc, ks, kb), mix.dequantize(vc, vs, vb)
    for j in range(3):
        for a in range(2):
            w = np.array([np.exp(0.125 * (k[t] @ q[j, a])) for t in range(32 + j)])
            assert np.allclose(out[j, a], (w[:, None] * v[:32 + j]).sum(0) / w.sum(), rtol=1e-12)
    # a window of one key is that key's value; more queries than keys: the first see nothing
    out, _ = mix.attention(q, c, [1, 2, 3], 34, 3, 0.125, window=1)
    assert np.allclose(out[1], v[32])
    out, _ = mix.attention(q, c, [1], 1, 3, 0.125)
    assert np.all(out[:2] == 0) and np.allclose(out[2], v[0])
    # an absent page is not seen
    a, _ = mix.attention(q[:1], c, [1, -1], 32, 1, 0.125, causal=False)
    b, _ = mix.attention(q[:1], c, [1], 16, 1, 0.125, causal=False)
    assert np.allclose(a, b)


def test_gdn_oracle_closed_forms():
    rng = np.random.default_rng(3)
    q, k = rng.standard_normal((4, 1, 8)), rng.standard_normal((4, 1, 8))
    v = rng.standard_normal((4, 2, 8))
    zero = np.zeros((2, 8, 8))
    g, beta = np.zeros((4, 2)), np.ones((4, 2))
    y, s = mix.gdn(q, k, v, g, beta, zero, 1.0, True)
    for h in range(2):  # full-strength writes: the last key reads its value back
        kn = k[3, 0] / np.sqrt((k[3, 0] ** 2).sum() + 1e-6)
        assert np.allclose(s[h] @ kn, v[3, h], atol=1e-5)
    y, s = mix.gdn(q, k, v, g, np.zeros((4, 2)), zero + 1.0, 1.0, False)  # nothing written
    assert np.allclose(s, 1.0) and np.allclose(y[2], q[2, 0].sum())
    y, s = mix.gdn(q, k, v, np.full((4, 2), -1.0), np.zeros((4, 2)), zero + 1.0, 1.0, False)
    assert np.allclose(s, np.exp(-4.0))
    a, sa = mix.gdn(q[:2], k[:2], v[:2], g[:2] - 0.3, beta[:2] * 0.4, zero, 0.5, True)  # split = whole
    b, sb = mix.gdn(q[2:], k[2:], v[2:], g[2:] - 0.3, beta[2:] * 0.4, sa, 0.5, True)
    y, s = mix.gdn(q, k, v, g - 0.3, beta * 0.4, zero, 0.5, True)
    assert np.allclose(np.concatenate([a, b]), y) and np.allclose(sb, s)
