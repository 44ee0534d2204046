"""The calls of a serving step as a server makes them: the fused QKV projection, the requests' adapters beside it, the
append with its rotation, attention with a window and sinks, the head's projection and the verification of drafts,
after which refused drafts' keys are taken back: two prompts, then rounds of drafted tokens."""
import numpy as np
import pytest
import torch

import gemm_affine_u4_amd as qmm
import synth
from oracle import mix_oracle as mix
from oracle import qmm_oracle as orc
from oracle import serve_oracle as srv
from tests.gpu_util import Guarded, assert_within, bf16_bits_to_f64, dev, dev_weight
from tests.serve_util import angles, bf16, few_rows, gpu_cache, ints

pytestmark = pytest.mark.gpu


def workspace(n):
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("n_q,n_kv,hd,rot,page,probs", [(6, 2, 128, 128, 32, True), (3, 1, 256, 64, 16, False),
                                                        (4, 4, 64, 64, 16, True)])
def test_prompts_then_drafted_tokens(n_q, n_kv, hd, rot, page, probs):
    """Each stage's expected values start from the results of the one before."""
    rng = np.random.default_rng([80, hd])
    K, V, rank, n_ad, window, sinks = 512, 700, 16, 3, 40, 4
    w = synth.gen_weight(synth.CFG_TEST, 7, synth.PROJ_QKV, (n_q + 2 * n_kv) * hd, K)
    head = synth.gen_weight(synth.CFG_TEST, 8, synth.PROJ_QKV, V, n_q * hd)
    weight, head_weight = dev_weight(w), dev_weight(head)
    a = bf16(rng.standard_normal((n_ad, 3 * rank, K)) / np.sqrt(K))
    b = bf16(rng.standard_normal((n_ad, (n_q + 2 * n_kv) * hd, rank)))
    ad_a, ad_b = dev(a[0]), dev(b[0])
    scales = rng.uniform(-1, 1, n_ad).astype(np.float32)
    cs = angles(rot, 512)
    c = srv.Cache(14, n_kv, page, hd, rng)
    g = gpu_cache(c)
    table = rng.permutation(14).reshape(2, 7).astype(np.int32)
    done, scale, kept_any = np.zeros(2, np.int64), None, 0
    for step, counts in enumerate(([44, 17], [3, 2], [1, 4], [0, 3], [2, 0])):
        prompt = step == 0
        q_lens = np.array(counts) + (0 if prompt else 1)  # drafts behind the last token
        T, lens = int(q_lens.sum()), done + q_lens
        starts = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        max_q = int(q_lens.max())
        kv_lens, q_start = dev(lens.astype(np.int32)), dev(starts)

        # the projection, and each request's adapter on its tokens (the second has one in every other step)
        x = synth.gen_x(synth.CFG_TEST, 7, step, T, K)
        outs = [Guarded((T, h * hd), True) for h in (n_q, n_kv, n_kv)]
        y = [o.t for o in outs]
        qmm.qmm_fused_qkv(dev(x), *weight, *y)
        torch.cuda.synchronize()
        base = [o.values().astype(np.float64) for o in outs]
        ids = np.repeat([step % n_ad, -1 if step % 2 else 1], q_lens).astype(np.int32)
        qmm.qmm_lora(dev(x), ad_a, ad_b, dev(ids), y, workspace(qmm.qmm_lora_workspace_bytes(T, K, rank, 3)),
                     scales=dev(scales))
        torch.cuda.synchronize()
        row = 0
        for p, o in enumerate(outs):
            ref, tol = srv.lora(bf16_bits_to_f64(x), a[1][:, p * rank:(p + 1) * rank], b[1][:, row:row + o.t.shape[1]], ids,
                                base[p], scales, 2.0 ** -24)
            assert_within(o.values(), ref, tol, f"step {step}: part {p} with adapters")
            row += o.t.shape[1]
        q, k, v = (o.values().reshape(T, -1, hd) for o in outs)

        # into the cache, rotated
        q_rot = Guarded((T, n_q, hd), False)
        qmm.qmm_kv8_append(g, y[1].view(T, n_kv, hd), y[2].view(T, n_kv, hd), dev(table), kv_lens, q_start=q_start,
                           max_q=max_q, cos_sin=dev(cs), q=y[0].view(T, n_q, hd), q_out=q_rot.t)
        pos = np.concatenate([np.arange(done[i], lens[i]) for i in range(2)])
        kr, qr = mix.rotate_f32(k, cs[pos]), mix.rotate_f32(q, cs[pos])
        for i in range(2):
            c.append(table[i], int(lens[i]), kr[starts[i]:starts[i + 1]], v[starts[i]:starts[i + 1]])
        torch.cuda.synchronize()
        back = srv.Cache(14, n_kv, page, hd)
        for to, t in zip(back.arrays(), g.tensors):
            to[...] = t.cpu().numpy()
        for i in range(2):
            for name, want, got in zip(("k", "v", "k scale", "v scale"), c.live(table[i], int(lens[i])),
                                       back.live(table[i], int(lens[i]))):
                assert np.array_equal(want, got), (step, i, name)
        assert np.array_equal(q_rot.values().reshape(T, n_q, hd), bf16(qr)[0]), f"step {step}: rotated queries"

        # attention
        qv = bf16(qr)[1]
        if scale is None:  # scores of a few units, as a trained model's
            scale = float(np.float32(6 / np.abs(np.einsum("ihgd,jhd->ihgj", qv.reshape(T, n_kv, -1, hd), kr)).max()))
        out = Guarded((T, n_q, hd), False)
        need = qmm.qmm_kv8_attn_workspace_bytes(T, 2, max_q, n_q, n_kv, hd, 7 * page, window, sinks)
        qmm.qmm_kv8_attn(q_rot.t, g, dev(table), kv_lens, out.t, workspace(need), q_start=q_start, max_q=max_q,
                         scale=scale, window=window, sinks=sinks)
        torch.cuda.synchronize()
        o = bf16_bits_to_f64(out.values()).reshape(T, n_q, hd)
        for i in range(2):
            part = slice(starts[i], starts[i + 1])
            ref, tol = srv.attention(qv[part], c, table[i], int(lens[i]), int(q_lens[i]), scale, True, window, sinks,
                                     few=few_rows(max_q * n_q // n_kv))
            assert_within(o[part], ref, tol, f"step {step}: attention of {i}")
        done = lens.copy()
        if prompt:
            continue

        # the head, and the drafts against its probabilities
        logits = torch.empty(T, V, dtype=torch.float32, device="cuda")
        qmm.qmm_linear(out.t.view(T, n_q * hd), *head_weight, logits)
        ref, tol = orc.linear(out.values().reshape(T, n_q * hd), head.codes, head.scales, head.biases, bf16_weights=True)
        assert_within(logits.cpu().numpy(), ref, tol, f"step {step}: head")
        target = torch.softmax(logits * (4 / logits.std()), -1)
        tv = target.cpu().numpy().astype(np.float64)
        start = np.concatenate([[0], np.cumsum(counts)])
        D = int(start[-1])
        rows = np.concatenate([start[i] + i + np.arange(counts[i]) for i in range(2)]).astype(int)
        other = tv[rows] * np.exp(0.3 * rng.standard_normal((D, V)))
        other = (other / other.sum(1, keepdims=True)).astype(np.float32)
        draft = np.array([rng.choice(V, p=z / z.sum()) for z in other.astype(np.float64)], np.int32).reshape(D)
        u = rng.random(T).astype(np.float32)
        tokens, accepted = torch.empty(2, max(counts) + 1, dtype=torch.int32, device="cuda"), ints(0, 0)
        qmm.qmm_spec_verify(dev(draft), target, dev(u), tokens, accepted, workspace(qmm.qmm_spec_verify_workspace_bytes(2, V)),
                            dev(start.astype(np.int32)), draft_probs=dev(other) if probs else None)
        torch.cuda.synchronize()
        want = srv.verify(draft, start, tv, other.astype(np.float64) if probs else None, u, max(counts))
        assert np.array_equal(tokens.cpu().numpy(), want[0]) and np.array_equal(accepted.cpu().numpy(), want[1])
        kept_any += int(want[1].sum())
        done -= np.array(counts) - want[1]  # refused drafts' keys are taken back
    if probs:
        assert kept_any > 0
