"""The token mixers as a decoder's layer calls them: the fused QKV projection with its rotation and output gate, the
append of its keys and values, and the attention over the cache with that gate, a prompt and single tokens after it."""
import numpy as np
import pytest
import torch

import gemm_affine_u4_amd as qmm
import synth
from oracle import mix_oracle as mix
from tests.gpu_util import Guarded, bf16_bits_to_f64, dev
from tests.mix_util import attention_check

pytestmark = pytest.mark.gpu

GATED = synth.RopeShape("gated QKV + RoPE (hidden 512, 3 q heads x 256 with gate, 1 kv head, rotary 64)", 512, 3, 1, 256,
                        True, 64, 1.0e7)
PLAIN = synth.RopeShape("QKV + RoPE (hidden 1024, 6 q / 2 kv heads x 128, full rotary)", 1024, 6, 2, 128, False, 128, 1.0e4)


@pytest.mark.parametrize("sh", [GATED, PLAIN], ids=["gated", "plain"])
def test_projection_append_attention(sh):
    """The projections' own tests are elsewhere: the expected cache and outputs start from their bf16 results."""
    rng = np.random.default_rng(70)
    n_q, n_kv, hd, page = sh.n_q, sh.n_kv, sh.head_dim, 16
    w = synth.gen_weight(synth.CFG_TEST, 6, synth.PROJ_QKV, sh.rows, sh.K)
    weight = [dev(a) for a in (w.codes, w.scales, w.biases)]
    tab = dev(synth.gen_rope_table(4096, sh.rot, sh.base))
    c = mix.Cache(9, n_kv, page, hd, rng)
    g = qmm.KV4Cache(*[dev(a) for a in c.arrays()])
    table = rng.permutation(9)[:7].astype(np.int32)
    done, scale = 0, None
    for step, n in enumerate((45, 1, 1, 3, 40)):
        x = dev(synth.gen_x(synth.CFG_TEST, 6, step, n, sh.K))
        pos = np.arange(done, done + n)
        slots = (table[pos // page] * page + pos % page).astype(np.int32)
        outs = [Guarded((n, h, hd), False) for h in (n_q, n_kv, n_kv, n_q)]
        q, k, v, gate = (o.t for o in outs)
        qmm.qmm_fused_qkv_rope(x, *weight, q, k, v, dev(pos.astype(np.int32)), tab, sh.rot, gate=gate if sh.q_gate else None)
        qmm.qmm_kv4_append(g, k, v, dev(slots))
        done += n
        qv, kv, vv = (bf16_bits_to_f64(o.values()) for o in outs[:3])
        gv = bf16_bits_to_f64(outs[3].values()) if sh.q_gate else None
        if scale is None:  # scores of a few units, as a trained model's
            scale = float(np.float32(6 / np.abs(np.einsum("ihgd,jhd->ihgj", qv.reshape(n, n_kv, -1, hd), kv)).max()))
        out = Guarded((n, n_q, hd), False)
        ws = torch.full((qmm.qmm_kv4_attn_workspace_bytes(n, 1, n, n_q, n_kv, hd, len(table) * page),), 0xFF,
                        dtype=torch.uint8, device="cuda")
        qmm.qmm_kv4_attn(q, g, dev(table[None]), dev(np.array([done], np.int32)), out.t, ws,
                         q_start=dev(np.array([0, n], np.int32)), max_q=n, scale=scale, gate=gate if sh.q_gate else None)
        torch.cuda.synchronize()
        c.put_rows(slots, kv.astype(np.float32), vv.astype(np.float32))
        for a, b, dt in zip(c.arrays(), g.tensors, (np.uint32, np.uint32, np.uint16, np.uint32)):
            assert np.array_equal(a, b.cpu().numpy().view(dt))
        few = n * n_q // n_kv <= (64 if hd == 256 else 128)
        ref = mix.attention_spread(qv, c, table, done, n, scale, few, gate=gv)
        attention_check(bf16_bits_to_f64(out.values()), *ref, f"{n} tokens, {done} keys")
