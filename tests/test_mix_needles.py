"""Attention over the 4-bit cache with inputs in which every key's place shows (tests/mix_util.py): a lost split, a
page-window step that is skipped, a wrong weight in a join, and lengths, windows and causal ends that are off by one
exceed what roundings explain.  The mistakes themselves are planted in the oracle, without a GPU."""
import numpy as np
import pytest
import torch

import gemm_affine_u4_amd as qmm
from oracle import mix_oracle as mix
from tests.gpu_util import Guarded, bf16_bits_to_f64, dev
from tests.mix_util import attention_check, needles

# n_q, n_kv, hd, page, kv_len, sequences, queries each, window
FEW = [(16, 2, 128, 32, 4100, 6, 1, 0), (8, 1, 64, 16, 9001, 10, 1, 0), (6, 1, 256, 64, 4097, 8, 1, 0),
       (8, 1, 128, 16, 20011, 1, 8, 0), (8, 2, 128, 128, 3000, 3, 5, 700), (5, 1, 128, 32, 290, 4, 2, 0),
       (12, 2, 64, 32, 131, 3, 1, 33)]
PROMPTS = [(5, 1, 128, 32, 1300, 1, 30, 0), (8, 2, 64, 16, 900, 2, 34, 0), (4, 1, 256, 64, 2600, 1, 20, 0),
           (3, 1, 128, 16, 5000, 1, 45, 0), (4, 1, 128, 32, 700, 1, 60, 150), (3, 1, 256, 16, 400, 2, 40, 64)]
# of the same kinds, smaller
PLANTED = [(8, 1, 128, 32, 1500, 5, 1, 0), (8, 1, 64, 16, 2001, 3, 2, 0), (6, 1, 256, 64, 1000, 4, 1, 0),
           (4, 1, 128, 128, 900, 2, 4, 300), (12, 2, 64, 32, 131, 3, 1, 33)]
PLANTED_PROMPTS = [(4, 1, 128, 32, 500, 1, 34, 0), (3, 1, 256, 16, 300, 1, 30, 64)]


def expected(case, c, table, q, **wrong):
    n_q, n_kv, hd, page, kv, seqs, n, window = case
    args = dict(few=case not in PROMPTS + PLANTED_PROMPTS, window=window)
    args.update(wrong)
    kv = args.pop("kv", kv)
    return [mix.attention_spread(q[b], c, table, kv, n, hd ** -0.5, **args) for b in range(seqs)]


def refused(case, c, table, q, right, **wrong):
    """Whether the check refuses the output of a planted mistake."""
    try:
        for (o, _, _), r in zip(expected(case, c, table, q, bounds=False, **wrong), right):
            attention_check(o, *r, "planted", quiet=True)
    except AssertionError:
        return True
    return False


@pytest.mark.parametrize("case", PLANTED + PLANTED_PROMPTS, ids=str)
def test_planted_mistakes_are_refused(case):
    n_q, n_kv, hd, page, kv, seqs, n, window = case
    c, table, _, q = needles(np.random.default_rng(sum(case)), n_q, n_kv, hd, page, kv, seqs, n, window)
    right = expected(case, c, table, q)
    assert not refused(case, c, table, q, right)
    rounded = [(o * (1 + 2.0 ** -8), s, f) for o, s, f in right]  # the output's own rounding passes
    for (o, _, _), r in zip(rounded, right):
        attention_check(o, *r, "rounded", quiet=True)
    rows = seqs * n * n_q // n_kv
    part = max(32, -(-kv // rows)) if not window else max(32, -(-min(kv, window + n) // rows))
    first = max(0, kv - n + 1 - window) if window else 0
    for at in np.linspace(first, kv - part, 7).astype(int):  # a stretch of keys is lost: as long as the needles are apart
        assert refused(case, c, table, q, right, hide=lambda t: (t >= at) & (t < at + 2 * part)), at
    mid = (first + kv) // 2
    assert refused(case, c, table, q, right, weight=lambda t: np.where(t < mid, 1.0, 1.1))  # parts joined wrongly
    assert refused(case, c, table, q, right, hide=lambda t: t == kv - 1)
    assert refused(case, c, table, q, right, kv=kv - 1)
    assert refused(case, c, table, q, right, kv=kv + 1)  # every query sees a key too many
    if window:
        assert refused(case, c, table, q, right, window=window - 1)
        assert refused(case, c, table, q, right, window=window + 1)
    zero = [np.zeros_like(o) for o, _, _ in right]
    with pytest.raises(AssertionError):
        attention_check(zero[0], *right[0], "zeros", quiet=True)


@pytest.mark.gpu
@pytest.mark.parametrize("case", FEW + PROMPTS, ids=str)
def test_attention_finds_every_key(case):
    n_q, n_kv, hd, page, kv, seqs, n, window = case
    gated = (FEW + PROMPTS).index(case) % 3 == 2
    rng = np.random.default_rng(sum(case))
    c, table, bits, q = needles(rng, n_q, n_kv, hd, page, kv, seqs, n, window)
    gate = torch.from_numpy(rng.standard_normal(q.shape)).to(torch.bfloat16) if gated else None
    T = seqs * n
    out = Guarded((T, n_q, hd), False)
    ws = torch.full((qmm.qmm_kv4_attn_workspace_bytes(T, seqs, n, n_q, n_kv, hd, len(table) * page),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    qmm.qmm_kv4_attn(dev(bits.reshape(T, n_q, hd)), qmm.KV4Cache(*[dev(a) for a in c.arrays()]),
                     dev(np.repeat(table[None], seqs, 0)), dev(np.full(seqs, kv, np.int32)), out.t, ws,
                     q_start=dev((n * np.arange(seqs + 1)).astype(np.int32)), max_q=n, window=window,
                     gate=gate.reshape(T, n_q, hd).cuda() if gated else None)
    torch.cuda.synchronize()
    got = bf16_bits_to_f64(out.values()).reshape(seqs, n, n_q, hd)
    for b in range(seqs):
        ref = mix.attention_spread(q[b], c, table, kv, n, hd ** -0.5, case in FEW, window=window,
                                   gate=gate[b].double().numpy() if gated else None)
        attention_check(got[b], *ref, f"sequence {b}")
