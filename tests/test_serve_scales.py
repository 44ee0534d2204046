"""GPU: attention over the paged 8-bit cache where scales are at the ends of their range, and what is stored for keys that
no query sees.  Calls of more than 256 rows per KV head are those of prompts."""
import numpy as np
import pytest
import torch

import gemm_affine_u4_amd as qmm
from tests.gpu_util import dev
from tests.serve_util import bf16, filled, gpu_cache, ints

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
