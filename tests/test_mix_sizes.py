"""The sizes that the token mixers take and refuse, without a GPU: nothing here is launched."""
import pytest

import gemm_affine_u4_amd as qmm
from tests.test_mix_abi import B0, MB, S, attn, cache

LIMIT = (1 << 31) - (1 << 16)  # keys of a page table: key numbers of tiles ahead stay below 2^31


@pytest.mark.parametrize("page", [16, 32, 4096])
def test_tables_near_two_to_the_31_keys_are_refused(page):
    table = dict(table=B0 + 4096 * MB, q_start=None, T=1, B=1, max_q=1)
    for max_pages in (((1 << 31) - 1) // page, LIMIT // page + 1):
        assert attn(cache(page_size=page, n_pages=8), max_pages=max_pages, **table) == S["QMM_ERR_SHAPE"]
        assert qmm.qmm_kv4_attn_workspace_bytes(1, 1, 1, 4, 2, 128, max_pages * page) == 0
    assert qmm.qmm_kv4_attn_workspace_bytes(1, 1, 1, 4, 2, 128, LIMIT) > 0
    assert qmm.qmm_kv4_attn_workspace_bytes(70, 1, 70, 4, 2, 128, LIMIT) > 0
