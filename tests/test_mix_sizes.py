"""The sizes that the token mixers take and refuse, without a GPU: nothing here is launched."""
import pytest

import gemm_affine_u4_amd as qmm
from tests.test_mix_abi import B0, MB, S, attn, cache, gdn

LIMIT = (1 << 31) - (1 << 16)  # keys of a page table: key numbers of tiles ahead stay below 2^31


@pytest.mark.parametrize("page", [16, 32, 4096])
def test_tables_near_two_to_the_31_keys_are_refused(page):
    table = dict(table=B0 + 4096 * MB, q_start=None, T=1, B=1, max_q=1)
    for max_pages in (((1 << 31) - 1) // page, LIMIT // page + 1):
        assert attn(cache(page_size=page, n_pages=8), max_pages=max_pages, **table) == S["QMM_ERR_SHAPE"]
        assert qmm.qmm_kv4_attn_workspace_bytes(1, 1, 1, 4, 2, 128, max_pages * page) == 0
    assert qmm.qmm_kv4_attn_workspace_bytes(1, 1, 1, 4, 2, 128, LIMIT) > 0
    assert qmm.qmm_kv4_attn_workspace_bytes(70, 1, 70, 4, 2, 128, LIMIT) > 0


@pytest.mark.parametrize("n_q,n_kv,hd", [(40, 8, 128), (64, 8, 128), (24, 4, 256), (32, 8, 64), (64, 64, 64)])
def test_long_prompts_are_taken(n_q, n_kv, hd):
    """A prompt's blocks hold 128 rows (query x head of a group), and a grid's second dimension 65535 blocks."""
    most = 65535 // n_kv * 128 // (n_q // n_kv)
    for n in (16384, 32768, 131072, most):
        if n <= most:
            assert qmm.qmm_kv4_attn_workspace_bytes(n, 1, n, n_q, n_kv, hd, n) > 0, n
    assert qmm.qmm_kv4_attn_workspace_bytes(most + 1, 1, most + 128, n_q, n_kv, hd, most + 128) == 0


def test_few_rows_of_many_heads_are_taken():
    """Blocks of 16 rows: as many as the heads allow."""
    assert qmm.qmm_kv4_attn_workspace_bytes(128, 1, 128, 1024, 1024, 128, 4096) > 0
    assert qmm.qmm_kv4_attn_workspace_bytes(64, 1, 64, 1024, 1024, 256, 4096) > 0


def test_more_delta_rule_prompts_than_a_launch_has_threads_for_are_refused():
    """The walk of longer sequences takes 512 threads for 32 columns of each head: 2^32 threads a launch."""
    assert qmm.qmm_gdn_workspace_bytes(1 << 20, 65535, 17, 8, 32, 128, 128) > 0
    assert qmm.qmm_gdn_workspace_bytes(1 << 20, 65535, 17, 8, 48, 128, 128) == 0
    assert qmm.qmm_gdn_workspace_bytes(1 << 20, 65535, 16, 8, 48, 128, 128) > 0  # token by token
    assert gdn(T=1 << 20, B=65535, max_len=17, Hk=8, Hv=48, n_slots=1, q=B0 + (1 << 40)) == S["QMM_ERR_SHAPE"]
