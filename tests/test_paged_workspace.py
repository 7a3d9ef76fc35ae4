"""The workspace query of the attention over a paged cache (CPU): 0 for every size that the call
itself rejects, however large."""
import ctypes

import pytest

SHAPE = 2
BIG = 2 ** 31 - 1


@pytest.mark.parametrize("B,q_heads,kv_heads,head_dim", [
    (1, BIG, 1, 64), (1, BIG, BIG, 64), (1, BIG - 1, 2, 128), (1, 1 << 25, 1, 64), (1, 1 << 23, 1, 256),
    (BIG, 2, 1, 64), (1 << 16, 1 << 15, 1, 64), (1, 1 << 23, 1 << 23, 64)])
def test_sizes_that_are_rejected(B, q_heads, kv_heads, head_dim):
    import gated_delta_rule_33_gb300 as kda
    from gated_delta_rule_33_gb300.kda import _CacheStruct
    kda.build()
    assert kda.kda_paged_decode_workspace_size(B, q_heads, kv_heads, head_dim) == 0
    P = ctypes.c_void_p(0x900000)
    c = _CacheStruct(0x10000, 0x20000, None, None, 16 * kv_heads * head_dim, kv_heads * head_dim,
                     head_dim, 0, 10, 16, kv_heads, head_dim)
    assert kda.load().kda_paged_decode(P, q_heads * head_dim, ctypes.byref(c), P, 4, P, B, q_heads,
                                       1.0, P, 0, None, P, 1 << 40, None) == SHAPE


@pytest.mark.parametrize("B,q_heads,kv_heads,head_dim", [(1, 1 << 24, 1, 64), (0, 4, 4, 256),
                                                         (BIG, 1, 1, 64), (1, 1 << 23, 1 << 22, 64)])
def test_sizes_that_are_taken(B, q_heads, kv_heads, head_dim):
    import gated_delta_rule_33_gb300 as kda
    kda.build()
    assert kda.kda_paged_decode_workspace_size(B, q_heads, kv_heads, head_dim) > 0
