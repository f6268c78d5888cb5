"""CPU: the decode workspace's sizes by the kinds that are attended."""
from __future__ import annotations

import ctypes

import pytest


@pytest.fixture(scope="module")
def K():
    from query_aware_sparse_block_gb300.build import build_library
    build_library()
    from query_aware_sparse_block_gb300 import kvsel
    kvsel.lib()
    return kvsel


def _bytes(p, tokens, warps):
    """States of (256 CTAs + segments) x warps, and 8 bytes a segment; a tile holds 64 rows of as many heads as divide."""
    h = min(p.n_kvheads, 64 // tokens)
    while h > 1 and p.n_kvheads % h:
        h -= 1
    segs = p.batch * (p.n_kvheads // h)
    return -(-segs * 8 // 256) * 256 + (256 + segs) * warps * (p.n_qheads // p.n_kvheads) * (p.head_dim + 4) * 4


@pytest.mark.parametrize("shape,warps", [((16, 32, 8, 128, 32, 64), 12), ((256, 8, 8, 64, 16, 64), 12),
                                         ((4096, 32, 2, 128, 64, 4), 8), ((4096, 32, 2, 64, 64, 4), 12),
                                         ((3, 12, 4, 64, 16, 8), 12), ((2, 5, 1, 128, 16, 8), 12)])
def test_bf16_callers_reserve_for_bf16_alone(K, shape, warps):
    p = K.problem(*shape)
    bf16 = _bytes(p, p.block_size, 8)
    q8 = _bytes(p, max(32, p.block_size), warps)
    assert K.kvsel_workspace_size(p, K.KVSEL_WS_SPARSE_DECODE_BF16) == bf16
    assert K.kvsel_workspace_size(p, K.KVSEL_WS_SPARSE_DECODE) == max(bf16, q8)
    from query_aware_sparse_block_gb300.runtime import SparseDecoder
    if p.batch < 1000:
        dec = SparseDecoder(*shape, device="cpu")
        assert dec.ws_decode.numel() == bf16 and dec.ws_decode_q8 is None
        paged, cache = K.kvsel_kv_src(), K.kvsel_kv_src()
        cache.kind = K.KVSEL_KV_PAGED_INT8
        assert dec.decode_workspace(paged) is dec.ws_decode
        assert dec.decode_workspace(cache).numel() == max(bf16, q8) and dec.decode_workspace(cache) is dec.ws_decode_q8


def test_each_kind_takes_its_own_size_and_no_less(K):
    p = K.problem(16, 32, 8, 128, 32, 64)
    small, large = (K.kvsel_workspace_size(p, w) for w in (K.KVSEL_WS_SPARSE_DECODE_BF16, K.KVSEL_WS_SPARSE_DECODE))
    assert 0 < small < large

    def code(kind, size):
        src = K.kvsel_kv_src()                                           # no pages: refused before any launch
        src.kind, src.block_table, src.n_pages = kind, 16, 4
        return K.lib().kvsel_sparse_decode(ctypes.byref(p), 16, ctypes.byref(src), 16, 16, 16, None, None, None, None,
                                           0.125, 16, None, 16, 16, size, None)
    enough = (K.KVSEL_ERR_INVALID_ARG, K.KVSEL_ERR_CUDA)
    assert code(K.KVSEL_KV_PAGED, small) in enough and code(K.KVSEL_KV_PAGED, small - 1) == K.KVSEL_ERR_WORKSPACE
    for kind in (K.KVSEL_KV_PAGED_E4M3, K.KVSEL_KV_PAGED_INT8):
        assert code(kind, large) in enough and code(kind, large - 1) == K.KVSEL_ERR_WORKSPACE
