"""CPU: what BoundLayer takes and refuses for a layer on 8-bit pages (no kernel runs here)."""
from __future__ import annotations

from types import SimpleNamespace

import pytest
import torch


@pytest.fixture(scope="module")
def K():
    from query_aware_sparse_block_gb300.build import build_library
    build_library()
    from query_aware_sparse_block_gb300 import kvsel
    kvsel.lib()
    return kvsel


def _layer(K, batch=3, hkv=2, d=64, cache_of=None, **kw):
    from query_aware_sparse_block_gb300.runtime import BoundLayer, SparseDecoder
    dec = SparseDecoder(batch, 4, hkv, d, 16, 8, device="cpu")
    desc = K.kvsel_q8_cache(K.KVSEL_KV_PAGED_E4M3, 16, 4, 16)
    q8 = SimpleNamespace(p=dec.p if cache_of is None else K.problem(*cache_of), desc=desc, kv=K.kv_paged_q8(desc))
    t = torch.zeros(1, dtype=torch.bfloat16)
    return BoundLayer(dec, t, None, None, t, None, dec.out, dec.lse, q8=q8, **kw)


def test_rows_of_a_projection_keep_their_strides(K):
    qkv = torch.zeros((3, 8, 64), dtype=torch.bfloat16)
    layer = _layer(K, new_k=qkv[:, 4:6], new_v=torch.zeros((3, 2, 64), dtype=torch.bfloat16))
    assert (layer.k_stride, layer.v_stride) == (512, 128)
    layer = _layer(K)
    assert (layer.k_stride, layer.v_stride) == (128, 128)
    layer = _layer(K, new_k=torch.zeros((3, 128), dtype=torch.bfloat16), new_v=torch.zeros((5, 2, 64), dtype=torch.bfloat16))
    assert (layer.k_stride, layer.v_stride) == (128, 128)                # contiguous rows of any shape, and more of them
    layer = _layer(K, new_k=torch.zeros((5, 8, 64), dtype=torch.bfloat16)[:, :2])
    assert layer.k_stride == 512


@pytest.mark.parametrize("bad,error", [
    (torch.zeros((3, 2, 64)), TypeError),
    (torch.zeros((2, 2, 64), dtype=torch.bfloat16), ValueError),
    (torch.zeros((3, 256), dtype=torch.bfloat16)[:, :128], ValueError),
    (torch.zeros((3, 2, 128), dtype=torch.bfloat16)[..., ::2], ValueError),
    (torch.zeros((2, 3, 64), dtype=torch.bfloat16).transpose(0, 1), ValueError),
], ids=["fp32", "two rows", "flat", "every second channel", "heads apart"])
@pytest.mark.parametrize("which", ["new_k", "new_v"])
def test_rows_that_cannot_be_read_are_refused(K, which, bad, error):
    with pytest.raises(error, match=which):
        _layer(K, **{which: bad})


@pytest.mark.parametrize("field,cache_of", [("batch", (2, 4, 2, 64, 16, 8)), ("n_kvheads", (3, 4, 4, 64, 16, 8)),
                                            ("head_dim", (3, 4, 2, 128, 16, 8)), ("block_size", (3, 4, 2, 64, 32, 8)),
                                            ("max_blocks", (3, 4, 2, 64, 16, 4))])
def test_a_cache_of_another_shape_is_refused(K, field, cache_of):
    """Its pages or its table would be read and written out of range."""
    with pytest.raises(ValueError, match=field):
        _layer(K, cache_of=cache_of)


@pytest.mark.parametrize("cache_of", [(3, 16, 2, 64, 16, 8), (7, 4, 2, 64, 16, 8)], ids=["query heads", "more sequences"])
def test_a_cache_that_the_layer_stays_inside_is_taken(K, cache_of):
    _layer(K, cache_of=cache_of)
