"""CPU: a descriptor's pages have to be on the device that a call is launched on (stand-ins for tensors of two GPUs)."""
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


class _On:
    """What the checks look at in a contiguous CUDA tensor."""
    is_cuda = True

    def __init__(self, device, dtype, *shape):
        self.device_index, self.dtype, self.shape = device, dtype, shape
        self.device = f"cuda:{device}"

    def get_device(self):
        return self.device_index

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def element_size(self):
        return 1

    def stride(self):
        return tuple(int(torch.tensor(self.shape[i + 1:]).prod()) for i in range(len(self.shape)))

    def data_ptr(self):
        return 1024


def _stand_ins(K, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    launched = []
    fake = SimpleNamespace(**{n: lambda *a, n=n: launched.append(n) or 0 for n in (
        "kvsel_q8_write", "kvsel_q8_read", "kvsel_sparse_decode", "kvsel_prefix_decode")})
    monkeypatch.setattr(K, "lib", lambda: fake)
    monkeypatch.setattr(K, "_stream", lambda s=None: 0)
    return launched


@pytest.mark.parametrize("device", [0, 1])
def test_8_bit_pages_of_another_device_are_refused(K, monkeypatch, device):
    p = K.problem(2, 8, 4, 64, 16, 8)
    i32, bf, u8, f32 = torch.int32, torch.bfloat16, torch.uint8, torch.float32
    launched = _stand_ins(K, monkeypatch)
    cache = K.q8_cache(K.KVSEL_KV_PAGED_INT8, _On(device, u8, 16, 4, 2080), _On(device, i32, 2, 8))
    rows = _On(0, i32, 3), _On(0, i32, 2), _On(0, bf, 5, 4, 64), _On(0, bf, 5, 4, 64)
    q, out, lse, ws = _On(0, bf, 2, 8, 64), _On(0, f32, 2, 8, 64), _On(0, f32, 2, 8), _On(0, u8, 1 << 20)
    calls = (lambda: K.kvsel_q8_write(p, cache, *rows), lambda: K.kvsel_q8_read(p, cache, *rows),
             lambda: K.kvsel_sparse_decode(p, q, K.kv_paged_q8(cache), rows[1], _On(0, i32, 2, 8), rows[1], out, lse, ws, 0.1))
    for call in calls:
        if device:
            with pytest.raises(ValueError, match="cuda:1"):
                call()
        else:
            call()
    assert len(launched) == (0 if device else 3)


@pytest.mark.parametrize("device", [0, 1])
def test_prefix_pages_of_another_device_are_refused(K, monkeypatch, device):
    p = K.problem(2, 8, 4, 64, 16, 8)
    i32, bf, u8, f32 = torch.int32, torch.bfloat16, torch.uint8, torch.float32
    launched = _stand_ins(K, monkeypatch)
    x = K.prefix(_On(device, bf, 16, 4, 2, 1, 16, 64), _On(device, i32, 1, 4), _On(device, i32, 1), _On(device, i32, 2))
    q, out, lse, ws = _On(0, bf, 2, 8, 64), _On(0, f32, 2, 8, 64), _On(0, f32, 2, 8), _On(0, u8, 1 << 20)
    if device:
        with pytest.raises(ValueError, match="cuda:1"):
            K.kvsel_prefix_decode(p, x, q, out, lse, ws, 0.1)
    else:
        K.kvsel_prefix_decode(p, x, q, out, lse, ws, 0.1)
    assert len(launched) == (0 if device else 1)


def test_a_table_on_another_device_than_the_pages_is_refused(K):
    with pytest.raises(ValueError, match="one device"):
        K.q8_cache(K.KVSEL_KV_PAGED_INT8, _On(0, torch.uint8, 16, 4, 2080), _On(1, torch.int32, 2, 8))
