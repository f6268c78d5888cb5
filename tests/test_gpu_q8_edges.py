"""GPU: the 8-bit KV pages where the arithmetic's range and order show: tails of
small weights beside peaks, sums that round, strided rows of a bound layer."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import _q8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from query_aware_sparse_block_gb300.build import build_library
    build_library()
    from query_aware_sparse_block_gb300 import kvsel
    kvsel.lib()
    torch.cuda.set_device(0)
    return kvsel


@pytest.fixture(autouse=True)
def _no_device_error(K):
    K.kvsel_get_error()
    yield
    assert K.kvsel_get_error() == 0, "a kernel latched a device error"


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("hq", [4, 12])
@pytest.mark.parametrize("fmt,d,B", [("e4m3", 128, 32), ("int8", 64, 16), ("e4m3", 64, 64)])
@pytest.mark.parametrize("peak", ["weight", "value"])
def test_a_tail_beside_peaks_keeps_its_part_of_every_channel(K, peak, fmt, d, B, hq):
    """4096 tokens, every 16th a peak whose V row is 0 but in channel 0: the other channels are the tail's alone, whose
    weights (peak "weight"), or weights against the peaks' V factors (peak "value"), are 2^-22 to 2^-30 of the peaks'."""
    from query_aware_sparse_block_gb300.runtime import Q8Cache, SparseDecoder
    T, mb = 4096, 4096 // B
    dec = SparseDecoder(1, hq, 1, d, B, mb, device="cuda:0")
    g = torch.Generator().manual_seed(d + B + hq)
    cache = Q8Cache(dec, fmt, torch.randperm(mb, generator=g).view(1, mb).to(torch.int32).cuda(), n_pages=mb)
    top = torch.zeros(T, dtype=torch.bool)
    top[::16] = True
    fall = 22 + 8 * torch.rand(T, generator=g)                           # log2 of a peak over the token
    k, v = torch.zeros((T, 1, d)), torch.randn((T, 1, d), generator=g).abs()
    v[top] = 0
    v[top, 0, 0] = 1.0
    if peak == "weight":
        k[:, 0, 0] = torch.where(top, 0.0, -fall * float(np.log(2)) / 4)  # the score is 4 k_0
    else:
        v *= torch.where(top, 1.0, 2.0 ** -fall)[:, None, None]
    q = torch.zeros((1, hq, d))
    q[..., 0] = 4 / dec.scale
    k, v, q = (x.to(torch.bfloat16).cuda() for x in (k, v, q))
    cache.write(_i32([0, T]), _i32([0]), k, v)
    dec.n_sel[0] = mb
    dec.sel_idx[0] = torch.arange(mb, dtype=torch.int32)
    dec.attend(q, cache.kv, _i32([T]))
    torch.cuda.synchronize()
    x = _q8.values(cache.pages.cpu().numpy(), B, d, fmt)
    ks, vs = (np.concatenate([x[n, 0, w] for n in cache.block_table[0].tolist()]) for w in (0, 1))
    qd = q[0].double().cpu().numpy()
    ref, z, reach = _q8.attend(qd, ks, vs, dec.scale)
    p = np.exp(qd @ ks.T * dec.scale - z[:, None])                       # [hq][T]
    # A channel's sum is off by the relative error of a weight and of the sums (as _q8.tolerances counts them, the
    # weight's own rounding 2^-22 of it), and by the weights' smallest step: 2^-40 of the largest weight times V
    # factor in a state, times a code. A row's largest code is at least half the format's largest (e4m3: 224 of 448;
    # int8: 64 of 127), so step times code is at most 2^-40 * 2 of the largest weight times value.
    w = (d + 4) * 2.0 ** -23 * reach + 2.0 ** -22
    rel = 2 * w + 2 * (T / 16 + 32) * 2.0 ** -23 + 2.0 ** -22
    step = T * 2.0 ** -39 * (p * np.abs(vs).max(-1)).max(-1)
    bound = (p @ np.abs(vs)) * rel[:, None] + step[:, None]
    got = dec.out[0].double().cpu().numpy()
    # the bound tells the tail from nothing: every channel but the peaks' is far above it
    assert (np.median(np.abs(ref[:, 1:]), axis=1) > 100 * np.median(bound[:, 1:], axis=1)).all()
    assert (np.abs(got - ref) <= bound).all(), (np.abs(got - ref) / bound).max()
    assert (np.abs(dec.lse[0].double().cpu().numpy() - z) <= rel + 2.0 ** -23 * np.abs(z)).all()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d,B", [(64, 16), (64, 64), (128, 32)])
def test_summaries_do_not_depend_on_how_a_block_was_split_into_calls(K, fmt, d, B):
    """Keys of very different sizes, the large ones in pairs that cancel, so that the fp32 sum is inexact and its order
    shows: a block written at once, in odd chunks and a row at a time."""
    from query_aware_sparse_block_gb300.runtime import Q8Cache, SparseDecoder
    batch, H, mb = 2, 2, 3
    T = mb * B
    dec = SparseDecoder(batch, H, H, d, B, mb, device="cuda:0")
    table = torch.arange(batch * mb, dtype=torch.int32).view(batch, mb).cuda()
    g = torch.Generator().manual_seed(d + B)
    k = torch.randn((batch, T, H, d), generator=g)
    k *= 2.0 ** torch.randint(0, 25, (batch, T, 1, 1), generator=g)
    order = torch.stack([n * B + torch.randperm(B, generator=g) for n in range(mb)]).view(-1)
    k[:, order[1::2]] = -k[:, order[::2]] * (1 + 2.0 ** -6)               # nearly: its code is another one at times
    k = k.to(torch.bfloat16).cuda()
    got = []
    for sizes in ([T], [7, B, 1, 2 * B], [5, 3, 11], [1]):
        cache = Q8Cache(dec, fmt, table, n_pages=batch * mb)
        summ = torch.zeros((batch, mb, H, d), dtype=torch.bfloat16, device="cuda")
        at, i = 0, 0
        while at < T:
            n = min(sizes[i % len(sizes)], T - at)
            x = k[:, at:at + n].reshape(batch * n, H, d)
            cache.write(_i32([0, n, 2 * n]), _i32([at, at]), x, x, summ)
            at, i = at + n, i + 1
        torch.cuda.synchronize()
        got.append((cache.pages, summ))
    assert torch.isfinite(got[0][1]).all() and (got[0][1] != 0).any()
    for pages, summ in got[1:]:
        assert torch.equal(pages, got[0][0])
        assert torch.equal(summ, got[0][1])


@pytest.mark.parametrize("start,first", [([0, 100, 50, 60], [15, 0, 0]), ([0, 40, 20, 90], [3, 0, 9]),
                                         ([90, 100, 0, 80], [0, 1, 16])])
def test_a_row_start_that_decreases_between_good_sequences(K, start, first):
    """Latched; rows of the good sequences may be left out, but a handled row is right and nothing else is touched."""
    from query_aware_sparse_block_gb300.runtime import Q8Cache, SparseDecoder
    batch, B, d, H, mb, fmt = 3, 16, 64, 2, 8, "e4m3"
    dec = SparseDecoder(batch, H, H, d, B, mb, device="cuda:0")
    table = torch.arange(batch * mb, dtype=torch.int32).view(batch, mb)
    cache = Q8Cache(dec, fmt, table.cuda(), n_pages=batch * mb + 2)
    g = torch.Generator().manual_seed(3)
    cache.pages.copy_(torch.randint(0, 120, cache.pages.shape, generator=g, dtype=torch.uint8))
    before = cache.pages.cpu().numpy()
    k, v = _q8.rows(g, (100, H, d)).cuda(), _q8.rows(g, (100, H, d)).cuda()
    good = [b for b in range(batch) if start[b + 1] >= start[b]]
    want = before.copy()
    for b in good:
        one, _ = _q8.write(before, table[b:b + 1].numpy(), [start[b], start[b + 1]], first[b:b + 1],
                           k.double().cpu().numpy(), v.double().cpu().numpy(), B, fmt, mb)
        mine = table[b].numpy()
        want[mine] = one[mine]
    cache.write(_i32(start), _i32(first), k, v)
    assert K.kvsel_get_error() == K.KVSEL_ERR_BOUNDS
    got = cache.pages.cpu().numpy()
    gc, gs = _q8.split(got, B, d)                                        # a row's codes and its scale byte
    wc, ws = _q8.split(want, B, d)
    bc, bs = _q8.split(before, B, d)
    new = ((gc == wc).all(-1) & (gs == ws))
    old = ((gc == bc).all(-1) & (gs == bs))
    assert (new | old).all()
    # read back: a row is what the page holds, or as it was
    kb, vb = (torch.full_like(k, 3.0) for _ in range(2))
    cache.read(_i32(start), _i32(first), kb, vb)
    assert K.kvsel_get_error() == K.KVSEL_ERR_BOUNDS
    x = _q8.values(got, B, d, fmt)
    for r in range(100):
        at = [(b, first[b] + r - start[b]) for b in good if start[b] <= r < start[b + 1]]
        for which, y in enumerate((kb, vb)) if len(at) < 2 else ():      # a row that two sequences claim is theirs in parts
            row = y[r].double().cpu().numpy()
            may = [x[table[b, pos // B], :, which, pos % B] for b, pos in at]
            assert (row == 3).all() or any(np.array_equal(row, m) for m in may), r


def test_bound_layer_appends_rows_of_a_projection(K):
    """new_k and new_v as slices of one projection's rows, of different strides, and a step's own pointers."""
    import ctypes
    from query_aware_sparse_block_gb300.runtime import BoundLayer, Q8Cache, SparseDecoder
    batch, hq, hkv, d, B, mb = 3, 4, 2, 64, 16, 4
    dec = SparseDecoder(batch, hq, hkv, d, B, mb, device="cuda:0")
    table = torch.arange(batch * mb, dtype=torch.int32).view(batch, mb).cuda()
    g = torch.Generator().manual_seed(8)
    qkv, other = (_q8.rows(g, (batch, hq + 2 * hkv, d)).cuda() for _ in range(2))
    v = _q8.rows(g, (batch, hkv, d)).cuda()
    pos, one = _i32([5, 17, 0]), _i32(range(batch + 1))
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)

    def fresh():
        return Q8Cache(dec, "int8", table, n_pages=batch * mb), torch.zeros((batch, mb, hkv, d), dtype=torch.bfloat16,
                                                                            device="cuda")
    for k, given in ((qkv[:, hq:hq + hkv], None), (qkv[:, hq:hq + hkv], other[:, hq:hq + hkv])):
        want, ws = fresh()
        want.write(one, pos, (k if given is None else given).contiguous(), v, ws)
        cache, summ = fresh()
        layer = BoundLayer(dec, qkv, None, None, summ, None, dec.out, dec.lse, new_k=k, new_v=v, q8=cache)
        layer.append(ptr(pos), s, None if given is None else ptr(given))
        torch.cuda.synchronize()
        assert (cache.pages != 0).any() and torch.equal(cache.pages, want.pages) and torch.equal(summ, ws)


@pytest.mark.parametrize("fmt,batch,hq,hkv,d,B,most", [("e4m3", 25, 32, 32, 128, 64, 10), ("int8", 3, 8, 8, 128, 64, 600),
                                                       ("int8", 61, 28, 4, 64, 16, 40), ("e4m3", 5, 32, 2, 128, 32, 500)])
def test_ragged_decode_over_the_whole_grid(K, fmt, batch, hq, hkv, d, B, most):
    """Segments of unequal length over every CTA: CTAs of one segment, which join their states, CTAs of several, rings
    that pass over a segment without a tile of theirs, some sequences empty. The pages are random codes."""
    from query_aware_sparse_block_gb300.runtime import Q8Cache, SparseDecoder
    g = torch.Generator().manual_seed(batch + most)
    lens = torch.randint(0, most * B + 1, (batch,), generator=g)
    lens[0], lens[-1] = most * B, 0
    mb = most + 1
    dec = SparseDecoder(batch, hq, hkv, d, B, mb, device="cuda:0")
    table = torch.randperm(batch * mb, generator=g).view(batch, mb)
    cache = Q8Cache(dec, fmt, table.to(torch.int32).cuda(), n_pages=batch * mb)
    codes, byte = cache.pages[..., :2 * B * d], cache.pages[..., 2 * B * d:]
    c = torch.randint(0, 256, codes.shape, generator=g, dtype=torch.uint8)
    if fmt == "e4m3":
        c[(c & 127) > 0x70] = 0x30                                        # up to 128; no NaN
    codes.copy_(c)
    byte.copy_(torch.randint(118, 122, byte.shape, generator=g, dtype=torch.uint8))
    q = torch.randn((batch, hq, d), generator=g).to(torch.bfloat16).cuda()
    dec.dense_flag.fill_(1)
    dec.attend(q, cache.kv, lens.to(torch.int32).cuda())
    torch.cuda.synchronize()
    values = torch.from_numpy(_q8.code_values(fmt)).cuda()
    at = torch.from_numpy(_q8.chunk_index(B, d)).cuda()
    G = hq // hkv
    for b, T in enumerate(lens.tolist()):
        if T == 0:
            assert (dec.out[b] == 0).all() and (dec.lse[b] == -float("inf")).all()
            continue
        raw = cache.pages[table[b, :-(-T // B)].cuda()]
        kv = []
        for w in (0, 1):
            x = values[raw[..., w * B * d:(w + 1) * B * d].long()][..., at]           # [n][H][B][d]
            f = 2.0 ** (raw[..., 2 * B * d + w * B:2 * B * d + (w + 1) * B].double() - 127)
            kv.append((x * f[..., None]).transpose(0, 1).reshape(hkv, -1, d)[:, :T])
        k, v = kv
        qd = q[b].double().view(hkv, G, d)
        s = qd @ k.transpose(-1, -2) * dec.scale
        z = torch.logsumexp(s, -1)
        ref = torch.exp(s - z[..., None]) @ v
        reach = (qd.abs() @ k.abs().transpose(-1, -2) * dec.scale).amax(-1)
        t_out, t_lse = _q8.tolerances(reach, T, v.abs().amax((1, 2))[:, None], d)
        assert ((dec.out[b].double().view(hkv, G, d) - ref).abs().amax(-1) <= t_out).all(), b
        assert ((dec.lse[b].double().view(hkv, G) - z).abs() <= t_lse + 2.0 ** -23 * z.abs()).all(), b


def test_a_cache_of_more_rows_than_int32_counts_is_attended(K):
    """A pool of 2^31 rows and more (140 GB at d = 64): the descriptor names that many pages, the table only the first."""
    from query_aware_sparse_block_gb300.runtime import Q8Cache, SparseDecoder
    H, d, B, mb = 2, 64, 16, 4
    dec = SparseDecoder(1, H, H, d, B, mb, device="cuda:0")
    cache = Q8Cache(dec, "int8", torch.arange(mb, dtype=torch.int32).view(1, mb).cuda(), n_pages=mb)
    g = torch.Generator().manual_seed(2)
    k, v = (_q8.rows(g, (60, H, d)).cuda() for _ in range(2))
    cache.write(_i32([0, 60]), _i32([0]), k, v)
    q = torch.randn((1, H, d), generator=g).to(torch.bfloat16).cuda()
    dec.n_sel[0], dec.sel_idx[0] = mb, torch.arange(mb, dtype=torch.int32)
    dec.attend(q, cache.kv, _i32([60]))
    want = dec.out.clone()
    cache.kv.n_pages = (1 << 31) // (H * 2 * B) + 1
    dec.attend(q, cache.kv, _i32([60]))
    torch.cuda.synchronize()
    assert torch.isfinite(want).all() and torch.equal(dec.out, want)
    cache.kv.n_pages = (1 << 31) // H
    with pytest.raises(K.KvselError) as e:
        dec.attend(q, cache.kv, _i32([60]))
    assert e.value.code == K.KVSEL_ERR_UNSUPPORTED
