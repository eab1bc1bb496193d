"""The paged cache on the GPU: writing (16-bit and e4m3), reading back, skipped and out-of-range tokens."""
import math

import pytest
import torch

from tests import _seq as sq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cq():
    import exact_long_context_tcgen05_gb300 as m
    return m


def _problem(new, lengths, hkv, d, page, dtype, seed, behind=0):
    total = sum(new) + behind
    k, v = sq.normal((total, hkv, d), dtype, seed, 2.0), sq.normal((total, hkv, d), dtype, seed + 1)
    _, _, kc, vc, table = sq.make_cache(lengths, hkv, d, page, dtype, seed + 2, fill=0.0)
    cu = torch.tensor(sq.starts(new), dtype=torch.int32, device="cuda")
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    return k, v, kc, vc, table, cu, lens


def _written(cache, x, table, new, lengths, page):
    want = cache.clone()
    at = 0
    for s, n in enumerate(new):
        for i in range(n):
            pos = lengths[s] - n + i
            want[int(table[s, pos // page]), :, pos % page] = x[at + i]
        at += n
    return want


CASES = [([1], [1], 1, 64, 16), ([1, 1, 1], [17, 1, 400], 2, 128, 16), ([5, 0, 40, 7], [5, 9, 333, 64], 3, 64, 32),
         ([130, 1], [300, 129], 8, 128, 64), ([33] * 40, [33 + 7 * i for i in range(40)], 5, 128, 256),
         ([70, 3], [70, 130], 33, 64, 128)]


@pytest.mark.parametrize("new,lengths,hkv,d,page", CASES)
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_write_and_read_16bit(cq, new, lengths, hkv, d, page, dt):
    dtype = sq.DT[dt]
    k, v, kc, vc, table, cu, lens = _problem(new, lengths, hkv, d, page, dtype, 5, behind=3)
    want_k, want_v = _written(kc, k, table, new, lengths, page), _written(vc, v, table, new, lengths, page)
    cq.kv_cache_write(k, v, kc, vc, table, cu, lens)
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)
    out = tuple(torch.full_like(k, 7.0) for _ in range(2))
    cq.kv_cache_read(kc, vc, table, cu, lens, k.shape[0], dtype, out=out)
    n = sum(new)
    for got, x in zip(out, (k, v)):
        assert torch.equal(got[:n], x[:n])
        assert (got[n:] == 7.0).all()  # rows behind the last sequence are left as they were


@pytest.mark.parametrize("new,lengths,hkv,d,page", CASES)
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_write_and_read_e4m3(cq, new, lengths, hkv, d, page, dt):
    dtype = sq.DT[dt]
    k, v, kc, vc, table, cu, lens = _problem(new, lengths, hkv, d, page, dtype, 9)
    # vectors of every size: zeros, one large value, tiny ones, values at the border 448 * 2^e, NaN and infinities
    k[0] = 0
    v[-1] *= 2.0 ** -14
    k[-1, :, 0] = 448.0
    if sum(new) > 4:
        v[1] *= 512.0
        k[2, :, 1], k[2, 0, 2], v[2, :, 3] = math.inf, math.nan, -math.inf
        if dt == "bf16":
            k[3] *= 2.0 ** 100
            v[3] *= 2.0 ** -120
    kq, vq = (torch.zeros(c.shape, dtype=torch.uint8, device="cuda") for c in (kc, vc))
    ks, vs = (torch.zeros(c.shape[:3], dtype=torch.uint8, device="cuda") for c in (kc, vc))
    cq.kv_cache_write(k, v, kq, vq, table, cu, lens, k_scale=ks, v_scale=vs)
    values = []
    for x, codes, scale in ((k, kq, ks), (v, vq, vs)):
        c, e, val = sq.quantise(x)
        nan = torch.isnan(val)
        want_c = _written(torch.zeros_like(codes), torch.where(nan, torch.zeros_like(c), c), table, new, lengths, page)
        want_nan = _written(torch.zeros_like(codes, dtype=torch.bool), nan, table, new, lengths, page)
        assert torch.equal(scale, _written(torch.zeros_like(scale), e, table, new, lengths, page))
        assert torch.equal(torch.where(want_nan, torch.zeros_like(codes), codes), want_c)
        assert ((codes & 0x7f)[want_nan] == 0x7f).all()
        values.append(val)
    got = cq.kv_cache_read(kq, vq, table, cu, lens, k.shape[0], dtype, k_scale=ks, v_scale=vs)
    for g, val in zip(got, values):
        want = val.float().to(dtype)  # code * 2^e is exact in 32 bits, rounded once
        assert torch.equal(torch.isnan(g), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(g, 0.0), torch.nan_to_num(want, 0.0))


def test_skipped_tokens(cq):
    """Positions below zero, beyond the table, and pages outside the cache are skipped; nothing else changes."""
    page, hkv, d, dtype = 16, 2, 64, torch.float16
    kc = torch.zeros(4, hkv, page, d, dtype=dtype, device="cuda")
    vc = torch.zeros_like(kc)
    table = torch.tensor([[0, 99], [1, -5], [2, 3]], dtype=torch.int32, device="cuda")
    new, lens = [20, 17, 40], [20, 17, 36]  # page 99; page -5; a length smaller than the new tokens, and beyond two pages
    k = sq.normal((sum(new), hkv, d), dtype, 3)
    cu = torch.tensor(sq.starts(new), dtype=torch.int32, device="cuda")
    kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cq.kv_cache_write(k, k, kc, vc, table, cu, kv)
    want = torch.zeros_like(kc)
    want[0] = k[0:16].transpose(0, 1)
    want[1] = k[20:36].transpose(0, 1)
    want[2] = k[41:57].transpose(0, 1)  # position 0 is new token 4 of sequence 2
    want[3] = k[57:73].transpose(0, 1)
    assert torch.equal(kc, want) and torch.equal(vc, want)
    got, _ = cq.kv_cache_read(kc, vc, table, cu, kv, sum(new), dtype)
    assert (got[37:41] == 0).all() and (got[73:77] == 0).all()  # positions below zero, and beyond the table
    assert torch.equal(got[41:73], k[41:73])


def test_strides_streams_and_graph(cq):
    """k and v as slices of a fused projection, on a stream that is not the current one, captured and replayed."""
    page, hkv, d, dtype = 16, 4, 128, torch.bfloat16
    new, lengths = [3, 50], [100, 50]
    k0, _, kc, vc, table, cu, lens = _problem(new, lengths, hkv, d, page, dtype, 21)
    fused = sq.normal((53, 3, hkv, d), dtype, 22)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want_k, want_v = (_written(c, fused[:, i], table, new, lengths, page) for c, i in ((kc, 1), (vc, 2)))
    cq.kv_cache_write(fused[:, 1], fused[:, 2], kc, vc, table, cu, lens, stream=side)
    side.synchronize()
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cq.kv_cache_write(fused[:, 1], fused[:, 2], kc, vc, table, cu, lens)
        got = cq.kv_cache_read(kc, vc, table, cu, lens, 53, dtype)
    fused.copy_(sq.normal(fused.shape, dtype, 23))
    kc.zero_()
    graph.replay()
    assert torch.equal(got[0], fused[:, 1]) and torch.equal(got[1], fused[:, 2])


def test_no_tokens(cq):
    kc = torch.zeros(2, 2, 16, 64, dtype=torch.float16, device="cuda")
    z = torch.empty(0, 2, 64, dtype=torch.float16, device="cuda")
    ints = torch.zeros(2, dtype=torch.int32, device="cuda")
    cq.kv_cache_write(z, z, kc, kc.clone(), ints[:1, None], ints, ints[:1])
    k, v = cq.kv_cache_read(kc, kc, ints[:1, None], ints, ints[:1], 0, torch.float16)
    assert k.shape == (0, 2, 64) and v.shape == (0, 2, 64)
