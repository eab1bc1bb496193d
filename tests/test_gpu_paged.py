"""Attention over the paged cache on the GPU against its definition in 64 bits: single tokens, a few, chunks; grouped
heads; 16-bit and e4m3 pages; ragged lengths; empty rows; what lies in unused slots."""
import math

import pytest
import torch

from tests import _seq as sq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cq():
    import exact_long_context_tcgen05_gb300 as m
    return m


def _call(cq, q, kc, vc, table, new, lengths, causal=True, scales=(None, None), **kw):
    cu = torch.tensor(sq.starts(new), dtype=torch.int32, device="cuda")
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    out, lse = cq.attention_paged(q, kc, vc, table, cu, lens, max(new), max(lengths), causal=causal, k_scale=scales[0],
                                  v_scale=scales[1], return_lse=True, out=out, **kw)
    torch.cuda.synchronize()
    rc, code, _ = cq.cqsa_device_error()
    assert rc == cq.CQSA_OK and code == 0
    return out, lse


def _check(out, lse, q, ks, vs, new, lengths, causal, p_dtype, what, spread=1.0):
    """`spread`: how much larger a value's exponent may be than another's. Probabilities are kept as 2^14 p in fp16,
    relative to the largest exponent, so one below fp16's normal numbers is off by 2^-39 * spread, times values under 32 here."""
    at = 0
    for s, n in enumerate(new):
        if n == 0:
            continue
        ref, rl, mass = sq.attend(q[at:at + n], ks[s], vs[s], lengths[s] - n, causal)
        sq.check_out(out[at:at + n], ref, mass, q.dtype, p_dtype, f"{what} sequence {s}", lengths[s] * spread * 2.0 ** -34)
        sq.check_lse(lse[:, at:at + n], rl, f"{what} sequence {s}")
        at += n
    assert (out[at:] == 7.0).all(), f"{what}: rows behind the last sequence"


CASES = [
    # new tokens, lengths, Hq, Hkv, page
    ([1], [1], 1, 1, 16),
    ([1], [3001], 8, 2, 16),
    ([1, 1, 1, 1, 1], [1, 16, 17, 129, 1000], 8, 2, 32),
    ([1] * 37, [1 + 61 * i for i in range(37)], 4, 1, 64),
    ([1, 0, 1], [5000, 77, 300], 5, 1, 128),
    ([1] * 200, [(i * 37) % 90 + 1 for i in range(200)], 2, 2, 16),   # more sequences than the kernel has threads
    ([2, 2, 1, 3], [2, 200, 64, 127], 8, 2, 256),
    ([4, 4], [900, 64], 32, 4, 16),                                   # 32 rows
    ([3, 1, 5], [3, 1, 700], 7, 1, 16),                               # a group of 7 heads, more than 32 rows
    ([64, 1, 0, 130], [64, 400, 9, 1130], 8, 2, 16),
    ([300], [2300], 4, 4, 64),
    ([257, 128], [257, 129], 6, 2, 32),
    ([70], [70], 64, 1, 16),                                          # one key head for 64
    ([40, 3, 2], [0, 2, 1], 4, 2, 16),                                # sequences shorter than their new tokens: empty rows
    ([1, 1], [0, 40], 4, 2, 16),
]


@pytest.mark.parametrize("new,lengths,hq,hkv,page", CASES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_paged_16bit(cq, new, lengths, hq, hkv, page, d, dt):
    dtype = sq.DT[dt]
    ks, vs, kc, vc, table = sq.make_cache(lengths, hkv, d, page, dtype, 11 + len(new), sharp=1.5)
    q = sq.normal((sum(new) + 2, hq, d), dtype, 3)
    for causal in (True, False):
        out, lse = _call(cq, q, kc, vc, table, new, lengths, causal)
        _check(out, lse, q, ks, vs, new, lengths, causal, dtype, f"causal={causal}")


@pytest.mark.parametrize("new,lengths,hq,hkv,page", CASES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_paged_e4m3(cq, new, lengths, hq, hkv, page, d, dt):
    dtype = sq.DT[dt]
    ks, vs, kc, vc, table = sq.make_cache(lengths, hkv, d, page, torch.float32, 13 + len(new), fill=0.0, sharp=1.5)
    # tokens of very different sizes, as a cache holds them
    (kq, kse, kval), (vq, vse, vval) = sq.quantise(kc), sq.quantise(vc * torch.exp2((torch.arange(page, device="cuda") % 7 - 3).float())[None, None, :, None])
    used = torch.zeros(kc.shape[:3], dtype=torch.bool, device="cuda")
    kk, vv = [], []
    for s, n in enumerate(lengths):
        t = torch.arange(n, device="cuda")
        pg = table[s].long()[t // page] if n else t
        used[pg, :, t % page] = True
        kk.append(kval[pg, :, t % page])
        vv.append(vval[pg, :, t % page])
    for codes, scale in ((kq, kse), (vq, vse)):  # unused slots: NaN codes under the largest scales
        codes[~used] = 0x7f
        scale[~used] = 0xff
    q = sq.normal((sum(new) + 2, hq, d), dtype, 3)
    for causal in (True, False):
        out, lse = _call(cq, q, kq, vq, table, new, lengths, causal, (kse, vse))
        _check(out, lse, q, kk, vv, new, lengths, causal, torch.float16, f"causal={causal}", 2.0 ** 9)


@pytest.mark.parametrize("hq,new", [(4, 1), (4, 60)])
@pytest.mark.parametrize("cache", ["same", "e4m3"])
def test_equal_pages_and_table_order(cq, hq, new, cache):
    """The result does not depend on where pages lie or who else is in the batch, and repeats bit by bit."""
    d, page, dtype, n = 128, 32, torch.float16, 777
    got = []
    for seed_order in (1, 2):
        ks, vs, kc, vc, table = sq.make_cache([n, n], 2, d, page, dtype, 31, fill=0.0)
        order = torch.randperm(kc.shape[0], generator=torch.Generator().manual_seed(seed_order)).cuda()
        inverse = torch.argsort(order)
        kc, vc = kc[order].contiguous(), vc[order].contiguous()
        table = torch.where(table >= 0, inverse[table.long().clamp(min=0)].int(), table)
        scales = (None, None)
        if cache == "e4m3":
            (kc, a, _), (vc, b, _) = sq.quantise(kc), sq.quantise(vc)
            scales = (a, b)
        q = sq.normal((2 * new, hq, d), dtype, 3)
        for _ in range(2):
            got.append(_call(cq, q, kc, vc, table, [new, new], [n, n], True, scales))
    for o, l in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(l, got[0][1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cache", ["same", "e4m3"])
def test_chunk_ranges(cq, cache, d):
    """Chunks whose work is cut into ranges over units of very different lengths, in one phase of key heads or several (which
    the caller's longest length sets), and by one CTA where the caller says that there is hardly anything."""
    new, lengths, hq, hkv, page = [300, 0, 45, 700, 33], [300, 9, 4000, 1500, 20], 8, 4, 32
    dtype = torch.float16
    ks, vs, kc, vc, table = sq.make_cache(lengths, hkv, d, page, torch.float32 if cache == "e4m3" else dtype, 5,
                                          fill=0.0 if cache == "e4m3" else float("nan"), sharp=1.5)
    scales = {}
    if cache == "e4m3":
        (kc, kse, kval), (vc, vse, vval) = sq.quantise(kc), sq.quantise(vc)
        scales = {"k_scale": kse, "v_scale": vse}
        for s, n in enumerate(lengths):
            t = torch.arange(n, device="cuda")
            pg = table[s].long()[t // page]
            ks[s], vs[s] = kval[pg, :, t % page], vval[pg, :, t % page]
    q = sq.normal((sum(new), hq, d), dtype, 3)
    cu, kl = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (sq.starts(new), lengths))
    for causal in (True, False):
        for most in (1, 4000, 2_000_000):
            got = [cq.attention_paged(q, kc, vc, table, cu, kl, max(new), most, causal=causal, return_lse=True, **scales) for _ in range(2)]
            torch.cuda.synchronize()
            rc, code, _ = cq.cqsa_device_error()
            assert rc == cq.CQSA_OK and code == 0
            assert all(torch.equal(x, y) for x, y in zip(*got))
            out, lse = got[0]
            at = 0
            for s, n in enumerate(new):
                if n:
                    ref, rl, mass = sq.attend(q[at:at + n], ks[s], vs[s], lengths[s] - n, causal)
                    what = f"causal={causal} most={most} sequence {s}"
                    sq.check_out(out[at:at + n], ref, mass, dtype, dtype, what, lengths[s] * 2.0 ** (-25 if cache == "e4m3" else -34))
                    sq.check_lse(lse[:, at:at + n], rl, what)
                at += n


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cache", ["same", "e4m3"])
def test_units_without_keys(cq, cache, d):
    """Sequences without positions, and new tokens before the first position, between long ones: empty rows are 0 and -inf, the
    others' are right, and all of it repeats bit by bit."""
    new, lengths, hq, hkv, page = [150, 300, 40, 200] * 12, [0, 1900, 10, 700] * 12, 8, 2, 64
    dtype = torch.float16
    ks, vs, kc, vc, table = sq.make_cache(lengths, hkv, d, page, torch.float32 if cache == "e4m3" else dtype, 7,
                                          fill=0.0 if cache == "e4m3" else float("nan"), sharp=1.5)
    scales = {}
    if cache == "e4m3":
        (kc, kse, kval), (vc, vse, vval) = sq.quantise(kc), sq.quantise(vc)
        scales = {"k_scale": kse, "v_scale": vse}
        for s, n in enumerate(lengths):
            t = torch.arange(n, device="cuda")
            pg = table[s].long()[t // page] if n else t
            ks[s], vs[s] = kval[pg, :, t % page], vval[pg, :, t % page]
    q = sq.normal((sum(new), hq, d), dtype, 3)
    cu, kl = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (sq.starts(new), lengths))
    first = cq.attention_paged(q, kc, vc, table, cu, kl, max(new), max(lengths), return_lse=True, **scales)
    for _ in range(40):
        again = cq.attention_paged(q, kc, vc, table, cu, kl, max(new), max(lengths), return_lse=True, **scales)
        assert all(torch.equal(x, y) for x, y in zip(again, first))
    rc, code, _ = cq.cqsa_device_error()
    assert rc == cq.CQSA_OK and code == 0
    out, lse = first
    at = 0
    for s, n in enumerate(new):
        ref, rl, mass = sq.attend(q[at:at + n], ks[s], vs[s], lengths[s] - n, True)
        sq.check_out(out[at:at + n], ref, mass, dtype, dtype, f"sequence {s}", lengths[s] * 2.0 ** (-25 if cache == "e4m3" else -34))
        sq.check_lse(lse[:, at:at + n], rl, f"sequence {s}")
        empty = max(0, n - lengths[s])
        assert (out[at:at + empty] == 0).all() and (lse[:, at:at + empty] == float("-inf")).all()
        at += n


def test_graph_streams_and_workspaces(cq):
    """Captured with its own workspace and replayed on another stream beside an eager call, for lengths that change between replays."""
    d, page, dtype = 128, 16, torch.bfloat16
    lengths = [1000, 333, 64]
    ks, vs, kc, vc, table = sq.make_cache(lengths, 2, d, page, dtype, 41)
    q = sq.normal((3, 8, d), dtype, 4)
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    cq.attention_paged(q, kc, vc, table, cu, lens, 1, 1000)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = cq.attention_paged(q, kc, vc, table, cu, lens, 1, 1000, return_lse=True)
    other = sq.normal((3, 8, d), dtype, 5)
    for now in (lengths, [17, 333, 1], [1000, 2, 63]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        eager, elses = cq.attention_paged(other, kc, vc, table, cu, lens, 1, 1000, return_lse=True, stream=side)
        graph.replay()
        torch.cuda.synchronize()
        for o, l, x in ((out, lse, q), (eager, elses, other)):
            for s, n in enumerate(now):
                ref, rl, mass = sq.attend(x[s:s + 1], ks[s][:n], vs[s][:n], n - 1, True)
                sq.check_out(o[s:s + 1], ref, mass, dtype)
                sq.check_lse(l[:, s:s + 1], rl)


def test_query_stride_and_scale(cq):
    d, page, dtype = 64, 16, torch.float16
    ks, vs, kc, vc, table = sq.make_cache([100, 40], 2, d, page, dtype, 51)
    fused = sq.normal((45, 8, d), dtype, 6)
    q = fused[:, :4]
    for new in ([1, 1], [5, 40]):
        n = sum(new)
        out, lse = cq.attention_paged(q[:n], kc, vc, table, torch.tensor(sq.starts(new), dtype=torch.int32, device="cuda"),
                                      torch.tensor([100, 40], dtype=torch.int32, device="cuda"), max(new), 100, scale=0.25,
                                      return_lse=True)
        at = 0
        for s, c in enumerate(new):
            ref, rl, mass = sq.attend(q[at:at + c], ks[s], vs[s], [100, 40][s] - c, True, 0.25)
            sq.check_out(out[at:at + c], ref, mass, dtype)
            sq.check_lse(lse[:, at:at + c], rl)
            at += c
