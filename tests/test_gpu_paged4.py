"""Attention over a cache held in 4 bits on the GPU against its definition in 64 bits: single tokens and a few; grouped heads;
ragged lengths; empty rows; scales of every size; what lies in unused slots."""
import math

import pytest
import torch

from tests import _seq as sq
from tests import _seq4 as s4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cq():
    import exact_long_context_tcgen05_gb300 as m
    return m


def make_cache4(lengths, hkv, d, page, seed, sizes=(0,), sharp=1.5):
    """Keys and values of each sequence (64 bits, what the cache stands for), and the cache: pages in a shuffled order, unused slots of codes 0
    under NaN scales. `sizes`: powers of two that the values of successive slots are multiplied by."""
    _, _, kc, vc, table = sq.make_cache(lengths, hkv, d, page, torch.float32, seed, fill=0.0, sharp=sharp)
    factor = torch.exp2(torch.tensor(sizes, dtype=torch.float32, device="cuda"))[torch.arange(page, device="cuda") % len(sizes)]
    (kq, kse, kval), (vq, vse, vval) = s4.quantise4(kc), s4.quantise4(vc * factor[None, None, :, None])
    used = torch.zeros(kc.shape[:3], dtype=torch.bool, device="cuda")
    kk, vv = [], []
    for s, n in enumerate(lengths):
        t = torch.arange(n, device="cuda")
        pg = table[s].long()[t // page] if n else t
        used[pg, :, t % page] = True
        kk.append(kval[pg, :, t % page])
        vv.append(vval[pg, :, t % page])
    for codes, scale in ((kq, kse), (vq, vse)):
        codes[~used] = 0
        scale[~used] = 0xff
    return kk, vv, kq, vq, kse, vse, table


def call(cq, q, kq, vq, kse, vse, table, new, lengths, causal=True, **kw):
    cu = torch.tensor(sq.starts(new), dtype=torch.int32, device="cuda")
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out, lse = cq.attention_paged(q, kq, vq, table, cu, lens, max(new), max(lengths), causal=causal, k_scale=kse, v_scale=vse,
                                  return_lse=True, out=torch.full_like(q, 7.0), **kw)
    torch.cuda.synchronize()
    rc, code, _ = cq.cqsa_device_error()
    assert rc == cq.CQSA_OK and code == 0
    return out, lse


def check(out, lse, q, ks, vs, new, lengths, causal, what, scale=None):
    """Probabilities are rounded to fp16, and once more when their value's scale is multiplied in: twice 2^-11 relative. They are kept as
    2^14 p (a chunk's: as 2^5 p at least), times a scale relative to the largest power of two of one: a product below fp16's normal
    numbers is off by 2^-25, that is by 2^-39 (2^-30) times the largest scale at most, times a whole number up to 7."""
    at = 0
    for s, n in enumerate(new):
        if n == 0:
            continue
        ref, rl, mass = sq.attend(q[at:at + n], ks[s], vs[s], lengths[s] - n, causal, scale)
        chunk = max(new) * (q.shape[1] // ks[s].shape[1]) > 32
        largest = vs[s].abs().max().item() if lengths[s] else 0.0
        floor = lengths[s] * 2.0 * largest * 2.0 ** (-30 if chunk else -39)
        assert torch.isfinite(out[at:at + n]).all(), what
        u = sq.U[q.dtype]
        tol = 1.01 * (u * ref.abs() + (2 * 2.0 ** -11 + 2.0 ** -16) * mass) + 2.0 ** -24 + floor
        excess = ((out[at:at + n].double() - ref).abs() - tol).max().item()
        assert excess <= 0, f"{what} sequence {s}: {excess:.3e} beyond the tolerance"
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
    ([1, 1], [700, 33], 9, 1, 16),                                    # 9 rows
    ([1, 1], [700, 129], 32, 1, 256),                                 # 32 heads of a key head
    ([2, 2, 1, 3], [2, 200, 64, 127], 8, 2, 256),
    ([4, 4], [900, 64], 32, 4, 16),                                   # 32 rows
    ([17, 2], [333, 2], 2, 2, 64),                                    # 17 rows
    ([6, 3, 2], [0, 2, 1], 4, 2, 16),                                 # sequences shorter than their new tokens: empty rows
    ([1, 1], [0, 40], 4, 2, 16),
]


@pytest.mark.parametrize("new,lengths,hq,hkv,page", CASES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("sizes", [(0,), (0, 3, -5, 1, -2), (-9, -8, -13)])
def test_paged_4bit(cq, new, lengths, hq, hkv, page, d, dt, sizes):
    ks, vs, *cache = make_cache4(lengths, hkv, d, page, 17 + len(new), sizes)
    q = sq.normal((sum(new) + 2, hq, d), sq.DT[dt], 3)
    for causal in (True, False):
        out, lse = call(cq, q, *cache, new, lengths, causal)
        check(out, lse, q, ks, vs, new, lengths, causal, f"causal={causal}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq", [4, 12])
def test_large_and_rising_scales(cq, d, hq):
    """Values from 2^-14's to 2^14's scales, rising and falling along the sequence; keys of large and small scales under queries that bring
    their scores back."""
    lengths, page = [700], 16
    for powers in ([-12, 0, 12], [12, 0, -12], [-3, 10, 2]):
        ks, vs, kq, vq, kse, vse, table = make_cache4(lengths, 1, d, page, 5, sharp=1.0)
        at = torch.arange(700, device="cuda") // 256
        pg, slot = table[0].long()[torch.arange(700, device="cuda") // page], torch.arange(700, device="cuda") % page
        by = torch.tensor(powers, device="cuda")[at]
        vse[pg, :, slot] = (vse[pg, :, slot].int() + 8 * by[:, None, None].int()).clamp(8, 247).to(torch.uint8)
        vs[0] = s4.values4(vq[pg, :, slot], vse[pg, :, slot])
        for dt, kpow in (("f16", 0), ("bf16", 10), ("bf16", -10)):
            k_now = kse.clone()
            k_now[pg, :, slot] = (kse[pg, :, slot].int() + 8 * kpow).clamp(8, 247).to(torch.uint8)
            k64 = s4.values4(kq[pg, :, slot], k_now[pg, :, slot])
            q = (sq.normal((1, hq, d), torch.float32, 3) * 2.0 ** -kpow).to(sq.DT[dt])
            out, lse = call(cq, q, kq, vq, k_now, vse, table, [1], lengths)
            ref, rl, mass = sq.attend(q, k64, vs[0], 699, True)
            scale = s4.scale_of(vse[pg, :, slot]).max().item()
            tol = 1.01 * (sq.U[q.dtype] * ref.abs() + (2.0 ** -10 + 2.0 ** -16) * mass) + 2.0 ** -24 + 700 * 14 * scale * 2.0 ** -38
            assert ((out.double() - ref).abs() <= tol).all()
            sq.check_lse(lse, rl)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 3, 7])
def test_not_a_number(cq, d, new):
    """A NaN scale of a key makes the rows that see it NaN, one of a value its 32 features; sequences beside it are untouched, and so are rows
    before a NaN key and empty rows."""
    hq, hkv, page, lengths = 4, 2, 16, [300, 200]
    ks, vs, kq, vq, kse, vse, table = make_cache4(lengths, hkv, d, page, 9)
    q = sq.normal((2 * new + 2, hq, d), torch.float16, 3)
    clean = call(cq, q, kq, vq, kse, vse, table, [new, new], lengths)
    bad_v, bad_k = vse.clone(), kse.clone()
    bad_v[table[0, 100 // page], 1, 100 % page, 1] = 255
    out, lse = call(cq, q, kq, vq, kse, bad_v, table, [new, new], lengths)
    want = torch.zeros_like(out, dtype=torch.bool)
    want[:new, 2:, 32:64] = True
    n = 2 * new  # (lse of the rows behind the last sequence is left as it was allocated)
    assert torch.equal(torch.isnan(out), want) and torch.equal(lse[:, :n], clean[1][:, :n])
    assert torch.equal(out[new:], clean[0][new:]) and torch.equal(out[:, :2], clean[0][:, :2])
    last = lengths[0] - 1  # the last token's own key: the rows before it do not see it
    bad_k[table[0, last // page], 0, last % page, 0] = 255
    out, lse = call(cq, q, kq, vq, bad_k, vse, table, [new, new], lengths)
    want = torch.zeros_like(out, dtype=torch.bool)
    want[new - 1, :2] = True
    assert torch.equal(torch.isnan(out), want) and torch.equal(torch.isnan(lse[:, :n]), want[:n, :, 0].T)
    empty, elses = call(cq, q, kq, vq, kse, bad_v, table, [new, new], [0, 200])
    assert (empty[:new] == 0).all() and (elses[:, :new] == -math.inf).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 3, 7])
@pytest.mark.parametrize("powers", [(-10,), (0,), (0, 9, -6)])
def test_numbers_beside_a_nan_value(cq, d, new, powers):
    """A NaN scale of a value takes nothing from the other features of its head, however small their values are: they are as near to the formula as without it."""
    hq, page, lengths = 4, 16, [300]
    ks, vs, kq, vq, kse, vse, table = make_cache4(lengths, 1, d, page, 9, powers)
    q = sq.normal((new, hq, d), torch.float16, 3)
    pad = torch.full((1, hq, d), 7.0, dtype=q.dtype, device="cuda")
    clean = call(cq, q, kq, vq, kse, vse, table, [new], lengths)
    bad = vse.clone()
    for at in (0, 131):  # a warp's first key, and one in mid-sequence
        bad[table[0, at // page], 0, at % page, 1] = 255
    out, lse = call(cq, q, kq, vq, kse, bad, table, [new], lengths)
    assert torch.isnan(out[..., 32:64]).all() and torch.equal(lse, clean[1])
    rest = torch.cat([out[..., :32], clean[0][..., 32:64], out[..., 64:]], -1)
    check(torch.cat([rest, pad]), torch.cat([lse, torch.zeros_like(lse[:, :1])], 1), q, ks, vs, [new], lengths, True, "beside a NaN")


@pytest.mark.parametrize("hq,new", [(4, 1), (4, 5)])
def test_equal_pages_and_table_order(cq, hq, new):
    """The result does not depend on where pages lie, and repeats bit by bit."""
    d, page, n = 128, 32, 777
    got = []
    for seed_order in (1, 2):
        ks, vs, kq, vq, kse, vse, table = make_cache4([n, n], 2, d, page, 31)
        order = torch.randperm(kq.shape[0], generator=torch.Generator().manual_seed(seed_order)).cuda()
        inverse = torch.argsort(order)
        kq, vq, kse, vse = (x[order].contiguous() for x in (kq, vq, kse, vse))
        table = torch.where(table >= 0, inverse[table.long().clamp(min=0)].int(), table)
        q = sq.normal((2 * new, hq, d), torch.float16, 3)
        for _ in range(2):
            got.append(call(cq, q, kq, vq, kse, vse, table, [new, new], [n, n]))
    for o, l in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(l, got[0][1])


@pytest.mark.parametrize("d", [64, 128])
def test_long_sums(cq, d):
    """One sequence long enough for a warp's sums to be folded many times, values of one sign: what the tensor core cuts off as it accumulates
    stays below 2^-13 of the sum (256 products, 2^-23 each at most, twice)."""
    n, page, hq, hkv = 2 ** 18 + 77, 256, 4, 1
    pages = -(-n // page)
    g = torch.Generator(device="cuda").manual_seed(3)
    kc = torch.randn(pages, hkv, page, d, generator=g, device="cuda") * 0.05
    vc = torch.rand(pages, hkv, page, d, generator=g, device="cuda") + 0.5
    (kq, kse, kval), (vq, vse, vval) = s4.quantise4(kc), s4.quantise4(vc)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    q = sq.normal((1, hq, d), torch.float16, 5)
    cu, lens = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([n], dtype=torch.int32, device="cuda")
    for most in (1, n):  # one CTA for all of it, and one a range
        out = cq.attention_paged(q, kq, vq, table, cu, lens, 1, most, k_scale=kse, v_scale=vse)
        k, v = kval[:, 0].reshape(-1, d)[:n, None], vval[:, 0].reshape(-1, d)[:n, None]
        ref, _, mass = sq.attend(q, k, v, n - 1, True)
        # (roundings of 2^18 probabilities that point either way add little)
        assert ((out.double() - ref).abs() <= (2.0 ** -11 + 2.0 ** -13 + 2.0 ** -13) * mass).all()


def test_graph_streams_and_workspaces(cq):
    """Captured with its own workspace and replayed beside an eager call on another stream, for lengths that change between replays."""
    d, page, lengths = 128, 16, [1000, 333, 64]
    ks, vs, kq, vq, kse, vse, table = make_cache4(lengths, 2, d, page, 41)
    q, other = sq.normal((3, 8, d), torch.bfloat16, 4), sq.normal((3, 8, d), torch.bfloat16, 5)
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # (the kernel's first call, maybe)
        out, lse = cq.attention_paged(q, kq, vq, table, cu, lens, 1, 1000, return_lse=True, k_scale=kse, v_scale=vse)
    for now in (lengths, [17, 333, 1], [1000, 2, 63]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        eager, elses = cq.attention_paged(other, kq, vq, table, cu, lens, 1, 1000, return_lse=True, stream=side, k_scale=kse, v_scale=vse)
        graph.replay()
        torch.cuda.synchronize()
        for o, l, x in ((out, lse, q), (eager, elses, other)):
            pad = torch.full((1, 8, d), 7.0, dtype=x.dtype, device="cuda")
            check(torch.cat([o, pad]), l, x, [k[:n] for k, n in zip(ks, now)], [v[:n] for v, n in zip(vs, now)], [1, 1, 1], now, True, "graph")


def test_waits_give_up(cq):
    """A key tile that never arrives: the kernel gives up after the limit, the error word says so, and the next call is right."""
    ks, vs, *cache = make_cache4([1000], 2, 64, 32, 3)
    q = sq.normal((1, 8, 64), torch.float16, 3)
    pad = torch.full((1, 8, 64), 7.0, dtype=q.dtype, device="cuda")
    cq.cqsa_set_timeout_ms(200)
    try:
        cq.cqsa_debug_set_fault(1)
        cu, lens = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([1000], dtype=torch.int32, device="cuda")
        cq.attention_paged(q, cache[0], cache[1], cache[4], cu, lens, 1, 1000, k_scale=cache[2], v_scale=cache[3])
        torch.cuda.synchronize()
        rc, code, _ = cq.cqsa_device_error(clear=True)
        assert rc == cq.CQSA_ERR_TIMEOUT and code != 0
    finally:
        cq.cqsa_debug_set_fault(0)
        cq.cqsa_set_timeout_ms(0)
    out, lse = call(cq, q, *cache, [1], [1000])
    check(torch.cat([out, pad]), lse, q, ks, vs, [1], [1000], True, "after")


CHUNKS = [
    # new tokens, lengths, Hq, Hkv, page
    ([3, 1, 5], [3, 1, 700], 14, 2, 16),                              # a group of 7 heads, just over 32 rows
    ([64, 1, 0, 130], [64, 400, 9, 1130], 8, 2, 16),
    ([300], [2300], 4, 4, 64),
    ([257, 128], [257, 129], 6, 2, 32),
    ([70], [70], 64, 1, 16),                                          # one key head for 64
    ([40, 3, 2], [0, 2, 1], 4, 2, 16),                                # sequences shorter than their new tokens: empty rows
    ([33, 40], [5000, 33], 1, 1, 256),
]


@pytest.mark.parametrize("new,lengths,hq,hkv,page", CHUNKS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("sizes", [(0,), (0, 3, -5, 1, -2), (-9, -8, -13)])
def test_chunks_4bit(cq, new, lengths, hq, hkv, page, d, dt, sizes):
    ks, vs, *cache = make_cache4(lengths, hkv, d, page, 17 + len(new), sizes)
    q = sq.normal((sum(new) + 2, hq, d), sq.DT[dt], 3)
    for causal in (True, False):
        out, lse = call(cq, q, *cache, new, lengths, causal)
        check(out, lse, q, ks, vs, new, lengths, causal, f"causal={causal}")


@pytest.mark.parametrize("d", [64, 128])
def test_chunk_ranges(cq, d):
    """Chunks whose work is cut into ranges over units of very different lengths, in one phase of key heads or several, and by one
    CTA; twice the same bit by bit."""
    new, lengths, hq, hkv, page = [300, 0, 45, 700, 33], [300, 9, 4000, 1500, 20], 8, 4, 32
    ks, vs, kq, vq, kse, vse, table = make_cache4(lengths, hkv, d, page, 5, (0, 2, -1))
    q = sq.normal((sum(new), hq, d), torch.float16, 3)
    cu, kl = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (sq.starts(new), lengths))
    pad = torch.full((1, hq, d), 7.0, dtype=q.dtype, device="cuda")
    for causal in (True, False):
        for most in (1, 4000, 2_000_000):
            got = [cq.attention_paged(q, kq, vq, table, cu, kl, max(new), most, causal=causal, return_lse=True, k_scale=kse, v_scale=vse)
                   for _ in range(2)]
            torch.cuda.synchronize()
            assert cq.cqsa_device_error()[1] == 0
            assert all(torch.equal(x, y) for x, y in zip(*got))
            check(torch.cat([got[0][0], pad]), got[0][1], q, ks, vs, new, lengths, causal, f"causal={causal} most={most}")


@pytest.mark.parametrize("powers", [[0, 3, 6], [5, -3, 1], [-2, -2, 7]])
@pytest.mark.parametrize("d,dt", [(128, "f16"), (128, "bf16"), (64, "f16"), (64, "bf16")])
def test_chunks_with_running_sums(cq, d, dt, powers):
    """Units long enough for running sums of O, values whose sizes rise and fall from one segment to the next, through the cache's own
    write."""
    dtype, hq, hkv, page, new = sq.DT[dt], 8, 2, 64, [300, 130]
    segment = 4096 if d == 128 else 16384
    lengths = [2 * segment + 900, segment + 1100]
    per = [-(-n // page) for n in lengths]
    kc, vc = (torch.zeros(sum(per), hkv, page, d // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
    scales = {n: torch.zeros(sum(per), hkv, page, d // 32, dtype=torch.uint8, device="cuda") for n in ("k_scale", "v_scale")}
    table = torch.zeros(2, max(per), dtype=torch.int32, device="cuda")
    order = torch.randperm(sum(per), generator=torch.Generator().manual_seed(3)).to(torch.int32).cuda()
    table[0, :per[0]], table[1, :per[1]] = order[:per[0]], order[per[0]:]
    ks, vs = [], []
    for s, n in enumerate(lengths):
        by = torch.exp2(torch.tensor(powers, dtype=torch.float64, device="cuda"))[(torch.arange(n, device="cuda") // segment).clamp(max=2)][:, None, None]
        k = (sq.normal((n, hkv, d), torch.float64, 10 + s) * by ** 0.25).to(dtype)
        v = (sq.normal((n, hkv, d), torch.float64, 20 + s) * by).to(dtype)
        cq.kv_cache_write(k, v, kc, vc, table[s:s + 1].contiguous(), torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                          torch.tensor([n], dtype=torch.int32, device="cuda"), **scales)
        ks.append(s4.quantise4(k)[2])
        vs.append(s4.quantise4(v)[2])
    q = sq.normal((sum(new), hq, d), dtype, 5)
    cu, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (sq.starts(new), lengths))
    pad = torch.full((1, hq, d), 7.0, dtype=dtype, device="cuda")
    for most in (1, max(lengths)):
        for causal in (True, False):
            out, lse = cq.attention_paged(q, kc, vc, table, cu, lens, max(new), most, causal=causal, return_lse=True, **scales)
            torch.cuda.synchronize()
            assert cq.cqsa_device_error()[1] == 0
            check(torch.cat([out, pad]), lse, q, ks, vs, new, lengths, causal, f"most={most} causal={causal}")


def test_chunk_nan(cq):
    """A NaN scale of a key makes the rows that see it NaN; a value's the 32 features of its head's rows; other sequences and heads are untouched."""
    d, hq, hkv, page, new, lengths = 128, 4, 2, 16, [40, 50], [300, 200]
    ks, vs, kq, vq, kse, vse, table = make_cache4(lengths, hkv, d, page, 9)
    q = sq.normal((90, hq, d), torch.bfloat16, 3)
    clean = call(cq, q, kq, vq, kse, vse, table, new, lengths)
    bad_v, bad_k = vse.clone(), kse.clone()
    bad_v[table[0, 100 // page], 1, 100 % page, 1] = 255
    bad_k[table[0, 279 // page], 0, 279 % page, 3] = 255  # the position of new token 19
    out, lse = call(cq, q, kq, vq, kse, bad_v, table, new, lengths)
    want = torch.zeros_like(out, dtype=torch.bool)
    want[:40, 2:, 32:64] = True
    assert torch.equal(torch.isnan(out), want) and torch.equal(out[~want], clean[0][~want])
    out, lse = call(cq, q, kq, vq, bad_k, vse, table, new, lengths)
    want[:] = False
    want[19:40, :2] = True
    assert torch.equal(torch.isnan(out), want) and torch.equal(torch.isnan(lse), want[..., 0].T)


def _checked(cq, q, kq, vq, kse, vse, table, ks, vs, new, lengths, most, what):
    """Twice the same bit by bit and captured, and right with either rounding of the probabilities (which sequences are unpacked is the workspace's matter)."""
    cu, kl = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (sq.starts(new), lengths))
    for causal in (True, False):
        def run():
            return cq.attention_paged(q, kq, vq, table, cu, kl, max(new), most, causal=causal, return_lse=True, k_scale=kse, v_scale=vse)
        out, lse = run()
        assert all(torch.equal(x, y) for x, y in zip(run(), (out, lse)))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            again = run()
        graph.replay()
        torch.cuda.synchronize()
        assert cq.cqsa_device_error()[1] == 0
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
        at = 0
        for s, n in enumerate(new):
            if n:
                ref, rl, mass = sq.attend(q[at:at + n], ks[s], vs[s], lengths[s] - n, causal)
                tol = 1.01 * (sq.U[q.dtype] * ref.abs() + (max(sq.U[q.dtype], 2.0 ** -10) + 2.0 ** -16) * mass) + 2.0 ** -24 + lengths[s] * 2.0 ** -25
                assert ((out[at:at + n].double() - ref).abs() <= tol).all(), (what, causal, s)
                sq.check_lse(lse[:, at:at + n], rl, f"{what} {causal} {s}")
            at += n


def _space(cq, q, new, hkv, page, most, packed):
    """The workspace's size beyond what the packed kernel alone needs (a longest length of 1 asks for no more)."""
    T, hq, d = q.shape
    size = [cq.cqsa_attn_paged_workspace_size(len(new), T, hq, hkv, d, page, max(new), m, cq.dtype_code(q.dtype), cq.CQSA_INT4) for m in (most, packed)]
    return size[0] - size[1]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_unpacked_sequences(cq, d, dt):
    """A batch whose longer sequences are unpacked (by a longest length that says much work) or not: lengths beside multiples of a scratch page, sequences
    without positions and of a few tokens among them."""
    new = [130, 1, 128, 0, 127, 300, 129, 4, 200]
    lengths = [129, 900, 128, 70, 1000, 2049, 0, 40, 3000]
    hq, hkv, page = 8, 2, 16
    ks, vs, *cache = make_cache4(lengths, hkv, d, page, 5, (0, 2, -1))
    q = sq.normal((sum(new), hq, d), sq.DT[dt], 3)
    assert _space(cq, q, new, hkv, page, 100_000, 3000) > 200 << 20
    for most in (100_000, 3000, 0):
        _checked(cq, q, *cache, ks, vs, new, lengths, most, most)


def test_more_than_the_scratch_pages(cq):
    """Sequences longer than the caller said: the first are unpacked as far as the scratch pages go, the others are read packed."""
    d, hq, hkv, page = 64, 32, 8, 64
    new, lengths = [1500, 900, 20, 1700, 1000, 600, 64, 2000], [1500, 1000, 700, 6000, 5000, 600, 640, 4100]
    ks, vs, *cache = make_cache4(lengths, hkv, d, page, 6)
    q = sq.normal((sum(new), hq, d), torch.float16, 3)
    # 16 pages of 128 for each of 8 sequences; the six that are long enough need 145
    assert 128 * 128 * hkv * d * 4 <= _space(cq, q, new, hkv, page, 2000, 500) < 200 * 128 * hkv * d * 4
    _checked(cq, q, *cache, ks, vs, new, lengths, 2000, "2000")


def test_unpacked_extremes(cq):
    """Values past fp16's largest are held at it where a sequence is unpacked to fp16, a NaN scale stays one, and bf16 holds all of a 4-bit cache's range."""
    d, hq, hkv, page, n, new = 128, 8, 2, 32, 400, 130
    for dt in ("f16", "bf16"):
        ks, vs, kq, vq, kse, vse, table = make_cache4([n], hkv, d, page, 9)
        t = torch.arange(n, device="cuda")
        pg, slot = table[0].long()[t // page], t % page
        big = vse.clone()
        big[pg, :, slot, 0] = 246  # scales of 14 / 8 * 2^15 = 57,344: multiples up to 401,408
        v64 = s4.values4(vq[pg, :, slot], big[pg, :, slot])
        if dt == "f16":
            v64 = v64.clamp(-65504, 65504)
        q = sq.normal((new, hq, d), sq.DT[dt], 3)
        cu, lens = torch.tensor([0, new], dtype=torch.int32, device="cuda"), torch.tensor([n], dtype=torch.int32, device="cuda")

        def run(v_scale):  # (a longest length that says much work: the sequence is unpacked)
            return cq.attention_paged(q, kq, vq, table, cu, lens, new, 1_000_000, k_scale=kse, v_scale=v_scale)
        out = run(big)
        ref, rl, mass = sq.attend(q, ks[0], v64, n - new, True)
        tol = 1.01 * (sq.U[q.dtype] * ref.abs() + (max(sq.U[q.dtype], 2.0 ** -10) + 2.0 ** -16) * mass) + 2.0 ** -24
        fits = ref.abs() < (60000 if dt == "f16" else 1e9)
        assert ((out.double() - ref).abs() <= tol)[fits].all()
        bad = vse.clone()
        bad[pg[100], 1, slot[100], 1] = 255
        out = run(bad)
        want = torch.zeros_like(out, dtype=torch.bool)
        want[:, 4:, 32:64] = True
        assert torch.equal(torch.isnan(out), want)
