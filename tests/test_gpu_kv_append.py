"""Appending to the paged cache with the position rotation, and the 4-bit cache's write and read, on the GPU."""
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


def _caches(kind, pages, hkv, page, d, dtype):
    """k_cache, v_cache, k_scale, v_scale of zeros (bytes of 7 in the scales)."""
    if kind == "same":
        return [torch.zeros(pages, hkv, page, d, dtype=dtype, device="cuda") for _ in range(2)] + [None, None]
    width, more = (d, ()) if kind == "e4m3" else (d // 2, (d // 32,))
    return [torch.zeros(pages, hkv, page, width, dtype=torch.uint8, device="cuda") for _ in range(2)] + \
        [torch.full((pages, hkv, page, *more), 7, dtype=torch.uint8, device="cuda") for _ in range(2)]


def _place(table, new, lengths, page):
    """Position, page and slot of every new token."""
    at = [(lengths[s] - n + i, int(table[s, (lengths[s] - n + i) // page]), (lengths[s] - n + i) % page)
          for s, n in enumerate(new) for i in range(n)]
    return torch.tensor(at, dtype=torch.long, device="cuda").reshape(-1, 3).unbind(-1)


def _problem(new, lengths, page, seed):
    _, _, _, _, table = sq.make_cache(lengths, 1, 64, page, torch.float16, seed)
    cu = torch.tensor(sq.starts(new), dtype=torch.int32, device="cuda")
    return table, cu, torch.tensor(lengths, dtype=torch.int32, device="cuda"), int(table.max()) + 2


def _check_cache(kind, cache, scale, x, page, slot):
    """The cache holds x [T, Hkv, d] (32 bits, not rounded) in its slots, and zeros elsewhere."""
    want = torch.zeros_like(cache)
    if kind == "same":
        want[page, :, slot] = x.to(cache.dtype)
        assert torch.equal(cache, want)
        return
    if kind == "4bit":
        code, byte, val = s4.quantise4(x)
    else:
        code, byte, val = sq.quantise(x)
    got, got_byte = cache[page, :, slot], scale[page, :, slot]
    nan = torch.isnan(val)
    assert torch.equal(got_byte, byte)
    if kind == "4bit":
        nan = nan[..., 0::2]
    assert torch.equal(got[~nan], code[~nan])
    cache, scale = cache.clone(), scale.clone()
    cache[page, :, slot], scale[page, :, slot] = 0, 7
    assert (cache == 0).all() and (scale == 7).all()


CASES = [([1], [1], 3, 1, 64, 16), ([1, 1, 1], [17, 1, 400], 8, 2, 128, 16), ([5, 0, 40, 7], [5, 9, 333, 64], 6, 3, 64, 32),
         ([130, 1], [300, 129], 32, 8, 128, 64), ([33] * 40, [33 + 7 * i for i in range(40)], 5, 5, 128, 256),
         ([70, 3], [70, 130], 0, 33, 64, 128)]


@pytest.mark.parametrize("kind", ["same", "e4m3", "4bit"])
@pytest.mark.parametrize("rot,inter", [(None, False), (None, True), (16, False), (48, True), (48, False), (32, False)])
@pytest.mark.parametrize("new,lengths,hq,hkv,d,page", CASES)
def test_append(cq, new, lengths, hq, hkv, d, page, rot, inter, kind):
    dtype = torch.bfloat16 if (hkv + page // 16) % 2 else torch.float16
    rot, T, behind = rot or d, sum(new), 3
    table, cu, lens, pages = _problem(new, lengths, page, 3)
    q = sq.normal((T + behind, hq, d), dtype, 11) if hq else None
    k, v = sq.normal((T + behind, hkv, d), dtype, 12, 2.0), sq.normal((T + behind, hkv, d), dtype, 13)
    turn = cq.rotary_table(max(lengths) + 1, rot, base=500.0)
    kc, vc, ks, vs = _caches(kind, pages, hkv, page, d, dtype)
    q_out = torch.full_like(q, 7.0) if hq else None
    got = cq.kv_cache_append(q, k, v, turn, kc, vc, table, cu, lens, interleaved=inter, k_scale=ks, v_scale=vs, q_out=q_out)
    position, pg, slot = _place(table, new, lengths, page)
    _check_cache(kind, kc, ks, s4.turned(k[:T], turn, position, inter), pg, slot)
    _check_cache(kind, vc, vs, v[:T].float(), pg, slot)
    assert got is q_out
    if hq:
        assert torch.equal(got[:T], s4.turned(q[:T], turn, position, inter).to(dtype))
        assert (got[T:] == 7.0).all()  # rows behind the last sequence are left as they were
        # and against 64 bits: three 32-bit roundings of at most |x c| + |y s|, and the rounding to 16 bits
        half = rot // 2
        pair = [(2 * j, 2 * j + 1) if inter else (j, j + half) for j in range(half)]
        a, b = (q[:T, :, [p[i] for p in pair]].double() for i in (0, 1))
        f = 500.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") * 2 / rot)
        angle = (position[:, None].double() * f)[:, None]
        for want, at in ((a * angle.cos() - b * angle.sin(), 0), (b * angle.cos() + a * angle.sin(), 1)):
            err = (got[:T][:, :, [p[at] for p in pair]].double() - want).abs()
            assert (err <= 1.01 * sq.U[dtype] * want.abs() + 4 * 2.0 ** -24 * (a.abs() + b.abs()) + 2.0 ** -25).all()


@pytest.mark.parametrize("new,lengths,hq,hkv,d,page", CASES)
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_write_and_read_4bit(cq, new, lengths, hq, hkv, d, page, dt):
    dtype = sq.DT[dt]
    T = sum(new)
    table, cu, lens, pages = _problem(new, lengths, page, 5)
    k, v = sq.normal((T + 2, hkv, d), dtype, 21, 2.0), sq.normal((T + 2, hkv, d), dtype, 22)
    # groups of every size: zeros, one large value, tiny ones, exact ties of scale and code, NaN and infinities
    k[0] = 0
    v[T - 1] *= 2.0 ** -16
    k[T - 1, :, 0] = 448.0
    if T > 4:
        k[1, 0, :32] = torch.arange(-16, 16, device="cuda") / 2.0  # amax 8
        k[1, 0, 32:64] = torch.arange(-16, 16, device="cuda") * 0.4375  # amax 7: scale 1, codes of 0.4375 steps
        k[1, 0, 40] = 2.5
        v[1] *= 512.0
        v[1, 0, 0] = 7.0 * 1.0625  # a scale half way between two
        k[2, 0, 1], v[2, 0, 40], v[3, 0, 5] = math.inf, math.nan, -math.inf
        if dt == "bf16":
            k[3] *= 2.0 ** 100
            v[3] *= 2.0 ** -120
            v[3, 0, 5] = -math.inf
        else:
            k[3] = 65504.0
    kc, vc, ks, vs = _caches("4bit", pages, hkv, page, d, dtype)
    cq.kv_cache_write(k, v, kc, vc, table, cu, lens, k_scale=ks, v_scale=vs)
    _, pg, slot = _place(table, new, lengths, page)
    _check_cache("4bit", kc, ks, k[:T].float(), pg, slot)
    _check_cache("4bit", vc, vs, v[:T].float(), pg, slot)
    out = tuple(torch.full_like(k, 5.0) for _ in range(2))
    got = cq.kv_cache_read(kc, vc, table, cu, lens, T + 2, dtype, k_scale=ks, v_scale=vs, out=out)
    for g, x in zip(got, (k, v)):
        val = s4.quantise4(x[:T])[2]
        want = val.clamp(-65504, 65504).to(dtype) if dt == "f16" else val.to(dtype)  # exact but for what fp16 cannot hold
        assert torch.equal(torch.isnan(g[:T]), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(g[:T], 0.0), torch.nan_to_num(want, 0.0))
        assert (g[T:] == 5.0).all()


def test_ties_of_every_scale(cq):
    """Values at and beside the borders between codes, for every scale that 16-bit values can ask for."""
    d, page, hkv = 64, 16, 1
    scale = s4.scale_of(torch.arange(8, 200, device="cuda"))  # 2^-14 .. 2^9: |x| below fp16's largest
    step = torch.tensor([1.0, 1 + 2.0 ** -8, 1 - 2.0 ** -8], dtype=torch.float64, device="cuda")
    tie = torch.tensor([i + 0.5 for i in range(-7, 7)], dtype=torch.float64, device="cuda")
    x = (tie[:, None] * step).flatten().repeat(2)[:62] * scale[:, None]
    x = torch.cat([x[:, :31], 7 * scale[:, None], x[:, 31:], -7 * scale[:, None]], -1)
    for dtype in (torch.float16, torch.bfloat16):
        k = x.to(dtype)[:, None]
        T = k.shape[0]
        table = torch.arange(-(-T // page), dtype=torch.int32, device="cuda")[None]
        cu, lens = torch.tensor([0, T], dtype=torch.int32, device="cuda"), torch.tensor([T], dtype=torch.int32, device="cuda")
        kc, vc, ks, vs = _caches("4bit", table.shape[1], hkv, page, d, dtype)
        cq.kv_cache_write(k, k, kc, vc, table, cu, lens, k_scale=ks, v_scale=vs)
        _, pg, slot = _place(table, [T], [T], page)
        _check_cache("4bit", kc, ks, k.float(), pg, slot)


@pytest.mark.parametrize("kind", ["same", "e4m3", "4bit"])
def test_what_stays_away(cq, kind):
    """Infinities and NaN reach their own pair and, in a quantised cache, their own vector or group, nothing else."""
    d, page, hkv, dtype = 128, 16, 2, torch.float16
    k = sq.normal((3, hkv, d), dtype, 31)
    q = sq.normal((3, 4, d), dtype, 32)
    k[1, 0, 3], q[1, 2, 127], q[1, 1, 70] = math.inf, math.nan, -math.inf
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    cu, lens = torch.tensor([0, 3], dtype=torch.int32, device="cuda"), torch.tensor([3], dtype=torch.int32, device="cuda")
    turn = cq.rotary_table(3, 64)
    kc, vc, ks, vs = _caches(kind, 1, hkv, page, d, dtype)
    got = cq.kv_cache_append(q, k, k, turn, kc, vc, table, cu, lens, k_scale=ks, v_scale=vs)
    want = s4.turned(q, turn, torch.arange(3, device="cuda"), False).to(dtype)
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
    assert torch.isfinite(got[1, 0]).all() and torch.isfinite(got[[0, 2]]).all() and int((~torch.isfinite(got)).sum()) == 2
    rk, rv = cq.kv_cache_read(kc, vc, table, cu, lens, 3, dtype, k_scale=ks, v_scale=vs)
    bad_k, bad_v = ~torch.isfinite(rk), ~torch.isfinite(rv)
    assert not bad_k[[0, 2]].any() and not bad_k[1, 1].any() and not bad_v[[0, 2]].any() and not bad_v[1, 1].any()
    if kind == "4bit":
        assert bad_k[1, 0].nonzero().flatten().tolist() == list(range(0, 64)) and bad_v[1, 0].nonzero().flatten().tolist() == list(range(32))
    else:
        assert bad_k[1, 0].nonzero().flatten().tolist() == [3, 35] and bad_v[1, 0].nonzero().flatten().tolist() == [3]


def test_skipped_tokens(cq):
    """Positions below zero or past the table of angles are skipped with their queries; a bad page skips keys and values alone."""
    page, hkv, d, dtype = 16, 2, 64, torch.float16
    table = torch.tensor([[0, 99], [1, -5], [2, 3]], dtype=torch.int32, device="cuda")
    new, lens = [20, 17, 40], [20, 17, 36]
    T = sum(new)
    k, q = sq.normal((T, hkv, d), dtype, 3), sq.normal((T, 4, d), dtype, 4)
    cu = torch.tensor(sq.starts(new), dtype=torch.int32, device="cuda")
    kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
    turn = cq.rotary_table(30, 64)
    kc, vc, _, _ = _caches("same", 4, hkv, page, d, dtype)
    got = cq.kv_cache_append(q, k, k, turn, kc, vc, table, cu, kv, q_out=torch.full_like(q, 9.0))
    position = torch.cat([torch.arange(n - m, n) for n, m in zip(lens, new)]).cuda()
    inside = (position >= 0) & (position < 30)
    want_q = s4.turned(q, turn, position.clamp(0, 29), False).to(dtype)
    assert torch.equal(got[inside], want_q[inside]) and (got[~inside] == 9.0).all()
    want_k, want_v = torch.zeros_like(kc), torch.zeros_like(vc)
    rk = s4.turned(k, turn, position.clamp(0, 29), False).to(dtype)
    for i in range(T):
        s = 0 if i < 20 else 1 if i < 37 else 2
        p = int(position[i])
        pg = int(table[s, p // page]) if 0 <= p < 30 else -1
        if 0 <= pg < 4:
            want_k[pg, :, p % page], want_v[pg, :, p % page] = rk[i], k[i]
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)


def test_in_place_strides_streams_and_graph(cq):
    """Slices of a fused projection, queries in place, on a stream that is not the current one, captured and replayed."""
    page, hkv, hq, d, dtype = 16, 2, 6, 128, torch.bfloat16
    new, lengths = [3, 50], [100, 50]
    T = sum(new)
    table, cu, lens, pages = _problem(new, lengths, page, 8)
    position, pg, slot = _place(table, new, lengths, page)
    turn = cq.rotary_table(128, d)
    fused = sq.normal((T, hq + 2 * hkv, d), dtype, 41)
    q, k, v = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    kc, vc, ks, vs = _caches("4bit", pages, hkv, page, d, dtype)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = cq.kv_cache_append(q, k, v, turn, kc, vc, table, cu, lens, k_scale=ks, v_scale=vs, stream=side)
    side.synchronize()
    assert torch.equal(got, s4.turned(q, turn, position, False).to(dtype))
    _check_cache("4bit", kc, ks, s4.turned(k, turn, position, False), pg, slot)
    own = q.contiguous()
    assert cq.kv_cache_append(own, k, v, turn, kc, vc, table, cu, lens, k_scale=ks, v_scale=vs, q_out=own) is own
    assert torch.equal(own, got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cq.kv_cache_append(q, k, v, turn, kc, vc, table, cu, lens, k_scale=ks, v_scale=vs)
    fused.copy_(sq.normal(fused.shape, dtype, 42))
    graph.replay()
    assert torch.equal(out, s4.turned(q, turn, position, False).to(dtype))
    _check_cache("4bit", vc, vs, v.float(), pg, slot)


def test_no_tokens(cq):
    kc, vc, ks, vs = _caches("4bit", 2, 2, 16, 64, torch.float16)
    z = torch.empty(0, 2, 64, dtype=torch.float16, device="cuda")
    ints = torch.zeros(2, dtype=torch.int32, device="cuda")
    got = cq.kv_cache_append(z, z, z, cq.rotary_table(4, 32), kc, vc, ints[:1, None], ints, ints[:1], k_scale=ks, v_scale=vs)
    assert got.shape == z.shape
    k, v = cq.kv_cache_read(kc, vc, ints[:1, None], ints, ints[:1], 0, torch.float16, k_scale=ks, v_scale=vs)
    assert k.shape == (0, 2, 64) and v.shape == (0, 2, 64)


@pytest.mark.parametrize("d", [64, 128])
def test_ties_under_the_largest_scale(cq, d):
    """Odd multiples of half of the largest scale, 61,440, go to the even whole number, and what lies past 7 of it is held there: groups whose largest is
    7 scales, and more, up to the type's largest."""
    page, half = 16, 61440.0 / 2
    x = torch.zeros(4, 1, d, dtype=torch.bfloat16, device="cuda")
    ties = torch.tensor([s * (2 * n + 1) * half for n in range(7) for s in (1, -1)], device="cuda")
    x[..., :14] = ties.to(x.dtype)
    assert torch.equal(x[0, 0, :14].float(), ties)  # (they are bf16 numbers)
    for i, top in enumerate((14 * half, 16 * half, 2.0 ** 100, float(torch.finfo(torch.bfloat16).max))):
        x[i, :, 31] = -top
    x[..., 32:64] = x[..., :32].flip(-1)
    kc, vc, ks, vs = _caches("4bit", 2, 1, page, d, x.dtype)
    table = torch.tensor([[1]], dtype=torch.int32, device="cuda")
    cu, lens = torch.tensor([0, 4], dtype=torch.int32, device="cuda"), torch.tensor([4], dtype=torch.int32, device="cuda")
    cq.kv_cache_write(x, x, kc, vc, table, cu, lens, k_scale=ks, v_scale=vs)
    code, byte, val = s4.quantise4(x)
    assert (byte[..., :2] == 247).all()
    want = torch.tensor([s * 2 * ((n + 1) // 2) * 61440.0 for n in range(7) for s in (1, -1)], dtype=torch.float64, device="cuda")
    assert torch.equal(val[0, 0, :14], want) and (val[:, 0, 31] == -7 * 61440.0).all()
    for cache, scale in ((kc, ks), (vc, vs)):
        assert torch.equal(cache[1, :, :4].transpose(0, 1), code) and torch.equal(scale[1, :, :4].transpose(0, 1), byte)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["same", "e4m3", "4bit"])
def test_read_without_a_position(cq, kind, dt, d):
    """Tokens before the first position, and behind the table's last, read as zeros from every kind of cache; the others as from a call without them."""
    page, hkv, dtype = 16, 3, sq.DT[dt]
    kc, vc, ks, vs = _caches(kind, 4, hkv, page, d, dtype)
    table = torch.tensor([[2], [1]], dtype=torch.int32, device="cuda")
    cu, lens = torch.tensor([0, 16, 32], dtype=torch.int32, device="cuda"), torch.tensor([16, 16], dtype=torch.int32, device="cuda")
    k, v = sq.normal((32, hkv, d), dtype, 3), sq.normal((32, hkv, d), dtype, 4)
    cq.kv_cache_write(k, v, kc, vc, table, cu, lens, k_scale=ks, v_scale=vs)
    every = cq.kv_cache_read(kc, vc, table, cu, lens, 32, dtype, k_scale=ks, v_scale=vs)
    # 10 tokens before and 5 of positions 0 .. 4; 4 of positions 12 .. 15 and 6 behind
    cu, lens = torch.tensor([0, 15, 25], dtype=torch.int32, device="cuda"), torch.tensor([5, 22], dtype=torch.int32, device="cuda")
    got = cq.kv_cache_read(kc, vc, table, cu, lens, 25, dtype, k_scale=ks, v_scale=vs, out=tuple(torch.full((25, hkv, d), 5.0, dtype=dtype, device="cuda") for _ in range(2)))
    for g, w in zip(got, every):
        assert (g[:10] == 0).all() and (g[19:] == 0).all()
        assert torch.equal(g[10:15], w[:5]) and torch.equal(g[15:19], w[28:])
