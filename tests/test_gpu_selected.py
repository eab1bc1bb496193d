"""Bounds of pages, and attention over pages selected by them, on the GPU against their definitions in 64 bits."""
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


def whole(x, dims):
    """x as whole multiples (64 bits) of the smallest power of two, 2^-126 or more, under which all over `dims` are at most 127, and its exponent."""
    top = x.abs().amax(dims, keepdim=True)
    e = torch.full_like(top, -126.0)
    for k in range(-125, 122):
        e = torch.where(top > 127 * 2.0 ** (k - 1), torch.full_like(e, float(k)), e)
    return torch.round(x * torch.exp2(-e)), e


def make(kind, lengths, hkv, d, page, dtype, seed, alike=0.0):
    """A cache of that kind with NaN (16-bit) or NaN scales in its unused slots: k and v of each sequence in 64 bits, the cache's tensors, the
    table. `alike`: how much of a key its neighbours in a page share."""
    _, _, kc, vc, table = sq.make_cache(lengths, hkv, d, page, torch.float32 if kind != "same" else dtype, seed, fill=0.0, sharp=1.5)
    shift = sq.normal((kc.shape[0], hkv, 1, d), torch.float32, seed + 1) * alike
    kc = (kc.float() + shift).to(kc.dtype)
    used = torch.zeros(kc.shape[:3], dtype=torch.bool, device="cuda")
    for s, n in enumerate(lengths):
        t = torch.arange(n, device="cuda")
        if n:
            used[table[s].long()[t // page], :, t % page] = True
    if kind == "same":
        kval, vval = kc.double(), vc.double()
        kc[~used], vc[~used] = math.nan, math.nan
        scales = (None, None)
    else:
        f = sq.quantise if kind == "e4m3" else s4.quantise4
        (kc, ks, kval), (vc, vs, vval) = f(kc), f(vc)
        for c, z in ((kc, ks), (vc, vs)):
            c[~used] = 0x7f if kind == "e4m3" else 0
            z[~used] = 255
        scales = (ks, vs)
    kk, vv = [], []
    for s, n in enumerate(lengths):
        t = torch.arange(n, device="cuda")
        pg = table[s].long()[t // page] if n else t
        kk.append(kval[pg, :, t % page])
        vv.append(vval[pg, :, t % page])
    return kk, vv, kc, vc, *scales, table


def want_bounds(k, page):
    """Bounds [pages, Hkv, 2, d] and exponents [pages, Hkv] of one sequence's keys [n, Hkv, d] in 64 bits."""
    b, e = whole(torch.stack([torch.stack([x.amax(0), x.amin(0)], 1) for x in k.split(page)]), (-1, -2))
    return b, e[:, :, 0, 0]


def want_pages(q, k, page, first, n_select, hkv):
    """The choice for tokens q [n, Hq, d] at positions first..: [n][kv head] ascending lists of page indices."""
    if len(k) == 0:
        return [[[] for _ in range(hkv)] for _ in range(len(q))]
    b, e = want_bounds(k, page)
    val = b * torch.exp2(e)[:, :, None, None]
    w, we = whole(q.double(), -1)
    w = w * torch.exp2(we)
    out = []
    for i in range(q.shape[0]):
        row = []
        for g in range(hkv):
            own = (first + i) // page
            if first + i < 0:
                row.append([])
                continue
            x = w[i].reshape(hkv, -1, w.shape[-1])[g][:, None]  # [group, 1, d]
            score = torch.maximum(x * val[None, :own, g, 0], x * val[None, :own, g, 1]).sum(-1).amax(0).tolist()
            best = sorted(range(own), key=lambda p: (-score[p], p))[:n_select - 1]
            row.append(sorted(best) + [own])
        out.append(row)
    return out


def run(cq, q, kc, vc, ks, vs, table, new, lengths, n_select, most=None, update=True, bounds=None, **kw):
    cu = torch.tensor(sq.starts(new), dtype=torch.int32, device="cuda")
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    pages, hkv, page = kc.shape[:3]
    d = q.shape[2]
    if bounds is None:  # of whole sequences, as after their prompts
        bounds = (torch.zeros(pages, hkv, 2, d, dtype=torch.int8, device="cuda"), torch.zeros(pages, hkv, dtype=torch.uint8, device="cuda"))
        all_cu = torch.tensor(sq.starts(lengths), dtype=torch.int32, device="cuda")
        cq.kv_page_bounds(kc, table, all_cu, lens, *bounds, max(lengths), k_scale=ks)
    got = cq.attention_selected(q, kc, vc, table, cu, lens, *bounds, n_select, max(lengths) if most is None else most, k_scale=ks, v_scale=vs,
                                return_lse=True, return_pages=True, out=torch.full_like(q, 7.0), **kw)
    torch.cuda.synchronize()
    assert cq.cqsa_device_error()[1] == 0
    return *got, bounds


def check(out, lse, pages, q, ks, vs, new, lengths, n_select, page, kind):
    hkv = ks[0].shape[1]
    group = q.shape[1] // hkv
    p_err = {"same": 1.0, "e4m3": 1.0, "4bit": 2.0}[kind]
    p_type = q.dtype if kind == "same" else torch.float16
    at = 0
    for s, n in enumerate(new):
        chosen = want_pages(q[at:at + n], ks[s], page, lengths[s] - n, n_select, hkv) if n else []
        for i in range(n):
            for g in range(hkv):
                want = chosen[i][g]
                assert pages[at + i, g].tolist() == want + [-1] * (n_select - len(want)), (s, i, g)
                t = torch.tensor([p * page + j for p in want for j in range(page) if p * page + j <= lengths[s] - n + i], dtype=torch.long, device="cuda")
                heads = slice(g * group, (g + 1) * group)
                ref, rl, mass = sq.attend(q[at + i:at + i + 1, heads], ks[s][t][:, g:g + 1], vs[s][t][:, g:g + 1], 0, False)
                tol = 1.01 * (sq.U[q.dtype] * ref.abs() + (p_err * sq.U[p_type] + 2.0 ** -16) * mass) + 2.0 ** -24 + len(t) * 2.0 ** -30
                assert torch.isfinite(out[at + i, heads]).all()
                assert ((out[at + i:at + i + 1, heads].double() - ref).abs() <= tol).all(), (s, i, g)
                sq.check_lse(lse[heads, at + i:at + i + 1], rl)
        at += n
    assert (out[at:] == 7.0).all()


CASES = [
    # new tokens, lengths, Hq, Hkv, page, n_select
    ([1], [1], 1, 1, 16, 1),
    ([1], [700], 8, 2, 16, 5),
    ([1, 1, 1], [16, 17, 1000], 8, 2, 32, 1),
    ([1, 0, 1], [900, 77, 300], 5, 1, 64, 3),
    ([1] * 40, [1 + 17 * i for i in range(40)], 4, 2, 16, 7),
    ([3, 1, 6], [3, 129, 700], 12, 4, 16, 4),
    ([40], [300], 4, 2, 16, 6),                                       # a chunk: pages that its own tokens fill
    ([4, 2], [2, 40], 4, 2, 16, 3),                                   # tokens before the first position
    ([1, 1], [0, 40], 4, 2, 16, 3),
    ([1], [6000], 32, 1, 16, 100),                                    # 32 heads of a key head, hundreds of pages
    ([2], [1500], 9, 1, 256, 20),                                     # more than there are
]


@pytest.mark.parametrize("new,lengths,hq,hkv,page,n_select", CASES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind,dt", [("same", "f16"), ("same", "bf16"), ("e4m3", "f16"), ("4bit", "bf16"), ("4bit", "f16")])
def test_selected(cq, new, lengths, hq, hkv, page, n_select, d, kind, dt):
    dtype = sq.DT[dt]
    ks, vs, *cache = make(kind, lengths, hkv, d, page, dtype, 11 + len(new), 1.0)
    q = sq.normal((sum(new) + 2, hq, d), dtype, 3)
    out, lse, pages, _ = run(cq, q, *cache, new, lengths, n_select)
    check(out, lse, pages, q, ks, vs, new, lengths, n_select, page, kind)


@pytest.mark.parametrize("kind,dt", [("same", "f16"), ("same", "bf16"), ("e4m3", "bf16"), ("4bit", "f16")])
@pytest.mark.parametrize("page,d", [(16, 64), (64, 128), (256, 128)])
def test_bounds(cq, kind, dt, page, d):
    """Bounds of the pages that new tokens came into and of no others, of filled slots alone; keys of every size; a key that is not finite."""
    dtype, hkv = sq.DT[dt], 3
    new, lengths = [1, 70, 0, 300, 5], [1, 400, 90, 300, 1030]
    ks, vs, kc, vc, kse, vse, table = make(kind, lengths, hkv, d, page, dtype, 7)
    if kind == "same":
        by = torch.exp2(torch.randint(-14, 12, kc.shape[:2], generator=torch.Generator().manual_seed(1)).float()).cuda()
        kc *= by[:, :, None, None].to(dtype)
        ks = [torch.cat([kc[int(table[s, p])].transpose(0, 1) for p in range(-(-n // page))])[:n].double() for s, n in enumerate(lengths)]
    bad = int(table[1, 399 // page])
    if kind == "same":
        kc[bad, 1, 399 % page, 5] = math.inf
    else:
        kse[bad, 1, 399 % page] = 255
        if kind == "e4m3":
            kc[bad, 1, 399 % page, 0] = 0x7f
    bounds = torch.full((kc.shape[0], hkv, 2, d), 99, dtype=torch.int8, device="cuda")
    exps = torch.full((kc.shape[0], hkv), 99, dtype=torch.uint8, device="cuda")
    cu, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (sq.starts(new), lengths))
    want_b, want_e = bounds.clone(), exps.clone()
    for s, n in enumerate(new):
        b, e = want_bounds(ks[s], page)
        for p in range((lengths[s] - n) // page, -(-lengths[s] // page) if n else 0):
            want_b[int(table[s, p])], want_e[int(table[s, p])] = b[p].to(torch.int8), (e[p] + 127).to(torch.uint8)
    want_b[bad, 1], want_e[bad, 1] = 0, 255
    for most in (1, max(new), 2 ** 40):  # (it only sets the split)
        now_b, now_e = bounds.clone(), exps.clone()
        cq.kv_page_bounds(kc, table, cu, lens, now_b, now_e, most, k_scale=kse)
        assert torch.equal(now_e, want_e) and torch.equal(now_b, want_b)


def test_equal_scores(cq):
    """Of equal scores the first pages are chosen; a page whose key is not finite comes first of all."""
    d, page, hkv, n = 64, 16, 1, 16 * 40 + 3
    k = sq.normal((1, 1, page, d), torch.float16, 3)
    kc = k.expand(41, 1, page, d).contiguous()
    vc = sq.normal(kc.shape, torch.float16, 4)
    table = torch.randperm(41, generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()[None]
    q = sq.normal((1, 4, d), torch.float16, 5)
    out, lse, pages, bounds = run(cq, q, kc, vc, None, None, table, [1], [n], 9)
    assert pages[0, 0].tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 40]
    bounds[1][int(table[0, 30])] = 255
    bounds[1][int(table[0, 7])] += 1  # twice the score, or half where it is negative
    _, _, pages, _ = run(cq, q, kc, vc, None, None, table, [1], [n], 5, bounds=bounds)
    b, e = want_bounds(k[0, 0][:, None], page)
    w, we = whole(q[0].double(), -1)
    top = (torch.maximum(w[:, None] * b[None, 0, 0, 0], w[:, None] * b[None, 0, 0, 1]).sum(-1) * torch.exp2(we[:, 0])[:, None]).max().item()
    assert pages[0, 0].tolist() == ([0, 1, 7, 30, 40] if top > 0 else [0, 1, 2, 30, 40])


def test_many_pages_and_extremes(cq):
    """A choice among tens of thousands of pages, scores of both signs and many equal ones, against a stable sort."""
    d, page, hkv, P = 64, 16, 2, 40000
    g = torch.Generator(device="cuda").manual_seed(5)
    bounds = torch.randint(-3, 4, (P + 1, hkv, 2, d), generator=g, device="cuda").to(torch.int8)
    exps = torch.randint(126, 129, (P + 1, hkv), generator=g, device="cuda").to(torch.uint8)
    kc = torch.randn(P + 1, hkv, page, d, generator=g, device="cuda").half()
    table = torch.randperm(P + 1, generator=g, device="cuda").to(torch.int32)[None].contiguous()
    q = torch.randint(-2, 3, (2, 6, d), generator=g, device="cuda").half()
    q[:, :, 0] = 127.0  # one power of two for all
    n = P * page + 2
    cu, lens = torch.tensor([0, 2], dtype=torch.int32, device="cuda"), torch.tensor([n], dtype=torch.int32, device="cuda")
    b = bounds[table[0, :P].long()].float()
    unit = torch.exp2(exps[table[0, :P].long()].float() - 127)
    for n_select in (1, 2, 33, 5000, P, P + 1, P + 5):
        _, pages = cq.attention_selected(q, kc, kc, table, cu, lens, bounds, exps, n_select, n, return_pages=True)
        for i in range(2):
            for h in range(hkv):
                x = q[i, h * 3:h * 3 + 3].float()
                score = (x.clamp(min=0) @ b[:, h, 0].T + x.clamp(max=0) @ b[:, h, 1].T).amax(0) * unit[:, h]
                best = torch.sort(score, dim=0, descending=True, stable=True)[1][:n_select - 1].sort()[0].int()
                want = torch.full((n_select,), -1, dtype=torch.int32, device="cuda")
                want[:len(best)], want[len(best)] = best, P
                assert torch.equal(pages[i, h], want), (n_select, i, h)
    # pages that begin at max_kv_len or behind are not selected, but for the token's own
    _, pages = cq.attention_selected(q, kc, kc, table, cu, lens, bounds, exps, 12, 10 * page, return_pages=True)
    assert (pages == torch.tensor(list(range(10)) + [P, -1], dtype=torch.int32, device="cuda")).all()


@pytest.mark.parametrize("kind", ["same", "4bit"])
def test_step_by_step(cq, kind):
    """Tokens appended one step at a time with their rotation, their pages' bounds kept up, attended over a selection: the same choice and results as
    from bounds of the whole sequence, and as full attention while every page is chosen."""
    d, page, hq, hkv, dtype, start, steps = 128, 16, 8, 2, torch.bfloat16, 250, 40
    turn = cq.rotary_table(400, d)
    total = start + steps
    q, k, v = (sq.normal((total, h, d), dtype, 60 + h) for h in (hq, hkv, hkv))
    table = torch.randperm(24, generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()[None, :20].contiguous()
    if kind == "same":
        kc, vc, scales = *(torch.zeros(24, hkv, page, d, dtype=dtype, device="cuda") for _ in range(2)), {}
    else:
        kc, vc = (torch.zeros(24, hkv, page, d // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
        scales = {x: torch.zeros(24, hkv, page, d // 32, dtype=torch.uint8, device="cuda") for x in ("k_scale", "v_scale")}
    bounds = torch.zeros(24, hkv, 2, d, dtype=torch.int8, device="cuda"), torch.zeros(24, hkv, dtype=torch.uint8, device="cuda")
    ks = scales.get("k_scale")

    def step(a, b):
        cu, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, b - a], [b]))
        rq = cq.kv_cache_append(q[a:b], k[a:b], v[a:b], turn, kc, vc, table, cu, lens, **scales)
        cq.kv_page_bounds(kc, table, cu, lens, *bounds, b - a, k_scale=ks)
        return rq, cu, lens

    step(0, start)
    for t in range(start, total):
        rq, cu, lens = step(t, t + 1)
        few = cq.attention_selected(rq, kc, vc, table, cu, lens, *bounds, 4, t + 1, return_lse=True, return_pages=True, **scales)
        fresh = tuple(torch.zeros_like(x) for x in bounds)
        cq.kv_page_bounds(kc, table, torch.tensor([0, t + 1], dtype=torch.int32, device="cuda"), lens, *fresh, t + 1, k_scale=ks)
        again = cq.attention_selected(rq, kc, vc, table, cu, lens, *fresh, 4, 400, return_lse=True, return_pages=True, **scales)
        assert all(torch.equal(x, y) for x, y in zip(few, again))
        every, lse, pages = cq.attention_selected(rq, kc, vc, table, cu, lens, *bounds, 20, t + 1, return_lse=True, return_pages=True, **scales)
        full, flse = cq.attention_paged(rq, kc, vc, table, cu, lens, 1, t + 1, return_lse=True, **scales)
        # two splits of the same sums: a rounding of the result each, and their probabilities' roundings
        assert (every.double() - full.double()).abs().max() <= 2.0 ** -6 and (lse - flse).abs().max() <= 2.0 ** -15
        assert pages[0, 0].tolist() == list(range(t // page + 1)) + [-1] * (20 - t // page - 1)


def test_graph_and_streams(cq):
    """Captured and replayed beside an eager call on another stream, for lengths that change between replays."""
    d, page, lengths, dtype = 64, 16, [1000, 333, 64], torch.float16
    ks, vs, *cache = make("4bit", lengths, 2, d, page, dtype, 41, 1.0)
    q, other = sq.normal((3, 8, d), dtype, 4), sq.normal((3, 8, d), dtype, 5)
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    _, _, _, bounds = run(cq, q, *cache, [1, 1, 1], lengths, 4)
    args = (cache[0], cache[1], cache[4], cu, lens, *bounds, 4, 1000)
    kw = {"k_scale": cache[2], "v_scale": cache[3], "return_lse": True, "return_pages": True}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = cq.attention_selected(q, *args, **kw)
    for now in (lengths, [17, 333, 1], [1000, 2, 63]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        eager = cq.attention_selected(other, *args, stream=side, **kw)
        graph.replay()
        torch.cuda.synchronize()
        for (o, l, p), x in ((got, q), (eager, other)):
            kn, vn = [k[:n] for k, n in zip(ks, now)], [v[:n] for v, n in zip(vs, now)]
            pad = torch.full((1, 8, d), 7.0, dtype=dtype, device="cuda")
            check(torch.cat([o, pad]), l, p, x, kn, vn, [1, 1, 1], now, 4, page, "4bit")


def test_no_tokens_and_refusals(cq):
    d, page = 64, 16
    _, _, kc, vc, _, _, table = make("same", [40], 2, d, page, torch.float16, 3)
    z = torch.empty(0, 4, d, dtype=torch.float16, device="cuda")
    cu, lens = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.tensor([40], dtype=torch.int32, device="cuda")
    bounds = torch.zeros(kc.shape[0], 2, 2, d, dtype=torch.int8, device="cuda"), torch.zeros(kc.shape[0], 2, dtype=torch.uint8, device="cuda")
    cq.kv_page_bounds(kc, table, cu, lens, *bounds, 0)
    assert (bounds[1] == 0).all()
    out, pages = cq.attention_selected(z, kc, vc, table, cu, lens, *bounds, 3, 40, return_pages=True)
    assert out.shape == z.shape and pages.shape == (0, 2, 3)
    q = sq.normal((1, 4, d), torch.float16, 3)
    for f in (lambda: cq.attention_selected(q, kc, vc, table, cu, lens, *bounds, 0, 40), lambda: cq.attention_selected(q, kc, vc, table, cu, lens, *bounds, 2 ** 21, 40),
              lambda: cq.attention_selected(q, kc, vc, table, cu, lens, bounds[0][:1], bounds[1], 3, 40),
              lambda: cq.attention_selected(q, kc, vc, table, cu, lens, bounds[0].int(), bounds[1], 3, 40),
              lambda: cq.kv_page_bounds(kc, table, cu, lens, bounds[0], bounds[1][:, :1], 1),
              lambda: cq.attention_selected(q, kc, vc, table, cu, lens, *bounds, 3, 40, k_scale=bounds[1])):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(cq.CqsaError):
        cq.attention_selected(q, kc, vc, table, cu, lens, *bounds, 3, -1)


@pytest.mark.parametrize("P", [1, 2, 31, 33, 255, 257, 1000, 5000, 11200, 16383, 16384, 20000])
def test_choice_against_a_sort(cq, P):
    """Choices of every kind of size among P pages whose scores have many equal values, one sign, or hardly any bits in common."""
    d, page, g = 64, 16, torch.Generator(device="cuda").manual_seed(P)
    kc = torch.zeros(P + 1, 1, page, d, dtype=torch.float16, device="cuda")
    table = torch.arange(P + 1, dtype=torch.int32, device="cuda")[None].contiguous()
    q = torch.zeros(1, 1, d, dtype=torch.float16, device="cuda")
    q[..., 0] = 1.0  # a page's score is its first bound, largest key
    cu, lens = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([P * page + 1], dtype=torch.int32, device="cuda")
    for kind in range(4):
        bounds = torch.zeros(P + 1, 1, 2, d, dtype=torch.int8, device="cuda")
        exps = torch.full((P + 1, 1), 127, dtype=torch.uint8, device="cuda")
        if kind == 0:
            bounds[..., 0] = torch.randint(-2, 3, (P + 1, 1, 1), generator=g, device="cuda").to(torch.int8)
        elif kind == 1:
            bounds[..., 0] = torch.randint(1, 128, (P + 1, 1, 1), generator=g, device="cuda").to(torch.int8)
        elif kind == 2:
            bounds[..., 0] = torch.randint(-127, 128, (P + 1, 1, 1), generator=g, device="cuda").to(torch.int8)
            exps = torch.randint(60, 190, (P + 1, 1), generator=g, device="cuda").to(torch.uint8)
        score = bounds[:P, 0, 0, 0].double() * torch.exp2(exps[:P, 0].double() - 127)
        for n_select in sorted({1, 2, P // 2 + 1, P, P + 1, P + 2}):
            _, pages = cq.attention_selected(q, kc, kc, table, cu, lens, bounds, exps, n_select, P * page + 1, return_pages=True)
            best = torch.sort(score, dim=0, descending=True, stable=True)[1][:n_select - 1].sort()[0].int()
            want = torch.full((n_select,), -1, dtype=torch.int32, device="cuda")
            want[:len(best)], want[len(best)] = best, P
            assert torch.equal(pages[0, 0], want), (kind, n_select)


@pytest.mark.parametrize("width,hkv", [(16384, 8), (300000, 2)])
def test_tokens_in_rounds(cq, width, hkv):
    """More scores than are held at a time (64 MiB: 128 tokens, 27 tokens), so that rounds begin and end inside of sequences: the same as in one round."""
    d, page, dtype, lengths, new = 64, 16, torch.float16, [900, 333, 64, 2000], [150, 1, 30, 120]
    ks, vs, kc, vc, kscale, vscale, table = make("4bit", lengths, hkv, d, page, dtype, 7, 1.0)
    q = sq.normal((sum(new) + 2, 2 * hkv, d), dtype, 3)
    assert sum(new) > (64 << 20) // (hkv * width * 4)
    out, lse, pages, bounds = run(cq, q, kc, vc, kscale, vscale, table, new, lengths, 6)
    check(out, lse, pages, q, ks, vs, new, lengths, 6, page, "4bit")
    wide = torch.zeros(len(lengths), width, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    again = run(cq, q, kc, vc, kscale, vscale, wide, new, lengths, 6, most=width * page, bounds=bounds)
    n = sum(new)
    assert torch.equal(out, again[0]) and torch.equal(lse[:, :n], again[1][:, :n]) and torch.equal(pages[:n], again[2][:n])
