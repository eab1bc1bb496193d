"""Sequences whose lengths pass what their row of the page table holds: every call gives a token the same position, kv_lens[s] - n + i, and those behind the
table see all of it."""
import pytest
import torch

from tests import _seq as sq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cq():
    import exact_long_context_tcgen05_gb300 as m
    return m


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _filled(cq, kind, dtype, hkv, d, page, room, new, lengths, hq):
    """Caches that hold `room` positions of each sequence, filled up to the new tokens by a write and with the new tokens by an append, both of which skip what is
    behind the table; the rotated queries, and the keys and values that the cache stands for."""
    pages = room // page
    width, more = {"same": (d, None), "e4m3": (d, ()), "4bit": (d // 2, (d // 32,))}[kind]
    kc, vc = (torch.zeros(len(new) * pages, hkv, page, width, dtype=dtype if kind == "same" else torch.uint8, device="cuda") for _ in range(2))
    scales = {} if kind == "same" else {x: torch.zeros(len(new) * pages, hkv, page, *more, dtype=torch.uint8, device="cuda") for x in ("k_scale", "v_scale")}
    table = torch.randperm(len(new) * pages, generator=torch.Generator().manual_seed(3)).view(len(new), pages).to(torch.int32).cuda()
    old = [n - m for n, m in zip(lengths, new)]
    k, v = (sq.normal((sum(old), hkv, d), dtype, s) for s in (1, 2))
    cq.kv_cache_write(k, v, kc, vc, table, _ints(sq.starts(old)), _ints(old), **scales)
    q, k, v = (sq.normal((sum(new), h, d), dtype, 5 + i) for i, h in enumerate((hq, hkv, hkv)))
    rq = cq.kv_cache_append(q, k, v, cq.rotary_table(max(lengths), d), kc, vc, table, _ints(sq.starts(new)), _ints(lengths), **scales)
    held = [min(n, room) for n in lengths]
    kk, vv = (x.double().split(held) for x in cq.kv_cache_read(kc, vc, table, _ints(sq.starts(held)), _ints(held), sum(held), dtype, **scales))
    return rq, kc, vc, scales, table, kk, vv


def _near(out, lse, q, k, v, first, kind):
    """Rows of one sequence, the first at position `first` of the keys given."""
    ref, rl, mass = sq.attend(q, k, v, first, True)
    up = max(sq.U[q.dtype], 2.0 ** -10) if kind == "4bit" else max(sq.U[q.dtype], 2.0 ** -11)
    tol = 1.01 * (sq.U[q.dtype] * ref.abs() + (up + 2.0 ** -16) * mass) + 2.0 ** -24 + len(k) * 2.0 ** -25
    assert ((out.double() - ref).abs() <= tol).all()
    sq.check_lse(lse, rl)


CASES = [
    # positions that the table has room for, new tokens, lengths
    (64, [4, 2], [66, 40]),                # tokens on both sides of the table's end
    (64, [3, 1, 2], [70, 64, 65]),         # all behind it, the last slot, one each
    (1024, [1, 5], [1100, 1024]),
    (512, [300, 40, 1], [700, 513, 500]),  # chunks
    (256, [700, 200], [1000, 2000]),       # a chunk that passes the whole table, one behind it
]


@pytest.mark.parametrize("room,new,lengths", CASES)
@pytest.mark.parametrize("kind,dt", [("same", "bf16"), ("e4m3", "f16"), ("4bit", "f16"), ("4bit", "bf16")])
@pytest.mark.parametrize("d,hq", [(64, 4), (128, 8)])
def test_append_past_the_table_then_attend(cq, room, new, lengths, kind, dt, d, hq):
    hkv, page = 2, 16
    q, kc, vc, scales, table, ks, vs = _filled(cq, kind, sq.DT[dt], hkv, d, page, room, new, lengths, hq)
    for most in (max(lengths), 1, 200_000):
        out, lse = cq.attention_paged(q, kc, vc, table, _ints(sq.starts(new)), _ints(lengths), max(new), most, return_lse=True, **scales)
        torch.cuda.synchronize()
        assert cq.cqsa_device_error()[1] == 0
        at = 0
        for s, n in enumerate(new):
            _near(out[at:at + n], lse[:, at:at + n], q[at:at + n], ks[s], vs[s], lengths[s] - n, kind)
            at += n


@pytest.mark.parametrize("room,new,lengths", CASES[:3] + [(256, [50, 20], [280, 400])])
@pytest.mark.parametrize("kind,dt", [("same", "bf16"), ("e4m3", "f16"), ("4bit", "f16")])
@pytest.mark.parametrize("hq", [4, 18])
def test_selected_pages(cq, room, new, lengths, kind, dt, hq):
    """A token's own page is the one of its position, or the table's last; bounds are of the pages with new tokens and of no others."""
    d, hkv, page = 64, 2, 16
    q, kc, vc, scales, table, ks, vs = _filled(cq, kind, sq.DT[dt], hkv, d, page, room, new, lengths, hq)
    pages = table.numel()
    held, cu, lens = [min(n, room) for n in lengths], _ints(sq.starts(new)), _ints(lengths)

    def bounds_of(at, kl, most, fill=0):
        b = torch.full((pages, hkv, 2, d), fill, dtype=torch.int8, device="cuda"), torch.full((pages, hkv), fill, dtype=torch.uint8, device="cuda")
        cq.kv_page_bounds(kc, table, at, kl, *b, most, k_scale=scales.get("k_scale"))
        return b

    whole = bounds_of(_ints(sq.starts(held)), _ints(held), room)
    part = bounds_of(cu, lens, max(new), 99)
    for s, n in enumerate(new):
        first = max(lengths[s] - n, 0) // page
        for p in range(room // page):
            pg = int(table[s, p])
            if first <= p <= (held[s] - 1) // page:
                assert torch.equal(part[0][pg], whole[0][pg]) and torch.equal(part[1][pg], whole[1][pg]), (s, p)
            else:
                assert (part[0][pg] == 99).all() and (part[1][pg] == 99).all(), (s, p)
    for n_select in (1, room // page):
        out, lse, chosen = cq.attention_selected(q, kc, vc, table, cu, lens, *whole, n_select, max(lengths), return_lse=True, return_pages=True, **scales)
        torch.cuda.synchronize()
        assert cq.cqsa_device_error()[1] == 0
        at = 0
        for s, n in enumerate(new):
            last = [min(lengths[s] - n + i, room - 1) for i in range(n)]
            own = _ints([p // page for p in last])
            begin = own if n_select == 1 else torch.zeros_like(own)
            want = torch.where(begin[:, None] + _ints(list(range(n_select))) <= own[:, None], begin[:, None] + _ints(list(range(n_select))), -1)
            assert torch.equal(chosen[at:at + n], want[:, None].expand(n, hkv, n_select))
            for i, p in enumerate(last):
                a = int(begin[i]) * page
                _near(out[at + i:at + i + 1], lse[:, at + i:at + i + 1], q[at + i:at + i + 1], ks[s][a:], vs[s][a:], p - a, kind)
            at += n
