"""The calls for long contexts over pages far inside a cache, past 2^32 bytes of codes and 2^31 of bounds: the same bits as over the first ones."""
import pytest
import torch

from tests import _seq as sq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cq():
    import exact_long_context_tcgen05_gb300 as m
    return m


def _all_calls(cq, kind, n_pages, first, d=128, page=16, hq=32, hkv=8):
    """Prompts and tokens of two sequences whose pages begin at page `first` of a cache of n_pages, and everything that comes out of the calls."""
    dtype, lengths, new = torch.bfloat16, [700, 333], [128, 1]
    width, more = {"e4m3": (d, ()), "4bit": (d // 2, (d // 32,))}[kind]
    kc, vc = (torch.empty(n_pages, hkv, page, width, dtype=torch.uint8, device="cuda") for _ in range(2))
    scales = {x: torch.empty(n_pages, hkv, page, *more, dtype=torch.uint8, device="cuda") for x in ("k_scale", "v_scale")}
    bounds = torch.empty(n_pages, hkv, 2, d, dtype=torch.int8, device="cuda"), torch.empty(n_pages, hkv, dtype=torch.uint8, device="cuda")
    table = (first + torch.arange(2 * 44, dtype=torch.int32, device="cuda").reshape(2, 44)).contiguous()
    turn = cq.rotary_table(700, d)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    T = sum(lengths)
    q, k, v = sq.normal((T, hq, d), dtype, 3), sq.normal((T, hkv, d), dtype, 4), sq.normal((T, hkv, d), dtype, 5)
    cu, lens = ints(sq.starts(lengths)), ints(lengths)
    rq = cq.kv_cache_append(q, k, v, turn, kc, vc, table, cu, lens, **scales)
    cq.kv_page_bounds(kc, table, cu, lens, *bounds, 700, k_scale=scales["k_scale"])
    got = [rq, *cq.kv_cache_read(kc, vc, table, cu, lens, T, dtype, **scales), *(b[table.flatten().long()[:44 + 21]] for b in bounds)]
    one = torch.cat([rq[699:700], rq[-1:]])
    cu1 = ints([0, 1, 2])
    got += cq.attention_paged(one, kc, vc, table, cu1, lens, 1, 700, return_lse=True, **scales)
    some, cus = torch.cat([rq[700 - new[0]:700], rq[-1:]]), ints(sq.starts(new))
    for most in (700, 400000):  # (the longest that the caller names decides whether 4 bits are unpacked first)
        got += cq.attention_paged(some, kc, vc, table, cus, lens, new[0], most, return_lse=True, **scales)
    got += cq.attention_selected(one, kc, vc, table, cu1, lens, *bounds, 5, 700, return_lse=True, return_pages=True, **scales)
    got += cq.attention_selected(some, kc, vc, table, cus, lens, *bounds, 5, 700, return_lse=True, return_pages=True, **scales)
    torch.cuda.synchronize()
    assert cq.cqsa_device_error()[1] == 0
    return [x.clone() for x in got]


@pytest.mark.parametrize("kind", ["4bit", "e4m3"])
def test_far_pages(cq, kind):
    n_pages = 2 ** 20 + 200  # x 8 heads x 2 x 128 bytes of bounds; x 8 heads x 16 slots x 64 (128) bytes of codes
    near = _all_calls(cq, kind, 100, 3)
    far = _all_calls(cq, kind, n_pages, n_pages - 95)
    assert len(near) == len(far)
    for i, (a, b) in enumerate(zip(near, far)):
        assert torch.equal(a, b), i
    assert all(torch.isfinite(x.float()).all() for x in near)
    torch.cuda.empty_cache()
