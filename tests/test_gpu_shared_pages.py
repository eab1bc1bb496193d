"""Bounds of pages that several sequences share and fill to different slots: those of the longest, in any order and every time."""
import pytest
import torch

from tests import _seq as sq
from tests.test_gpu_selected import want_bounds

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cq():
    import exact_long_context_tcgen05_gb300 as m
    return m


@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("order", [0, 1, 2])
@pytest.mark.parametrize("n_seqs", [3, 200])
def test_page_that_two_sequences_fill(cq, d, page, order, n_seqs):
    """A sequence, another that went on from a place inside one of its pages, and shorter ones over the same pages, rebuilt together."""
    hkv, longest = 2, 5 * page - 3
    lengths = ([longest, 3 * page + 5, 3 * page + 1] + [1 + (i * 37) % (5 * page - 4) for i in range(n_seqs - 3)])
    shift = (0, 1, n_seqs // 2)[order]
    lengths = lengths[shift:] + lengths[:shift]
    kc = sq.normal((8, hkv, page, d), torch.float16, 3) * torch.arange(1, page + 1, device="cuda")[:, None].half()  # (every slot moves the bounds)
    table = torch.tensor([[6, 2, 7, 1, 4]] * n_seqs, dtype=torch.int32, device="cuda")
    cu, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (sq.starts(lengths), lengths))
    k = torch.cat([kc[int(p)].transpose(0, 1) for p in table[0]])[:longest].double()
    b, e = want_bounds(k, page)
    for _ in range(5):
        bounds = torch.zeros(8, hkv, 2, d, dtype=torch.int8, device="cuda"), torch.zeros(8, hkv, dtype=torch.uint8, device="cuda")
        cq.kv_page_bounds(kc, table, cu, lens, *bounds, longest)
        for i, p in enumerate(table[0].tolist()):
            assert torch.equal(bounds[0][p], b[i].to(torch.int8)) and torch.equal(bounds[1][p], (e[i] + 127).to(torch.uint8)), i


def test_new_tokens_of_one_of_them(cq):
    """A step of sequences that share whole pages and have their own last ones: the shared pages' bounds are left as they were."""
    d, page, hkv = 64, 16, 2
    kc = sq.normal((10, hkv, page, d), torch.float16, 3)
    table = torch.tensor([[1, 2, 3], [1, 2, 4], [1, 5, 6]], dtype=torch.int32, device="cuda")
    lengths = [40, 35, 17]
    cu, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 1, 2, 3], lengths))
    bounds = torch.full((10, hkv, 2, d), 99, dtype=torch.int8, device="cuda"), torch.full((10, hkv), 99, dtype=torch.uint8, device="cuda")
    cq.kv_page_bounds(kc, table, cu, lens, *bounds, 1)
    for s, (n, last) in enumerate(zip(lengths, (2, 2, 1))):
        pg = int(table[s, last])
        b, e = want_bounds(kc[pg].transpose(0, 1)[:n - last * page].double(), page)
        assert torch.equal(bounds[0][pg], b[0].to(torch.int8)) and torch.equal(bounds[1][pg], (e[0] + 127).to(torch.uint8))
    for pg in (0, 1, 2, 6, 7, 8, 9):
        assert (bounds[0][pg] == 99).all() and (bounds[1][pg] == 99).all()
