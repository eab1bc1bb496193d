"""attention_paged's lengths of the caller on the GPU: any that are long enough give the result."""
import pytest
import torch

from tests import _seq as sq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cq():
    import exact_long_context_tcgen05_gb300 as m
    return m


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("most_new,most", [(2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31), (2 ** 32, 2 ** 32), (2 ** 32 + 1, 10 ** 15)])
def test_lengths_past_32_bits(cq, new, most_new, most):
    """A caller that has no tighter bound may name any: none may read as a small one and leave rows out."""
    d, page, dtype, n = 64, 16, torch.float16, 300
    ks, vs, kc, vc, table = sq.make_cache([n], 2, d, page, dtype, 3)
    q = sq.normal((new, 4, d), dtype, 4)
    cu, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, new], [n]))
    out, lse = cq.attention_paged(q, kc, vc, table, cu, lens, most_new, most, return_lse=True, out=torch.full_like(q, 7.0))
    torch.cuda.synchronize()
    assert cq.cqsa_device_error()[1] == 0
    ref, rl, mass = sq.attend(q, ks[0], vs[0], n - new, True)
    sq.check_out(out, ref, mass, dtype)
    sq.check_lse(lse, rl)


def test_negative_lengths(cq):
    d, dtype = 64, torch.float16
    _, _, kc, vc, table = sq.make_cache([20], 2, d, 16, dtype, 3)
    q = sq.normal((1, 4, d), dtype, 4)
    cu, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 1], [20]))
    for bad in ((-1, 20), (1, -1)):
        with pytest.raises(cq.CqsaError) as e:
            cq.attention_paged(q, kc, vc, table, cu, lens, *bad)
        assert e.value.status == cq.CQSA_ERR_INVALID
