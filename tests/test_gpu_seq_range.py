"""Values near the end of bf16's range on the GPU: the calls over sequences are exact while a value's magnitude times the positions stays below
2^113, as the header says."""
import pytest
import torch

from tests import _seq as sq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cq():
    import exact_long_context_tcgen05_gb300 as m
    return m


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [100, -100])
def test_large_and_small_values(cq, d, power):
    n, hq, hkv, page, dtype = 1000, 8, 2, 16, torch.bfloat16
    q, k = sq.normal((n, hq, d), dtype, 1), sq.normal((n, hkv, d), dtype, 2)
    v = (sq.normal((n, hkv, d), torch.float64, 3).clamp(-4, 4) * 2.0 ** power).to(dtype)  # times 1,000 positions: below 2^112
    ref, rl, mass = sq.attend(q, k, v, 0, True)

    def check(out, lse, i, p_dtype=dtype):
        # scaled by the power, exactly, so that check_out's absolute term is small beside the values
        sq.check_out(out.double() * 2.0 ** -power, ref[i] * 2.0 ** -power, mass[i] * 2.0 ** -power, dtype, p_dtype)
        sq.check_lse(lse, rl[:, i])

    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out, lse = cq.attention_packed(q, k, v, cu, return_lse=True)
    check(out, lse, slice(0, n))
    kc, vc = (torch.zeros(63, hkv, page, d, dtype=dtype, device="cuda") for _ in range(2))
    table = torch.arange(63, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    cq.kv_cache_write(k, v, kc, vc, table, cu, lens)
    for new in (1, 4, 60):
        i = slice(n - new, n)
        out, lse = cq.attention_paged(q[i], kc, vc, table, torch.tensor([0, new], dtype=torch.int32, device="cuda"), lens, new, n, return_lse=True)
        check(out, lse, i)
    torch.cuda.synchronize()
    assert cq.cqsa_device_error()[1] == 0
