"""The ends of the types' ranges in an e4m3 cache on the GPU: what was written finite is read back finite."""
import pytest
import torch

from tests import _seq as sq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cq():
    import exact_long_context_tcgen05_gb300 as m
    return m


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_largest_values(cq, dt, d):
    """Vectors whose largest value is at, or a little below, the type's largest: e4m3 rounds some of them up past it."""
    dtype, hkv, page, n = sq.DT[dt], 2, 16, 40
    top = torch.finfo(dtype).max
    x = sq.normal((n, hkv, d), torch.float64, 1).clamp(-4, 4) / 4 * top  # (64 bits: the products are exact)
    part = torch.linspace(0.9, 1.0, n, dtype=torch.float64, device="cuda")
    x[:, 0, 3], x[:, 1, d - 1] = top * part, -top * part
    k = x.to(dtype)
    k[5, 0, 1], k[6, 1, 2] = float("inf"), float("nan")
    v = -k
    kc, vc = (torch.zeros(3, hkv, page, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    scales = {name: torch.zeros(3, hkv, page, dtype=torch.uint8, device="cuda") for name in ("k_scale", "v_scale")}
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    cu, lens = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in ([0, n], [n]))
    cq.kv_cache_write(k, v, kc, vc, table, cu, lens, **scales)
    for got, src in zip(cq.kv_cache_read(kc, vc, table, cu, lens, n, dtype, **scales), (k, v)):
        want = sq.quantise(src)[2].clamp(-top, top)  # (NaN stays)
        assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.isnan(want).sum() == 2
        assert torch.equal(torch.nan_to_num(got.double(), 0.0), torch.nan_to_num(want, 0.0))  # multiples of the step: exact in 16 bits
        assert (got.double().abs() == top).any()  # some were held
