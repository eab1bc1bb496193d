"""Sums over very many keys or queries on the GPU: the tensor core truncates as it accumulates, so the kernels fold their
accumulators into fp32 sums. Same-sign terms show the drift that is left as a mean signed error, in which roundings cancel."""
import math

import pytest
import torch

from tests import _seq as sq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cq():
    import exact_long_context_tcgen05_gb300 as m
    return m


def _drift(got, ref, n, products, what):
    """The mean relative error of n independent results whose sums are folded every `products` products. A product adds 16 terms to
    the sum; each is cut off at a quarter of the sum's last place and the sum at its last place (that loses 2.5 places on average, as
    unfolded sums measured do), at most 16 / 4 + 1 places of at most 2^-23 each. Over a growing sum of one sign that is at most
    products / 2 * 5 * 2^-23 of the result. Rounding the result is off by at most u either way, evenly where the results are spread over
    an octave: a deviation of u / sqrt(3 n) for the mean, taken six times. What rounding probabilities to 16 bits and fp32 sums
    shift the mean by is far less: 2^-18 together."""
    err = ((got.double() - ref) / ref).mean().item()
    bound = products / 2 * 5 * 2.0 ** -23 + 6 * sq.U[got.dtype] / math.sqrt(3 * n) + 2.0 ** -18
    assert abs(err) <= bound, f"{what}: mean relative error {err:.2e}, bound {bound:.2e}"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cache", ["same", "e4m3"])
def test_tokens_over_a_very_long_context(cq, cache, d):
    """One token each of sequences with 2^21 positions (their pages are shared), so many that a CTA takes whole ones alone."""
    n, page, hq, dtype, n_seqs = 1 << 21, 256, 4, torch.float16, 608
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn(n // page, 1, page, d, generator=g, device="cuda") * 0.02
    # values of one sign, of another size for each feature
    v = (torch.rand(n // page, 1, page, d, generator=g, device="cuda") * 0.4 + 0.8) * (1 + torch.arange(d, device="cuda") / d)
    q = torch.randn(1, hq, d, generator=g, device="cuda").to(dtype)
    scales = {}
    if cache == "e4m3":
        # one power of two for all vectors, so that codes and their 64-bit values are plain casts
        kc, vc = (x.mul(128).to(torch.float8_e4m3fn) for x in (k, v))
        keys, values = kc.double() / 128, vc.double() / 128
        kc, vc = kc.view(torch.uint8), vc.view(torch.uint8)
        scales = {name: torch.full(k.shape[:3], 127 - 7, dtype=torch.uint8, device="cuda") for name in ("k_scale", "v_scale")}
    else:
        kc, vc = k.to(dtype), v.to(dtype)
        keys, values = kc.double(), vc.double()
    table = torch.arange(n // page, dtype=torch.int32, device="cuda")[None].repeat(n_seqs, 1)
    cu = torch.arange(n_seqs + 1, dtype=torch.int32, device="cuda")
    lens = torch.full((n_seqs,), n, dtype=torch.int32, device="cuda")
    out, lse = cq.attention_paged(q.repeat(n_seqs, 1, 1), kc, vc, table, cu, lens, 1, n, return_lse=True, **scales)
    torch.cuda.synchronize()
    assert cq.cqsa_device_error()[1] == 0
    s = q[0].double() @ keys.reshape(n, d).T / math.sqrt(d)
    rl = torch.logsumexp(s, -1)
    ref = torch.exp(s - rl[:, None]) @ values.reshape(n, d)
    # whole units, and units that two ranges share
    for i in (0, 1, n_seqs // 2, n_seqs - 1):
        _drift(out[i], ref, hq * d, 256, f"sequence {i}")
        # a sum of n fp32 terms in no more than n / 16 steps a lane, each rounded at random: far less than 2^-16
        assert (lse[:, i].double() - rl).abs().max().item() <= 2.0 ** -15
