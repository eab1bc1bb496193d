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


@pytest.mark.parametrize("d,hkv", [(64, 4), (128, 2)])
def test_gradients_of_a_long_sequence_of_many_heads(cq, d, hkv):
    """32,768 tokens with 16 query heads a key head: equal scores, so that dv is the mean of dout over half a million rows."""
    n, group, dtype = 32768, 16, torch.float16
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.rand(n, group * hkv, d, generator=g, device="cuda").to(dtype)
    k = torch.zeros(n, hkv, d, dtype=dtype, device="cuda")
    v = torch.randn(n, hkv, d, generator=g, device="cuda").to(dtype)
    dout = ((torch.rand(n, group * hkv, d, generator=g, device="cuda") * 0.4 + 0.8) * (1 + torch.arange(d, device="cuda") / d)).to(dtype)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out, lse = cq.attention_packed(q, k, v, cu, causal=False, return_lse=True)
    dv = cq.attention_packed_backward(q, k, v, out, dout, lse, cu, causal=False)[2]
    torch.cuda.synchronize()
    assert cq.cqsa_device_error()[1] == 0
    ref = dout.reshape(n, hkv, group, d).sum((0, 2), dtype=torch.float64) / n
    for i in (0, 5, n // 2, n - 1):
        _drift(dv[i], ref, hkv * d, 1024, f"key {i}")


@pytest.mark.parametrize("lens,hq,hkv", [([5000, 300], 32, 1), ([6000, 10], 32, 8)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_gradients_with_running_sums(cq, lens, hq, hkv, d, dt):
    """Key tiles whose steps are more than a fold's, cut into ranges (the first sizes) and whole (the second): every gradient against
    the formula, dk and dv again bit by bit, and from a workspace that held NaN."""
    dtype, total = sq.DT[dt], sum(lens)
    q, k, v, g = (sq.normal((total, h, d), dtype, i, t) for i, h, t in ((1, hq, 1.0), (2, hkv, 1.5), (3, hkv, 1.0), (4, hq, 1.0)))
    cu = torch.tensor(sq.starts(lens), dtype=torch.int32, device="cuda")
    out, lse = cq.attention_packed(q, k, v, cu, return_lse=True)
    got = cq.attention_packed_backward(q, k, v, out, g, lse, cu)
    at = 0
    for n in lens:
        i = slice(at, at + n)
        ref, mass = sq.gradients(q[i], k[i], v[i], out[i], g[i], True)
        for name, x, r, m in zip(("dq", "dk", "dv"), got, ref, mass):
            sq.check_grad(x[i], r, m, dtype, f"{name} of {n} tokens")
        at += n
    need = cq.cqsa_attn_packed_bwd_workspace_size(len(lens), total, hq, hkv, d)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    again = [torch.empty_like(t) for t in (q, k, v)]
    cq.cqsa_attn_packed_bwd(q, k, v, 0, 0, 0, out, g, lse, *again, ws, need, cu, len(lens), total, hq, hkv, d, True, 0.0,
                            cq.dtype_code(dtype))
    assert torch.equal(again[1], got[1]) and torch.equal(again[2], got[2])
    torch.cuda.synchronize()
    assert cq.cqsa_device_error()[1] == 0


def test_running_sums_of_calls_at_once(cq):
    """Forward, backward and chunk calls whose running sums lie in the SMs' slots, on three streams at once: each gives what it gives
    alone."""
    d, hq, hkv, page, dtype = 128, 8, 2, 64, torch.float16
    n = [9000, 8200, 9500]
    q, k, v, g = ([sq.normal((m, h, d), dtype, 4 * i + j) for i, m in enumerate(n)] for j, h in enumerate((hq, hkv, hkv, hq)))
    cu = [torch.tensor([0, m], dtype=torch.int32, device="cuda") for m in n]
    out, lse = cq.attention_packed(q[1], k[1], v[1], cu[1], return_lse=True)
    pages = -(-n[2] // page)
    kc, vc = (torch.zeros(pages, hkv, page, d, dtype=dtype, device="cuda") for _ in range(2))
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    cq.kv_cache_write(k[2], v[2], kc, vc, table, cu[2], cu[2][1:])
    new = torch.tensor([0, 500], dtype=torch.int32, device="cuda")
    calls = [lambda s: [cq.attention_packed(q[0], k[0], v[0], cu[0], stream=s)],
             lambda s: list(cq.attention_packed_backward(q[1], k[1], v[1], out, g[1], lse, cu[1], stream=s)[1:]),
             lambda s: [cq.attention_paged(q[2][-500:], kc, vc, table, new, cu[2][1:], 500, 1, stream=s)]]
    want = [f(None) for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for i in range(20):
        got = [None] * 3
        for j in range(3):
            at = (i + j) % 3
            got[at] = calls[at](streams[at])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b)), f"pass {i}"
    assert cq.cqsa_device_error()[1] == 0
