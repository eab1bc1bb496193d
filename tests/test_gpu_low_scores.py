"""Rows whose scores are all far below zero on the GPU: a softmax does not depend on where its scores lie, so they are as exact as any others."""
import math

import pytest
import torch

from tests import _seq as sq

pytestmark = pytest.mark.gpu
SCALE = 0.125


@pytest.fixture(scope="module")
def cq():
    import exact_long_context_tcgen05_gb300 as m
    return m


def _problem(n, hq, hkv, d, dtype):
    """Scores between -160 and -330 that are exact in fp32: q and k are small whole numbers of opposite sign."""
    g = torch.Generator().manual_seed(n)
    q = torch.randint(3, 5, (n, hq, d), generator=g)
    k = -torch.full((n, hkv, d), 10 * 64 // d) - torch.randint(0, 2, (n, hkv, d), generator=g) * (torch.arange(d) < 4)
    return q.to(dtype).cuda(), k.to(dtype).cuda(), sq.normal((n, hkv, d), dtype, 3)


def _check(out, lse, ref, rl, mass, dtype, p_dtype=None, what=""):
    sq.check_out(out, ref, mass, dtype, p_dtype, what, 2.0 ** -20)
    # the score in base 2 is up to 480, off by the fp32 factor's half step and its own, and the result's: 3 * 480 * 2^-24 < 2^-13
    assert (lse.double() - rl).abs().max().item() <= 2.0 ** -13, what


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("causal", [True, False])
def test_packed_and_paged(cq, causal, dt, d):
    dtype, n, hq, hkv, page = sq.DT[dt], 333, 8, 2, 16
    q, k, v = _problem(n, hq, hkv, d, dtype)
    ref, rl, mass = sq.attend(q, k, v, 0, causal, SCALE)
    assert rl.max().item() < -150  # 2^-216 and less beside a score of zero
    cu, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n], [n]))
    out, lse = cq.attention_packed(q, k, v, cu, causal=causal, scale=SCALE, return_lse=True)
    _check(out, lse, ref, rl, mass, dtype, what="packed")
    pages = -(-n // page)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    for kind in (dtype, torch.uint8):
        kc, vc = (torch.zeros(pages, hkv, page, d, dtype=kind, device="cuda") for _ in range(2))
        scales = {} if kind == dtype else {x: torch.zeros(pages, hkv, page, dtype=torch.uint8, device="cuda") for x in ("k_scale", "v_scale")}
        cq.kv_cache_write(k, v, kc, vc, table, cu, lens, **scales)
        if kind == torch.uint8:  # whole numbers up to 16 are exact in e4m3, the values are not
            values = sq.quantise(v)[2]
            ref, rl, mass = sq.attend(q, k, values, 0, causal, SCALE)
        for new in (1, 4, n):
            i = slice(n - new, n)
            out, lse = cq.attention_paged(q[i], kc, vc, table, torch.tensor([0, new], dtype=torch.int32, device="cuda"), lens, new, n,
                                          causal=causal, scale=SCALE, return_lse=True, **scales)
            _check(out, lse, ref[i], rl[:, i], mass[i], dtype, torch.float16 if scales else dtype, f"{kind}, {new} tokens")
    torch.cuda.synchronize()
    assert cq.cqsa_device_error()[1] == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("causal", [True, False])
def test_dense(cq, causal, dt, d):
    """The call on [B, H, N, d] tensors, forward and backward."""
    dtype, n, h = sq.DT[dt], 333, 4
    q, k, v = _problem(n, h, h, d, dtype)
    g = sq.normal((n, h, d), dtype, 4)
    x = [t.transpose(0, 1)[None].contiguous() for t in (q, k, v, g)]
    out, lse = cq.attention(*x[:3], causal=causal, scale=SCALE, return_lse=True)
    ref, rl, mass = sq.attend(q, k, v, 0, causal, SCALE)
    _check(out[0].transpose(0, 1), lse[0], ref, rl, mass, dtype)
    got = cq.attention_backward(*x[:3], out, x[3], lse, causal=causal, scale=SCALE)
    torch.cuda.synchronize()
    assert cq.cqsa_device_error()[1] == 0
    want, size = sq.gradients(q, k, v, out[0].transpose(0, 1), g, causal, SCALE)
    for name, a, r, m in zip(("dq", "dk", "dv"), got, want, size):
        # scores of 480 in base 2 instead of 2^6: check_grad's 2^-14 for P becomes 2^-11
        extra = 2.0 ** -11 * m[0] * 1.01
        u = sq.U[dtype]
        tol = 1.01 * (u * r.abs() + u * m[0] + d * 2.0 ** -23 * m[1] + 2.0 ** -25 * m[2] + 2.0 ** -25) + extra
        assert ((a[0].transpose(0, 1).double() - r).abs() <= tol).all(), name


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("order", ["rising", "falling"])
def test_scores_that_move(cq, order, dt, d):
    """Scores that go from -300 to 300 along the keys, or back, a little every key: each tile's weights leave those of the one before far
    behind, or count for nothing beside them."""
    dtype, n, hq, hkv, page = sq.DT[dt], 700, 4, 2, 32
    g = torch.Generator().manual_seed(1)
    q = torch.zeros(n, hq, d)
    q[:, :, :2] = 8.0
    k = torch.zeros(n, hkv, d)
    step = torch.linspace(-300, 300, n) if order == "rising" else torch.linspace(300, -300, n)
    k[:, :, 0] = torch.round(step)[:, None]                                   # whole numbers up to 300: exact in fp16, and in bf16 to 256
    k[:, :, 0] = k[:, :, 0].to(dtype).float()
    k[:, :, 1] = torch.randint(-1, 2, (n, hkv), generator=g).float()
    q, k, v = q.to(dtype).cuda(), k.to(dtype).cuda(), sq.normal((n, hkv, d), dtype, 3)
    cu, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n], [n]))
    pages = -(-n // page)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    kc, vc = (torch.zeros(pages, hkv, page, d, dtype=dtype, device="cuda") for _ in range(2))
    cq.kv_cache_write(k, v, kc, vc, table, cu, lens)
    for causal in (True, False):
        ref, rl, mass = sq.attend(q, k, v, 0, causal, SCALE)
        out, lse = cq.attention_packed(q, k, v, cu, causal=causal, scale=SCALE, return_lse=True)
        _check(out, lse, ref, rl, mass, dtype, what=f"packed causal={causal}")
        for new in (1, 4, n):
            i = slice(n - new, n)
            out, lse = cq.attention_paged(q[i], kc, vc, table, torch.tensor([0, new], dtype=torch.int32, device="cuda"), lens, new, n,
                                          causal=causal, scale=SCALE, return_lse=True)
            _check(out, lse, ref[i], rl[:, i], mass[i], dtype, what=f"{new} tokens causal={causal}")
    torch.cuda.synchronize()
    assert cq.cqsa_device_error()[1] == 0
