"""Packed prompts with grouped heads on the GPU against their definition in 64 bits."""
import math

import pytest
import torch

from tests import _seq as sq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cq():
    import exact_long_context_tcgen05_gb300 as m
    return m


def _ok(cq):
    torch.cuda.synchronize()
    rc, code, _ = cq.cqsa_device_error()
    assert rc == cq.CQSA_OK and code == 0


def _check(out, lse, q, k, v, lens, causal, scale=None, what=""):
    at = 0
    for s, n in enumerate(lens):
        if n:
            ref, rl, mass = sq.attend(q[at:at + n], k[at:at + n], v[at:at + n], 0, causal, scale)
            sq.check_out(out[at:at + n], ref, mass, q.dtype, q.dtype, f"{what} sequence {s}", n * 2.0 ** -34)
            sq.check_lse(lse[:, at:at + n], rl, f"{what} sequence {s}")
        at += n


CASES = [([1], 1, 1), ([128], 2, 2), ([129, 1, 127], 4, 2), ([300, 0, 5, 640], 8, 2), ([17] * 50, 6, 2), ([1000], 5, 1),
         ([64, 65, 63], 64, 1), ([513, 255], 3, 3), ([2] * 130 + [700], 16, 1), ([256, 1300], 12, 4)]


@pytest.mark.parametrize("lens,hq,hkv", CASES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_forward(cq, lens, hq, hkv, d, dt):
    dtype, total = sq.DT[dt], sum(lens) + 3
    q, k, v = sq.normal((total, hq, d), dtype, 1), sq.normal((total, hkv, d), dtype, 2, 1.5), sq.normal((total, hkv, d), dtype, 3)
    # what lies behind the last sequence is nobody's: not even its NaN shows
    k[sum(lens):], v[sum(lens):] = math.nan, math.inf
    cu = torch.tensor(sq.starts(lens), dtype=torch.int32, device="cuda")
    for causal in (True, False):
        out = torch.full_like(q, 7.0)
        out, lse = cq.attention_packed(q, k, v, cu, causal=causal, return_lse=True, out=out)
        _ok(cq)
        _check(out, lse, q, k, v, lens, causal, what=f"causal={causal}")
        assert (out[sum(lens):] == 7.0).all()


@pytest.mark.parametrize("d", [64, 128])
def test_sequences_do_not_meet(cq, d):
    """NaN and infinities in one sequence leave the others bit by bit as they were, and a sequence's result does not depend
    on its place in the batch."""
    dtype, lens = torch.float16, [100, 333, 60]
    q, k, v = (sq.normal((sum(lens), h, d), dtype, i) for i, h in ((1, 4), (2, 2), (3, 2)))
    cu = torch.tensor(sq.starts(lens), dtype=torch.int32, device="cuda")
    out, lse = cq.attention_packed(q, k, v, cu, return_lse=True)
    k2, v2 = k.clone(), v.clone()
    k2[100:433], v2[100:433] = math.nan, math.inf
    out2, lse2 = cq.attention_packed(q, k2, v2, cu, return_lse=True)
    for a, b in ((out, out2), (lse.T, lse2.T)):
        assert torch.equal(a[:100], b[:100]) and torch.equal(a[433:], b[433:])
    alone, lalone = cq.attention_packed(q[100:433], k[100:433], v[100:433], torch.tensor([0, 333], dtype=torch.int32, device="cuda"),
                                        return_lse=True)
    assert torch.equal(alone, out[100:433]) and torch.equal(lalone, lse[:, 100:433])
    _ok(cq)


@pytest.mark.parametrize("d,dt", [(64, "f16"), (128, "bf16"), (128, "f16")])
def test_long_rows(cq, d, dt):
    """Sequences longer than the tensor-core accumulation's segments, peaked rows, on a sample of the queries."""
    dtype, lens = sq.DT[dt], [19000, 777]
    q, k, v = sq.normal((sum(lens), 2, d), dtype, 1), sq.normal((sum(lens), 1, d), dtype, 2, 3.0), sq.normal((sum(lens), 1, d), dtype, 3)
    cu = torch.tensor(sq.starts(lens), dtype=torch.int32, device="cuda")
    out, lse = cq.attention_packed(q, k, v, cu, return_lse=True)
    _ok(cq)
    for first in (0, 4095, 16383, 18900):
        ref, rl, mass = sq.attend(q[first:first + 100], k[:19000], v[:19000], first, True)
        sq.check_out(out[first:first + 100], ref, mass, dtype, dtype, f"from {first}", 19000 * 2.0 ** -34)
        sq.check_lse(lse[:, first:first + 100], rl, f"from {first}")


def test_long_rows_before_short_ones(cq):
    """Units long enough for the running sum in shared memory, followed on the same SMs by units whose second row tile is
    empty: the long sequence's rows are bit by bit what they are alone."""
    lens = [16500] + [100] * 200
    q, k, v = (sq.normal((sum(lens), 8, 64), torch.float16, i) for i in (1, 2, 3))
    cu = torch.tensor(sq.starts(lens), dtype=torch.int32, device="cuda")
    alone, lalone = cq.attention_packed(q[:16500], k[:16500], v[:16500], cu[:2], causal=False, return_lse=True)
    for _ in range(3):
        out, lse = cq.attention_packed(q, k, v, cu, causal=False, return_lse=True)
        assert torch.equal(out[:16500], alone) and torch.equal(lse[:, :16500], lalone)
    _ok(cq)
    for first in (0, 16384, 16400):
        ref, rl, mass = sq.attend(q[first:first + 100], k[:16500], v[:16500], first, False)
        sq.check_out(out[first:first + 100], ref, mass, torch.float16, torch.float16, f"from {first}", 16500 * 2.0 ** -34)
        sq.check_lse(lse[:, first:first + 100], rl, f"from {first}")


RAGGED = [1451, 67, 668, 202, 475, 107, 266, 2568, 403, 176, 0, 209, 1099, 421, 36, 95, 3230, 121, 794, 1170, 778, 1938, 110]


@pytest.mark.parametrize("d,dt", [(128, "bf16"), (128, "f16"), (64, "bf16")])
def test_many_units_repeat(cq, d, dt):
    """Some fourteen units on each SM, sequences that leave a unit's second row tile empty among them: every row against the
    definition, and bit by bit the same again and again, also behind work that has emptied L2."""
    dtype, hq, hkv = sq.DT[dt], 32, 8
    q, k, v = sq.normal((sum(RAGGED), hq, d), dtype, 1), sq.normal((sum(RAGGED), hkv, d), dtype, 2, 1.5), sq.normal((sum(RAGGED), hkv, d), dtype, 3)
    cu = torch.tensor(sq.starts(RAGGED), dtype=torch.int32, device="cuda")
    first = cq.attention_packed(q, k, v, cu, return_lse=True)
    _ok(cq)
    _check(*first, q, k, v, RAGGED, True)
    other = torch.empty(100_000_000, device="cuda")
    for i in range(60):
        if i % 3 == 0:
            other.fill_(i)
        again = cq.attention_packed(q, k, v, cu, return_lse=True)
        assert all(torch.equal(x, y) for x, y in zip(again, first)), f"pass {i}"


def test_strides_scale_streams_and_graph(cq):
    """Slices of a fused projection, another scale and stream, capture and replay with other lengths."""
    d, dtype, lens = 128, torch.bfloat16, [70, 200]
    fused = sq.normal((270, 8, d), dtype, 4)  # 4 query, 2 key, 2 value heads
    q, k, v = fused[:, :4], fused[:, 4:6], fused[:, 6:]
    cu = torch.tensor(sq.starts(lens), dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = cq.attention_packed(q, k, v, cu, scale=0.3, return_lse=True, stream=side)
    side.synchronize()
    _check(out, lse, q, k, v, lens, True, 0.3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = cq.attention_packed(q, k, v, cu, return_lse=True)
    for lens in ([270, 0], [1, 269], [135, 135]):
        cu.copy_(torch.tensor(sq.starts(lens), dtype=torch.int32))
        graph.replay()
        _ok(cq)
        _check(out, lse, q, k, v, lens, True, what=str(lens))


def test_counts_outside_the_tokens(cq):
    """Counts that fall or leave [0, T] are held inside it: nothing outside the buffers is touched."""
    d, dtype = 64, torch.float16
    q, k, v = (sq.normal((100, 2, d), dtype, i) for i in range(3))
    for counts in ([-5, 40, 1000], [90, 20, 60], [0, 100, 50]):
        out = cq.attention_packed(q, k, v, torch.tensor(counts, dtype=torch.int32, device="cuda"), out=torch.zeros_like(q))
        _ok(cq)
        assert torch.isfinite(out).all()


def test_no_tokens(cq):
    z = torch.empty(0, 2, 64, dtype=torch.float16, device="cuda")
    out, lse = cq.attention_packed(z, z, z, torch.zeros(3, dtype=torch.int32, device="cuda"), return_lse=True)
    assert out.shape == z.shape and lse.shape == (2, 0)


def test_a_wait_that_gives_up(cq):
    """The test hook: a key tile that never arrives ends in an error status, and the next call is right again."""
    d, dtype = 64, torch.float16
    q, k, v = (sq.normal((400, 2, d), dtype, i) for i in range(3))
    cu = torch.tensor([0, 400], dtype=torch.int32, device="cuda")
    cq.cqsa_set_timeout_ms(50)
    try:
        cq.cqsa_debug_set_fault(1)
        cq.attention_packed(q, k, v, cu)
        rc, code, _ = cq.cqsa_device_error()
        assert rc == cq.CQSA_ERR_TIMEOUT and code != 0
    finally:
        cq.cqsa_debug_set_fault(0)
        cq.cqsa_set_timeout_ms(0)
    out, lse = cq.attention_packed(q, k, v, cu, return_lse=True)
    _ok(cq)
    _check(out, lse, q, k, v, [400], True)


def _grads(cq, q, k, v, g, cu, causal, scale=None, **kw):
    out, lse = cq.attention_packed(q, k, v, cu, causal=causal, scale=scale, return_lse=True, out=torch.zeros_like(q))
    got = cq.attention_packed_backward(q, k, v, out, g, lse, cu, causal=causal, scale=scale, **kw)
    _ok(cq)
    return out, got


def _check_grads(got, q, k, v, out, g, lens, causal, scale=None, what=""):
    at = 0
    for s, n in enumerate(lens):
        if n:
            i = slice(at, at + n)
            ref, mass = sq.gradients(q[i], k[i], v[i], out[i], g[i], causal, scale)
            for name, x, r, m in zip(("dq", "dk", "dv"), got, ref, mass):
                sq.check_grad(x[i], r, m, q.dtype, f"{what} {name} of sequence {s}")
        at += n


@pytest.mark.parametrize("lens,hq,hkv", CASES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_backward(cq, lens, hq, hkv, d, dt):
    dtype, total = sq.DT[dt], sum(lens) + 3
    q, k, v = sq.normal((total, hq, d), dtype, 1), sq.normal((total, hkv, d), dtype, 2, 1.5), sq.normal((total, hkv, d), dtype, 3)
    g = sq.normal((total, hq, d), dtype, 4)
    for t in (q, k, v, g):
        t[sum(lens):] = math.nan  # nobody's
    cu = torch.tensor(sq.starts(lens), dtype=torch.int32, device="cuda")
    for causal in (True, False):
        into = tuple(torch.full_like(t, 7.0) for t in (q, k, v))
        out, got = _grads(cq, q, k, v, g, cu, causal, grads=into)
        _check_grads(got, q, k, v, out, g, lens, causal, what=f"causal={causal}")
        for t in got:
            assert (t[sum(lens):] == 7.0).all()


def test_backward_against_differences(cq):
    """Central differences of the loss sum(dout * out) in 64 bits, in directions drawn at random."""
    lens, hq, hkv, d, dtype = [37, 90], 4, 2, 64, torch.float16
    q, k, v = (sq.normal((127, h, d), dtype, i) for i, h in ((1, hq), (2, hkv), (3, hkv)))
    g = sq.normal((127, hq, d), dtype, 4)
    cu = torch.tensor(sq.starts(lens), dtype=torch.int32, device="cuda")
    _, got = _grads(cq, q, k, v, g, cu, True)

    def loss(q, k, v):
        total, at = 0.0, 0
        for n in lens:
            i = slice(at, at + n)
            total += (sq.attend(q[i], k[i], v[i], 0, True)[0] * g[i].double()).sum().item()
            at += n
        return total

    x = [t.double() for t in (q, k, v)]
    for which in range(3):
        for seed in range(3):
            w = sq.normal(x[which].shape, torch.float64, 50 + 3 * which + seed)
            h = 1e-4
            up, down = ([t + (h * sign * w if i == which else 0.0) for i, t in enumerate(x)] for sign in (1, -1))
            slope = (loss(*up) - loss(*down)) / (2 * h)
            mine = (got[which].double() * w).sum().item()
            # every element is off by at most about 4 u of the tensor's largest, at random: the sum over N of them by
            # 4 u sqrt(N) times that and the direction's spread of 1, taken four times
            bound = 16 * sq.U[dtype] * got[which].abs().max().item() * math.sqrt(w.numel())
            assert abs(mine - slope) <= bound, (which, mine, slope, bound)


@pytest.mark.parametrize("d", [64, 128])
def test_backward_sequences_do_not_meet(cq, d):
    """NaN and infinities in one sequence do not reach the others' gradients; dk and dv repeat bit by bit."""
    dtype, lens, hq, hkv = torch.bfloat16, [100, 333, 60], 6, 2
    q, k, v, g = (sq.normal((sum(lens), h, d), dtype, i) for i, h in ((1, hq), (2, hkv), (3, hkv), (4, hq)))
    cu = torch.tensor(sq.starts(lens), dtype=torch.int32, device="cuda")
    out, got = _grads(cq, q, k, v, g, cu, True)
    _, again = _grads(cq, q, k, v, g, cu, True)
    assert torch.equal(got[1], again[1]) and torch.equal(got[2], again[2])
    bad = [t.clone() for t in (q, k, v, g)]
    for t in bad:
        t[100:433] = math.nan
    bad[2][100:433] = math.inf
    _, got2 = _grads(cq, *bad, cu, True)
    for a, b in zip(got[1:], got2[1:]):
        assert torch.equal(a[:100], b[:100]) and torch.equal(a[433:], b[433:])
    _check_grads([t[:100] for t in got2], q[:100], k[:100], v[:100], out[:100], g[:100], [100], True)
    _check_grads([t[433:] for t in got2], q[433:], k[433:], v[433:], out[433:], g[433:], [60], True)


def test_backward_strides_scale_stream_and_graph(cq):
    d, dtype, lens = 64, torch.float16, [70, 200]
    fused, g = sq.normal((270, 8, d), dtype, 4), sq.normal((270, 4, d), dtype, 5)
    q, k, v = fused[:, :4], fused[:, 4:6], fused[:, 6:]
    cu = torch.tensor(sq.starts(lens), dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = cq.attention_packed(q, k, v, cu, scale=0.2, return_lse=True, stream=side)
    got = cq.attention_packed_backward(q, k, v, out, g, lse, cu, scale=0.2, stream=side)
    side.synchronize()
    _check_grads(got, q, k, v, out, g, lens, True, 0.2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = cq.attention_packed(q, k, v, cu, return_lse=True)
        got = cq.attention_packed_backward(q, k, v, out, g, lse, cu)
    for lens in ([270, 0], [1, 269], [135, 135]):
        cu.copy_(torch.tensor(sq.starts(lens), dtype=torch.int32))
        graph.replay()
        _ok(cq)
        _check_grads(got, q, k, v, out, g, lens, True, what=str(lens))


def test_backward_many_units_repeat(cq):
    """dk and dv repeat bit by bit over a ragged batch of many key tiles, and every gradient agrees with the formula's."""
    d, dtype, hq, hkv, lens = 128, torch.bfloat16, 8, 2, [n // 2 for n in RAGGED]
    q, g = (sq.normal((sum(lens), hq, d), dtype, i) for i in (1, 4))
    k, v = (sq.normal((sum(lens), hkv, d), dtype, i) for i in (2, 3))
    cu = torch.tensor(sq.starts(lens), dtype=torch.int32, device="cuda")
    out, lse = cq.attention_packed(q, k, v, cu, return_lse=True)
    first = cq.attention_packed_backward(q, k, v, out, g, lse, cu)
    _ok(cq)
    at = sq.starts(lens)
    for s, n in enumerate(lens):
        if n:
            i = slice(at[s], at[s + 1])
            ref, mass = sq.gradients(q[i], k[i], v[i], out[i], g[i], True)
            for x, r, m in zip(first, ref, mass):
                sq.check_grad(x[i], r, m, dtype, f"sequence {s}")
    for _ in range(30):
        again = cq.attention_packed_backward(q, k, v, out, g, lse, cu)
        assert torch.equal(again[1], first[1]) and torch.equal(again[2], first[2])


def test_backward_wait_that_gives_up(cq):
    d, dtype = 64, torch.float16
    q, k, v = (sq.normal((400, 2, d), dtype, i) for i in range(3))
    cu = torch.tensor([0, 400], dtype=torch.int32, device="cuda")
    out, lse = cq.attention_packed(q, k, v, cu, return_lse=True)
    cq.cqsa_set_timeout_ms(50)
    try:
        cq.cqsa_debug_set_fault(2)
        cq.attention_packed_backward(q, k, v, out, q, lse, cu)
        rc, code, _ = cq.cqsa_device_error()
        assert rc == cq.CQSA_ERR_TIMEOUT and code != 0
    finally:
        cq.cqsa_debug_set_fault(0)
        cq.cqsa_set_timeout_ms(0)
    out, got = _grads(cq, q, k, v, q, cu, True)
    _check_grads(got, q, k, v, out, q, [400], True)
