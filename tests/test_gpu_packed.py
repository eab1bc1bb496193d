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
