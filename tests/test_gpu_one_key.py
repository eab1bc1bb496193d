"""Rows that see one key on the GPU: a softmax over one score is 1, so the result is the key's value, to the bit, and the log-sum-exp its score."""
import math

import pytest
import torch

from tests import _seq as sq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cq():
    import exact_long_context_tcgen05_gb300 as m
    return m


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _score(q, k):
    return torch.einsum("nhd,nhd->hn", q.double(), k.double().repeat_interleave(q.shape[1] // k.shape[1], 1)) / math.sqrt(q.shape[2])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,sharp", [(8, 2, 1.0), (5, 1, 6.0), (1, 1, 0.01)])
def test_packed(cq, d, dt, hq, hkv, sharp):
    """Sequences of one token, and the first tokens of longer ones."""
    dtype, lens = sq.DT[dt], [1, 1, 40, 1, 300, 1, 1]
    q, k, v = (sq.normal((sum(lens), h, d), dtype, i, t) for i, h, t in ((1, hq, sharp), (2, hkv, 1.0), (3, hkv, 1.0)))
    out, lse = cq.attention_packed(q, k, v, _ints(sq.starts(lens)), return_lse=True)
    first = torch.tensor(sq.starts(lens)[:-1], device="cuda")
    assert torch.equal(out[first], v[first].repeat_interleave(hq // hkv, 1))
    assert (lse[:, first].double() - _score(q[first], k[first])).abs().max().item() <= 2.0 ** -15
    torch.cuda.synchronize()
    assert cq.cqsa_device_error()[1] == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("cache", ["same", "e4m3"])
def test_paged(cq, cache, d, dt):
    """The first token of a chunk that begins its sequence, and sequences of one position, alone and beside a chunk."""
    dtype, hq, hkv, page = sq.DT[dt], 8, 2, 16
    for lens in ([1, 1, 1], [60, 1, 33]):
        k, v = sq.normal((sum(lens), hkv, d), dtype, 2), sq.normal((sum(lens), hkv, d), dtype, 3)
        q = sq.normal((sum(lens), hq, d), dtype, 1)
        per = [-(-n // page) for n in lens]
        table = torch.zeros(3, max(per), dtype=torch.int32)
        for s, n in enumerate(per):
            table[s, :n] = torch.arange(sum(per[:s]), sum(per[:s + 1]))
        table, cu, kl = table.cuda(), _ints(sq.starts(lens)), _ints(lens)
        kc, vc = (torch.zeros(sum(per), hkv, page, d, dtype=dtype if cache == "same" else torch.uint8, device="cuda") for _ in range(2))
        scales = {} if cache == "same" else {n: torch.zeros(sum(per), hkv, page, dtype=torch.uint8, device="cuda") for n in ("k_scale", "v_scale")}
        cq.kv_cache_write(k, v, kc, vc, table, cu, kl, **scales)
        keys, values = cq.kv_cache_read(kc, vc, table, cu, kl, sum(lens), dtype, **scales)
        out, lse = cq.attention_paged(q, kc, vc, table, cu, kl, max(lens), max(lens), return_lse=True, **scales)
        first = torch.tensor(sq.starts(lens)[:-1], device="cuda")
        assert torch.equal(out[first], values[first].repeat_interleave(hq // hkv, 1)), lens
        assert (lse[:, first].double() - _score(q[first], keys[first])).abs().max().item() <= 2.0 ** -15
    torch.cuda.synchronize()
    assert cq.cqsa_device_error()[1] == 0
