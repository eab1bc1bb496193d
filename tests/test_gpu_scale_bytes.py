"""Every scale byte of a 4-bit cache means the same to every call: (1 + m / 8) 2^(e - 15) for 8 e + m, from 248 on a NaN."""
import pytest
import torch

from tests import _seq as sq
from tests import _seq4 as s4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cq():
    import exact_long_context_tcgen05_gb300 as m
    return m


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cache(d, beside):
    """256 sequences of one position: codes -7 .. 7 in turn, the first 32 features under scale byte s in sequence s, the others under `beside` (None: s too)."""
    page, n = 16, 256
    code = (torch.arange(d, device="cuda") % 15 + 1).to(torch.uint8)
    codes = torch.full((n, 1, page, d // 2), 0x88, dtype=torch.uint8, device="cuda")
    codes[:, 0, 0] = code[0::2] | (code[1::2] << 4)
    scales = torch.full((n, 1, page, d // 32), 255, dtype=torch.uint8, device="cuda")  # (unused slots: NaN)
    scales[:, 0, 0] = torch.arange(n, device="cuda").to(torch.uint8)[:, None]
    if beside is not None:
        scales[:, 0, 0, 1:] = beside
    return codes, scales, torch.arange(n, dtype=torch.int32, device="cuda")[:, None].contiguous(), s4.values4(codes[:, 0, 0], scales[:, 0, 0])


def _same(got, want, what):
    """Equal, a NaN where a NaN is wanted."""
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    assert torch.equal(got[~torch.isnan(got)], want[~torch.isnan(want)]), what


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("beside", [None, 8, 119, 120, 130])
def test_values(cq, d, dt, beside):
    """A row that sees one position gives its value: single tokens, a few and a chunk, and what is read back. Chunks hold a number as fp16 relative to the largest
    scale's power of two: (8 + m) 2^(-3 - r) for a scale r powers below it, a multiple of fp16's least number 2^-24 as long as r is at most 21."""
    dtype = sq.DT[dt]
    codes, scales, table, val = _cache(d, beside)
    ok = torch.full_like(scales, 255)
    ok[:, :, 0] = 120
    lens = _ints([1] * 256)
    want = val.to(dtype)
    k, v = cq.kv_cache_read(codes, codes, table, _ints(list(range(257))), lens, 256, dtype, k_scale=ok, v_scale=scales)
    most = torch.finfo(dtype).max
    _same(v[:, 0], val.clamp(-most, most).to(dtype), "read back")
    for new, hq in ((1, 1), (1, 12), (3, 8), (40, 1)):
        q = sq.normal((256 * new, hq, d), dtype, 3)
        out = cq.attention_paged(q, codes, codes, table, _ints([new * i for i in range(257)]), lens, new, 1, causal=False, k_scale=ok, v_scale=scales)
        torch.cuda.synchronize()
        assert cq.cqsa_device_error()[1] == 0
        e = torch.arange(256, device="cuda") // 8
        near = (e - (e if beside is None else beside // 8)).abs() <= 21 if new == 40 else e >= 0
        near = (near | (e == 31)).repeat_interleave(new)
        _same(out[near], want.repeat_interleave(new, 0)[:, None].expand_as(out)[near], (new, hq))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("beside", [None, 8, 120])
def test_keys(cq, d, dt, beside):
    """A row that sees one key: its lse is the score, a sum of up to 128 exact products in 32 bits (2^-18 of their magnitudes) times a factor rounded twice;
    a NaN where a group's scale is one. A query of one feature leaves no sum: the score of every byte to 2^-20 of itself. Sums of exponentials are kept as up to 2^14
    of them, whose logarithm is taken off a score in 32 bits: 2^-18 absolute."""
    dtype = sq.DT[dt]
    codes, scales, table, val = _cache(d, beside)
    ok = torch.full_like(scales, 255)
    ok[:, :, 0] = 120
    lens = _ints([1] * 256)
    for new, hq in ((1, 1), (1, 12), (3, 8), (40, 1)):
        for only in (None, 2):
            q = sq.normal((1, hq, d), dtype, 3)
            if only is not None:
                q = torch.zeros_like(q)
                q[..., only] = 1.0
            out, lse = cq.attention_paged(q.repeat(256 * new, 1, 1), codes, codes, table, _ints([new * i for i in range(257)]), lens, new, 1, causal=False,
                                          scale=1.0, k_scale=scales, v_scale=ok, return_lse=True)
            torch.cuda.synchronize()
            assert cq.cqsa_device_error()[1] == 0
            lse = lse.view(hq, 256, new).double()
            want = torch.einsum("hd,sd->hs", q[0].double(), val)[..., None].expand_as(lse)
            size = torch.einsum("hd,sd->hs", q[0].double().abs(), val.abs())[..., None].expand_as(lse)
            nan = (torch.isnan(val).any(-1) & (torch.arange(256, device="cuda") >= 248))[None, :, None].expand_as(lse)
            assert torch.equal(torch.isnan(lse), nan), (new, hq, only)
            off = (lse - want).abs() - size * (2.0 ** -18 if only is None else 2.0 ** -20) - 2.0 ** -18
            assert off[~nan].max().item() <= 0, (new, hq, only)


def test_slots_of_zeros(cq):
    """Slots that nothing was written to, of zeros as they were allocated, counted as positions: every form reads them alike (-8 times 2^-15)."""
    d, page, hkv, n = 128, 16, 2, 40
    kq, vq = (torch.zeros(3, hkv, page, d // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
    kse, vse = (torch.zeros(3, hkv, page, d // 32, dtype=torch.uint8, device="cuda") for _ in range(2))
    table, lens = _ints([[2, 0, 1]]), _ints([n])
    q = sq.normal((40, 8, d), torch.bfloat16, 3)
    want = -8 * 2.0 ** -15
    k, v = cq.kv_cache_read(kq, vq, table, _ints([0, n]), lens, n, torch.bfloat16, k_scale=kse, v_scale=vse)
    assert (k == want).all() and (v == want).all()
    for new in (1, 3, 40):
        out, lse = cq.attention_paged(q[:new], kq, vq, table, _ints([0, new]), lens, new, n, k_scale=kse, v_scale=vse, return_lse=True)
        assert (out == want).all(), new
        score = q[:new].double().sum(-1) * want / d ** 0.5
        seen = torch.arange(n - new + 1, n + 1, device="cuda").double().log()
        assert ((lse.double() - (score.T + seen)).abs() <= 2.0 ** -15).all(), new
