"""Chunks over a cache on the GPU whose units are long enough for running sums of O, in ranges that begin in the middle of a unit and in whole
units, with keys and values whose sizes rise and fall from one segment to the next."""
import pytest
import torch

from tests import _seq as sq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cq():
    import exact_long_context_tcgen05_gb300 as m
    return m


def _sizes(n, segment, powers):
    """A factor for each of n positions, 2^powers[i] in the i-th segment."""
    at = (torch.arange(n, device="cuda") // segment).clamp(max=len(powers) - 1)
    return torch.exp2(torch.tensor(powers, dtype=torch.float64, device="cuda"))[at][:, None, None]


@pytest.mark.parametrize("powers", [[0, 3, 6], [5, -3, 1], [-2, -2, 7]])
@pytest.mark.parametrize("d,dt", [(128, "f16"), (128, "bf16"), (64, "f16"), (64, "bf16")])
@pytest.mark.parametrize("cache", ["same", "e4m3"])
def test_chunks_with_running_sums(cq, cache, d, dt, powers):
    dtype, hq, hkv, page, new = sq.DT[dt], 8, 2, 64, [300, 130]
    # O is folded every 4,096 keys at d = 128, every 16,384 at d = 64
    segment = 4096 if d == 128 else 16384
    lengths = [2 * segment + 900, segment + 1100]
    per = [-(-n // page) for n in lengths]
    kc, vc = (torch.zeros(sum(per), hkv, page, d, dtype=dtype if cache == "same" else torch.uint8, device="cuda") for _ in range(2))
    scales = {} if cache == "same" else {n: torch.zeros(sum(per), hkv, page, dtype=torch.uint8, device="cuda") for n in ("k_scale", "v_scale")}
    table = torch.zeros(2, max(per), dtype=torch.int32, device="cuda")
    order = torch.randperm(sum(per), generator=torch.Generator().manual_seed(3)).to(torch.int32).cuda()
    table[0, :per[0]], table[1, :per[1]] = order[:per[0]], order[per[0]:]
    ks, vs = [], []
    for s, n in enumerate(lengths):
        k = (sq.normal((n, hkv, d), torch.float64, 10 + s) * _sizes(n, segment, [p / 4 for p in powers])).to(dtype)
        v = (sq.normal((n, hkv, d), torch.float64, 20 + s) * _sizes(n, segment, powers)).to(dtype)
        cq.kv_cache_write(k, v, kc, vc, table[s:s + 1].contiguous(), torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                          torch.tensor([n], dtype=torch.int32, device="cuda"), **scales)
        ks.append(sq.quantise(k)[2] if cache == "e4m3" else k)
        vs.append(sq.quantise(v)[2] if cache == "e4m3" else v)
    q = sq.normal((sum(new), hq, d), dtype, 5)
    cu, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (sq.starts(new), lengths))
    # the caller's longest length sets the CTAs: 8 (ranges of about two units, cut anywhere), one per SM, and one for the last 40 tokens
    # of the second sequence alone (whole units)
    for most, part in ((1, False), (max(lengths), False), (1, True)):
        if part:
            args = (q[390:], kc, vc, table[1:].contiguous(), torch.tensor([0, 40], dtype=torch.int32, device="cuda"), lens[1:], 40, most)
            which = [(1, 0, 390, 40)]
        else:
            args = (q, kc, vc, table, cu, lens, max(new), most)
            which = [(0, 0, 0, 300), (1, 300, 300, 130)]
        for causal in (True, False):
            out, lse = cq.attention_paged(*args, causal=causal, return_lse=True, **scales)
            again = cq.attention_paged(*args, causal=causal, **scales)
            torch.cuda.synchronize()
            assert cq.cqsa_device_error()[1] == 0
            assert torch.equal(out, again)
            for s, at, first, n in which:
                i = slice(at, at + n)
                ref, rl, mass = sq.attend(q[first:first + n], ks[s], vs[s], lengths[s] - n, causal)
                # a row's largest probability is held as more than 2^5 in fp16, whose steps below its normal numbers are 2^-24: a smaller one
                # is off by up to 2^-30 of it, times the largest value
                floor = 0.0 if dtype == torch.bfloat16 and cache == "same" else lengths[s] * 2.0 ** -30 * vs[s].abs().max().item()
                what = f"most={most} causal={causal} {n} tokens of sequence {s}"
                sq.check_out(out[i], ref, mass, dtype, torch.float16 if cache == "e4m3" else dtype, what, floor)
                sq.check_lse(lse[:, i], rl, what)
