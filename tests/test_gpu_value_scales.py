"""Values whose 4-bit scales lie many powers of two below another's: single tokens keep them to 2^-28 of the largest, whatever that one's probability."""
import pytest
import torch

from tests import _seq as sq
from tests import _seq4 as s4
from tests.test_gpu_paged4 import call, make_cache4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cq():
    import exact_long_context_tcgen05_gb300 as m
    return m


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("new,hq", [(1, 4), (1, 12), (2, 16), (3, 1)])
@pytest.mark.parametrize("n,where", [(7, 0), (7, 3), (300, 0), (300, 40), (300, 296)])
def test_small_scales_beside_a_large_one(cq, d, dt, new, hq, n, where):
    """One value has a scale 2^below times the others' (of 2^-14 to 15 / 8 * 2^-14) and next to no probability; the others carry the result.

    P times a scale is rounded twice, 2^-11 each, where it is a normal fp16 number. One below them is off by 2^-25, that is 2^-39 of the largest scale's power: times a
    code of up to 8, summed over the n keys at most, and divided by the sum of the probabilities relative to the largest, which is 1 or more."""
    ks, vs, kq, vq, kse, vse, table = make_cache4([n], 1, d, 16, 5, sharp=0.3)
    t = torch.arange(n, device="cuda")
    pg, slot = table[0].long()[t // 16], t % 16
    mantissa = torch.randint(0, 8, (n, d // 32), generator=torch.Generator().manual_seed(3)).cuda()
    vse[pg, 0, slot] = (8 + mantissa).to(torch.uint8)
    kq[pg[where], 0, slot[where]] = 0x11  # all codes -7, under a scale of 1
    kse[pg[where], 0, slot[where]] = 120
    k64 = s4.values4(kq[pg, :, slot], kse[pg, :, slot])
    q = (sq.normal((new, hq, d), torch.float32, 3).abs() + 1.0).to(sq.DT[dt])  # (a score of some -7 * 1.8 * sqrt(d): -100 and less)
    for below in (3, 13, 14, 15, 16, 20, 21, 22, 24, 26, 28):
        top = 1 + below
        vse[pg[where], 0, slot[where]] = 8 * top + 7
        v64 = s4.values4(vq[pg, :, slot], vse[pg, :, slot])
        out, lse = call(cq, q, kq, vq, kse, vse, table, [new], [n], causal=False)
        ref, rl, mass = sq.attend(q, k64, v64, 0, False)
        tol = 1.01 * (sq.U[q.dtype] * ref.abs() + (2 * 2.0 ** -11 + 2.0 ** -16) * mass) + n * 8 * 2.0 ** (top - 15 - 39)
        if q.dtype == torch.float16:
            tol += 2.0 ** -25  # half a step below its normal numbers
        excess = ((out.double() - ref).abs() - tol).max().item()
        assert excess <= 0, f"2^{below}: {excess:.3e} beyond the tolerance, of {ref.abs().max().item():.3e}"
        sq.check_lse(lse, rl)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq", [4, 12])
def test_every_power_in_a_vector(cq, d, hq):
    """Groups of one vector, and neighbouring keys, whose scales have every power of two, large and small probabilities mixed; 1,000 keys of a sequence whose
    scales rise and fall. A term of the sum is off by 2^-10 of itself or 2^-39 * 8 of the largest scale's power, whichever is more."""
    n = 1000
    ks, vs, kq, vq, kse, vse, table = make_cache4([n], 1, d, 16, 5)
    t = torch.arange(n, device="cuda")
    pg, slot = table[0].long()[t // 16], t % 16
    for seed, most in ((1, 31), (2, 24), (3, 17)):
        g = torch.Generator().manual_seed(seed)
        power = torch.randint(1, most, (n, d // 32), generator=g)
        vse[pg, 0, slot] = (8 * power + torch.randint(0, 8, (n, d // 32), generator=g)).cuda().to(torch.uint8)
        v64 = s4.values4(vq[pg, :, slot], vse[pg, :, slot])
        for dt in ("f16", "bf16"):
            q = sq.normal((1, hq, d), sq.DT[dt], 3)
            out, lse = call(cq, q, kq, vq, kse, vse, table, [1], [n])
            ref, rl, mass = sq.attend(q, ks[0], v64, n - 1, True)
            tol = 1.01 * (sq.U[q.dtype] * ref.abs() + (2.0 ** -10 + 2.0 ** -16) * mass) + n * 8 * 2.0 ** (most - 1 - 15 - 39) + 2.0 ** -25
            ok = ref.abs() < 60000
            assert ok.any() and ((out.double() - ref).abs() <= tol)[ok].all()
            sq.check_lse(lse, rl)
