"""Shared by the tests of the operators over sequences: ragged problems, and plain forms of them in 64 bits."""
import math

import torch

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
# half a step of a rounding, relative to the value
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def starts(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return out


def normal(shape, dtype, seed, times=1.0, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * times).to(dtype).to(device)


def attend(q, k, v, first, causal, scale=None):
    """softmax(scale q k^T) v in 64 bits: q [n, Hq, d] at positions first.., k and v [m, Hkv, d]. Returns out [n, Hq, d],
    lse [Hq, n] and sum_j p_j |v_j| [n, Hq, d]; a row that sees nothing is 0 / -inf."""
    n, hq, d = q.shape
    m, hkv = k.shape[0], k.shape[1]
    q, k, v = (x.double() for x in (q, k, v))
    k, v = (x.repeat_interleave(hq // hkv, 1) for x in (k, v))
    s = torch.einsum("nhd,mhd->hnm", q, k) * (1.0 / math.sqrt(d) if scale is None else scale)
    if causal:
        hide = torch.arange(m, device=q.device)[None, :] > first + torch.arange(n, device=q.device)[:, None]
        s = s.masked_fill(hide[None], -math.inf)
    if m == 0:
        zero = torch.zeros_like(q)
        return zero, torch.full((hq, n), -math.inf, dtype=torch.float64, device=q.device), zero
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None].masked_fill(lse[..., None] == -math.inf, 0.0))
    # a value that a row does not see does not reach it, whatever it is
    clean = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
    return torch.einsum("hnm,mhd->nhd", p, clean), lse, torch.einsum("hnm,mhd->nhd", p, clean.abs())


def held(x, like):
    return x.to(like.device)


def check_out(got, ref, mass, dtype, p_dtype=None, what="", floor=0.0):
    """|got - ref| element by element. The result is rounded once to dtype (u |ref|), every probability once to
    p_dtype (u p each, so at most u sum p |v|); sums, exponentials and scores in 32 bits add less than 64 * 2^-24 of
    sum p |v| at these sizes (scores under 2^6 in magnitude: 2^-18 relative per probability, the same for numerator and
    denominator), taken as 2^-16. Below fp16's normal numbers the steps are absolute: 2^-25 for the result, and `floor`
    for the probabilities."""
    u, up = U[dtype], U[p_dtype or dtype]
    tol = u * ref.abs() * 1.01 + (up + 2.0 ** -16) * mass * 1.01 + 2.0 ** -24 + floor
    excess = (got.double() - ref).abs() - tol
    assert torch.isfinite(got).all(), what
    assert excess.max().item() <= 0, f"{what}: {excess.max().item():.3e} beyond the tolerance"


def check_lse(got, ref, what=""):
    """fp32 scores and sum: 2^-16 absolute under scores of 2^6, and the fp32 rounding of the result."""
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), fin), f"{what}: empty rows differ"
    assert (got[~fin] == -math.inf).all(), what
    if fin.any():
        err = (got.double() - ref)[fin].abs().max().item()
        assert err <= 2.0 ** -15, f"{what}: lse off by {err:.3e}"


def make_cache(lengths, hkv, d, page, dtype, seed, device="cuda", spare=2, fill=float("nan"), sharp=1.0):
    """Keys and values of each sequence, in pages in a shuffled order whose unused slots hold `fill`. Returns
    (k list, v list, k_cache, v_cache, table)."""
    per = [-(-n // page) for n in lengths]
    total, most = sum(per) + spare, max(max(per), 1) + 1
    order = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).tolist()
    kc = torch.full((total, hkv, page, d), fill, dtype=dtype)
    vc = torch.full((total, hkv, page, d), fill, dtype=dtype)
    table = torch.full((len(lengths), most), -1, dtype=torch.int32)
    ks, vs, at = [], [], 0
    for s, n in enumerate(lengths):
        k = normal((n, hkv, d), dtype, seed * 77 + 2 * s, sharp, "cpu")
        v = normal((n, hkv, d), dtype, seed * 77 + 2 * s + 1, 1.0, "cpu")
        for i in range(per[s]):
            pg = order[at]
            at += 1
            table[s, i] = pg
            rows = min(page, n - i * page)
            kc[pg, :, :rows] = k[i * page:i * page + rows].transpose(0, 1)
            vc[pg, :, :rows] = v[i * page:i * page + rows].transpose(0, 1)
        ks.append(k.to(device))
        vs.append(v.to(device))
    return ks, vs, kc.to(device), vc.to(device), table.to(device)


def quantise(x):
    """e4m3 codes (uint8), exponent bytes and the values they stand for (64 bits), from the definition in 64 bits."""
    x = x.double()
    top = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(-1, keepdim=True)
    e, unit = torch.full_like(top, -126.0), torch.full_like(top, 2.0 ** -126)
    for k in range(-125, 128):  # the smallest power under which the largest value is at most 448
        up = top > 448 * 2.0 ** (k - 1)
        e, unit = torch.where(up, torch.full_like(top, k), e), torch.where(up, torch.full_like(top, 2.0 ** k), unit)
    y = x / unit
    exponent = torch.frexp(torch.nan_to_num(y, 0.0, 0.0, 0.0).abs().clamp(min=2.0 ** -6))[1].long() - 1  # -6 .. 8
    step = torch.tensor([2.0 ** (i - 6 - 3) for i in range(16)], dtype=torch.float64, device=x.device)[exponent + 6]
    val = torch.where(torch.isfinite(x), torch.round(y / step) * step, torch.full_like(x, math.nan))
    code = val.float().to(torch.float8_e4m3fn).view(torch.uint8)
    return code, (e[..., 0] + 127).to(torch.uint8), val * unit


def gradients(q, k, v, out, dout, causal, scale=None):
    """dq, dk, dv of the definition in 64 bits for one sequence ([n, heads, d]), with D from the forward's rounded `out` as the
    kernel takes it, and for each the sums of magnitudes that check_grad's bounds scale with."""
    n, hq, d = q.shape
    hkv = k.shape[1]
    sc = 1.0 / math.sqrt(d) if scale is None else scale
    q, k, v, out, dout = (x.double() for x in (q, k, v, out, dout))
    kk, vv = (x.repeat_interleave(hq // hkv, 1) for x in (k, v))
    s = torch.einsum("nhd,mhd->hnm", q, kk) * sc
    if causal:
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device=q.device).triu(1)[None], -math.inf)
    p = torch.softmax(s, -1)
    dp = torch.einsum("nhd,mhd->hnm", dout, vv)
    ds = p * (dp - (dout * out).sum(-1).T[:, :, None])

    def group(x):
        return x.reshape(n, hkv, hq // hkv, d).sum(2)

    def three(ds, p, q, kk, dout):
        return (torch.einsum("hnm,mhd->nhd", ds, kk) * sc, group(torch.einsum("hnm,nhd->mhd", ds, q)) * sc,
                group(torch.einsum("hnm,nhd->mhd", p, dout)))

    size = torch.einsum("nhd,mhd->hnm", dout.abs(), vv.abs()) + (dout * out).abs().sum(-1).T[:, :, None]
    seen = torch.isfinite(s).double()
    mags = q.abs(), kk.abs(), dout.abs()
    return three(ds, p, q, kk, dout), tuple(zip(three(ds.abs(), p, *mags), three(p * size, 0 * p, *mags), three(seen, seen, *mags)))


def check_grad(got, ref, mass, dtype, what=""):
    """|got - ref| element by element, from the three sums of magnitudes that gradients() gives beside a gradient:
    mass[0], sum |dS| |k| (or |q|; sum P |dout|): P and dS are rounded once to dtype, u each; exp of a score off by 2^-17 and an lse off
      by 2^-16 (scores under 2^6 in fp32) move P, and dS with it, by 2^-14 relative;
    mass[1], sum P (sum_d |dout v| + sum_d |dout out|) |k|: dP and D are sums of d products in fp32, off by at most d * 2^-23 of
      the magnitudes they add (2^-23 a step, as the tensor core truncates), and dS = P (dP - D) may cancel to less than that;
    mass[2], sum |k| over the visible pairs: below fp16's normal numbers P and dS are off by 2^-25 absolutely.
    The result is rounded once: u |ref|, at least fp16's 2^-25."""
    u, tiny = U[dtype], 2.0 ** -25 if dtype == torch.float16 else 0.0
    d = got.shape[-1]
    tol = 1.01 * (u * ref.abs() + (u + 2.0 ** -14) * mass[0] + d * 2.0 ** -23 * mass[1] + tiny * mass[2] + tiny) + 2.0 ** -40
    assert torch.isfinite(got).all(), what
    excess = ((got.double() - ref).abs() - tol).max().item()
    assert excess <= 0, f"{what}: {excess:.3e} beyond the tolerance"
