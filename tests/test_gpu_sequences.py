"""The calls over sequences as they are used together (a prompt, its keys into the cache, steps over it), and at the ends of
their ranges: thousands of sequences, tensors past 2^31 elements, a first call inside a graph capture, copies on another stream."""
import os
import random
import subprocess
import sys

import pytest
import torch

from tests import _seq as sq

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def cq():
    import exact_long_context_tcgen05_gb300 as m
    return m


def _ok(cq):
    torch.cuda.synchronize()
    rc, code, _ = cq.cqsa_device_error()
    assert rc == cq.CQSA_OK and code == 0


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 2), (128, 6, 2)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("cache", ["same", "e4m3"])
def test_prompt_cache_steps(cq, d, hq, hkv, dt, cache):
    """Three prompts, then steps of one token, of a few, and of a chunk; every result against 64 bits over the keys so far."""
    dtype, page, prompts = sq.DT[dt], 16, [50, 1, 200]
    steps = [[1, 1, 1], [4, 0, 2], [1, 90, 1], [1, 1, 1], [33, 1, 0]]
    most = [p + sum(s[i] for s in steps) for i, p in enumerate(prompts)]
    per = [-(-n // page) for n in most]
    order = torch.randperm(sum(per), generator=torch.Generator().manual_seed(1)).tolist()
    table = torch.zeros(3, max(per), dtype=torch.int32)
    for s in range(3):
        table[s, :per[s]] = torch.tensor(order[sum(per[:s]):sum(per[:s + 1])], dtype=torch.int32)
    table = table.cuda()
    shape = (sum(per), hkv, page, d)
    if cache == "e4m3":
        kc, vc = (torch.full(shape, 0x7f, dtype=torch.uint8, device="cuda") for _ in range(2))
        scales = {n: torch.full(shape[:3], 0xff, dtype=torch.uint8, device="cuda") for n in ("k_scale", "v_scale")}
    else:
        kc, vc = (torch.full(shape, float("nan"), dtype=dtype, device="cuda") for _ in range(2))
        scales = {}
    p_dtype = torch.float16 if cache == "e4m3" else dtype
    k_all, v_all = ([torch.empty(0, hkv, d, dtype=torch.float64, device="cuda") for _ in range(3)] for _ in range(2))
    length = [0, 0, 0]
    for i, new in enumerate([prompts] + steps):
        n = sum(new)
        q, k, v = sq.normal((n, hq, d), dtype, 3 * i), sq.normal((n, hkv, d), dtype, 3 * i + 1, 1.5), sq.normal((n, hkv, d), dtype, 3 * i + 2)
        length = [a + b for a, b in zip(length, new)]
        cu, lens = _ints(sq.starts(new)), _ints(length)
        cq.kv_cache_write(k, v, kc, vc, table, cu, lens, **scales)
        held = [sq.quantise(x)[2] if cache == "e4m3" else x.double() for x in (k, v)]
        at = sq.starts(new)
        for s in range(3):
            k_all[s] = torch.cat([k_all[s], held[0][at[s]:at[s + 1]]])
            v_all[s] = torch.cat([v_all[s], held[1][at[s]:at[s + 1]]])
        if i == 0:  # the prompts themselves, over the keys as they were before the cache rounds them
            out, lse = cq.attention_packed(q, k, v, cu, return_lse=True)
            _ok(cq)
            for s in range(3):
                j = slice(at[s], at[s + 1])
                ref, rl, mass = sq.attend(q[j], k[j], v[j], 0, True)
                sq.check_out(out[j], ref, mass, dtype, dtype, f"prompt {s}", 2.0 ** -24)
                sq.check_lse(lse[:, j], rl)
        out, lse = cq.attention_paged(q, kc, vc, table, cu, lens, max(new), max(length), return_lse=True, **scales)
        _ok(cq)
        for s in range(3):
            j = slice(at[s], at[s + 1])
            if new[s]:
                ref, rl, mass = sq.attend(q[j], k_all[s], v_all[s], length[s] - new[s], True)
                sq.check_out(out[j], ref, mass, dtype, p_dtype, f"step {i} sequence {s}", 2.0 ** -20)
                sq.check_lse(lse[:, j], rl)
    got = cq.kv_cache_read(kc, vc, table, _ints(sq.starts(length)), _ints(length), sum(length), dtype, **scales)
    for x, parts in zip(got, (k_all, v_all)):
        assert torch.equal(x, torch.cat(parts).float().to(dtype))


@pytest.mark.parametrize("n_seqs", [257, 3000])
def test_many_sequences(cq, n_seqs):
    """Batches that are walked through in their order instead of ranked: forward, gradients, and chunks over a cache."""
    d, hq, hkv, dtype = 64, 4, 2, torch.float16
    rng = random.Random(n_seqs)
    lens = [0 if rng.random() < 0.1 else rng.randrange(1, 40) if rng.random() < 0.97 else rng.randrange(200, 500) for _ in range(n_seqs)]
    at, total = sq.starts(lens), sum(lens)
    q, k, v, g = (sq.normal((total, h, d), dtype, i) for i, h in enumerate((hq, hkv, hkv, hq)))
    out, lse = cq.attention_packed(q, k, v, _ints(at), return_lse=True)
    grads = cq.attention_packed_backward(q, k, v, out, g, lse, _ints(at))
    _ok(cq)
    assert all(torch.isfinite(t).all() for t in (out, lse, *grads))
    page = 64
    per = [-(-n // page) for n in lens]
    first = sq.starts(per)
    table = torch.zeros(n_seqs, max(per), dtype=torch.int32)
    for s in range(n_seqs):
        table[s, :per[s]] = torch.arange(first[s], first[s + 1])
    table, cu, kl = table.cuda(), _ints(at), _ints(lens)
    kc, vc = (torch.full((sum(per), hkv, page, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    cq.kv_cache_write(k, v, kc, vc, table, cu, kl)
    chunk, clse = cq.attention_paged(q, kc, vc, table, cu, kl, max(lens), max(lens), return_lse=True)
    _ok(cq)
    for s in rng.sample(range(n_seqs), 60) + [0, n_seqs - 1, max(range(n_seqs), key=lambda i: lens[i])]:
        i = slice(at[s], at[s + 1])
        if not lens[s]:
            continue
        ref, rl, mass = sq.attend(q[i], k[i], v[i], 0, True)
        for o, l in ((out, lse), (chunk, clse)):
            sq.check_out(o[i], ref, mass, dtype, dtype, f"sequence {s}", 2.0 ** -24)
            sq.check_lse(l[:, i], rl)
        gref, gmass = sq.gradients(q[i], k[i], v[i], out[i], g[i], True)
        for x, r, m in zip(grads, gref, gmass):
            sq.check_grad(x[i], r, m, dtype, f"sequence {s}")


def test_tokens_past_32_bits(cq):
    """Packed tensors of more than 2^31 elements: the sequences lie at their end."""
    d, h, dtype, lens = 128, 8, torch.bfloat16, [300, 77]
    T = (1 << 21) + 400
    q, k, v, g, out, dq, dk, dv = (torch.empty(T, h, d, dtype=dtype, device="cuda") for _ in range(8))
    base = T - sum(lens)
    for i, t in enumerate((q, k, v, g)):
        t[base:] = sq.normal((sum(lens), h, d), dtype, i)
    cu = _ints([base, base + 300, T])
    out, lse = cq.attention_packed(q, k, v, cu, return_lse=True, out=out)
    cq.attention_packed_backward(q, k, v, out, g, lse, cu, grads=(dq, dk, dv))
    _ok(cq)
    for a, n in ((base, 300), (base + 300, 77)):
        i = slice(a, a + n)
        ref, rl, mass = sq.attend(q[i], k[i], v[i], 0, True)
        sq.check_out(out[i], ref, mass, dtype)
        sq.check_lse(lse[:, i], rl)
        gref, gmass = sq.gradients(q[i], k[i], v[i], out[i], g[i], True)
        for x, r, m in zip((dq, dk, dv), gref, gmass):
            sq.check_grad(x[i], r, m, dtype)


@pytest.mark.parametrize("cache", ["same", "e4m3"])
def test_cache_past_32_bits(cq, cache):
    """A cache of more than 2^31 elements: the sequences' pages are its last ones."""
    d, hq, hkv, page, dtype = 128, 16, 8, 256, torch.bfloat16
    n_pages = (1 << 31) // (hkv * page * d) + 200
    kind = torch.uint8 if cache == "e4m3" else dtype
    kc, vc = (torch.empty(n_pages, hkv, page, d, dtype=kind, device="cuda") for _ in range(2))
    scales = {} if cache == "same" else {n: torch.empty(n_pages, hkv, page, dtype=torch.uint8, device="cuda") for n in ("k_scale", "v_scale")}
    lens = [700, 300]
    table = _ints([[n_pages - 1, n_pages - 3, n_pages - 2], [n_pages - 5, n_pages - 4, 0]])
    k, v = sq.normal((1000, hkv, d), dtype, 1), sq.normal((1000, hkv, d), dtype, 2)
    cu, kl = _ints([0, 700, 1000]), _ints(lens)
    cq.kv_cache_write(k, v, kc, vc, table, cu, kl, **scales)
    got = cq.kv_cache_read(kc, vc, table, cu, kl, 1000, dtype, **scales)
    held = [sq.quantise(x)[2] if cache == "e4m3" else x.double() for x in (k, v)]
    for x, want in zip(got, held):
        assert torch.equal(x, want.float().to(dtype))
    for new in (1, 40):
        q = sq.normal((2 * new, hq, d), dtype, 3)
        out, lse = cq.attention_paged(q, kc, vc, table, _ints([0, new, 2 * new]), kl, new, 700, return_lse=True, **scales)
        _ok(cq)
        for s, (a, n) in enumerate(((0, 700), (700, 300))):
            i = slice(s * new, (s + 1) * new)
            ref, rl, mass = sq.attend(q[i], held[0][a:a + n], held[1][a:a + n], n - new, True)
            sq.check_out(out[i], ref, mass, dtype, torch.float16 if cache == "e4m3" else dtype, f"{new} tokens", 2.0 ** -20)
            sq.check_lse(lse[:, i], rl)


FIRST = """
import sys, torch
sys.path.insert(0, {root!r})
import exact_long_context_tcgen05_gb300 as cq
q, k, v = (torch.randn(70, h, 128, device="cuda", dtype=torch.float16) for h in (4, 2, 2))
kc, vc = (torch.zeros(8, 2, 16, 128, device="cuda", dtype=torch.float16) for _ in range(2))
table = torch.arange(8, device="cuda", dtype=torch.int32)[None]
cu, one, lens = (torch.tensor(x, device="cuda", dtype=torch.int32) for x in ([0, 70], [0, 1], [70]))
def run():
    out, lse = cq.attention_packed(q, k, v, cu, return_lse=True)
    grads = cq.attention_packed_backward(q, k, v, out, q, lse, cu)
    cq.kv_cache_write(k, v, kc, vc, table, cu, lens)
    return out, grads[1], cq.attention_paged(q, kc, vc, table, cu, lens, 70, 70), cq.attention_paged(q[69:], kc, vc, table, one, lens, 1, 70)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
for a, b in zip(got, run()):
    assert torch.equal(a, b)
print("equal")
"""


def test_first_call_in_a_capture():
    """A process whose first calls are captured: the same results as eager ones."""
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("equal"), r.stdout + r.stderr


def test_copies_belong_to_the_stream(cq):
    """Tensors that have to be copied first (heads apart, an odd offset) with another stream: the copies are made there."""
    d, dtype, lens = 64, torch.float16, [300, 200]
    heads_first = sq.normal((4, 500, d), dtype, 1)
    q = heads_first.transpose(0, 1)
    k, v = (sq.normal((500 * 2 * d + 1,), dtype, i)[1:].view(500, 2, d) for i in (2, 3))
    cu = _ints(sq.starts(lens))
    side = torch.cuda.Stream()
    busy = torch.empty(1 << 28, device="cuda")
    torch.cuda.synchronize()
    busy.fill_(1.0)  # work on the current stream that the side stream's calls do not wait for
    out, lse = cq.attention_packed(q, k, v, cu, return_lse=True, stream=side)
    got = cq.attention_packed_backward(q, k, v, out, q, lse, cu, stream=side.cuda_stream)
    _ok(cq)
    at = 0
    for n in lens:
        i = slice(at, at + n)
        ref, rl, mass = sq.attend(q[i], k[i], v[i], 0, True)
        sq.check_out(out[i], ref, mass, dtype, dtype, "", 2.0 ** -24)
        gref, gmass = sq.gradients(q[i], k[i], v[i], out[i], q[i], True)
        for x, r, m in zip(got, gref, gmass):
            sq.check_grad(x[i], r, m, dtype)
        at += n


def test_own_workspace(cq):
    d, dtype = 128, torch.float16
    ks, vs, kc, vc, table = sq.make_cache([3000], 2, d, 16, dtype, 5)
    for new in (1, 20):
        q = sq.normal((new, 8, d), dtype, 6)
        need = cq.cqsa_attn_paged_workspace_size(1, new, 8, 2, d, 16, new, 3000, cq.CQSA_F16, cq.CQSA_F16)
        ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")  # what it holds does not matter
        args = (q, kc, vc, table, _ints([0, new]), _ints([3000]), new, 3000)
        out = cq.attention_paged(*args, workspace=ws)
        assert torch.equal(out, cq.attention_paged(*args))
        with pytest.raises(cq.CqsaError) as e:
            cq.attention_paged(*args, workspace=ws[:need - 256])
        assert e.value.status == cq.CQSA_ERR_INVALID
    _ok(cq)


@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("cache", ["same", "e4m3"])
def test_paged_wait_that_gives_up(cq, new, cache):
    d, dtype = 64, torch.float16
    ks, vs, kc, vc, table = sq.make_cache([3000], 2, d, 16, dtype, 5, fill=0.0)
    scales = {}
    if cache == "e4m3":
        (kc, a, _), (vc, b, _) = sq.quantise(kc), sq.quantise(vc)
        scales = {"k_scale": a, "v_scale": b}
    q = sq.normal((new, 8, d), dtype, 6)
    args = (q, kc, vc, table, _ints([0, new]), _ints([3000]), new, 3000)
    want = cq.attention_paged(*args, **scales)
    cq.cqsa_set_timeout_ms(50)
    try:
        cq.cqsa_debug_set_fault(1)
        cq.attention_paged(*args, **scales)
        rc, code, _ = cq.cqsa_device_error()
        assert rc == cq.CQSA_ERR_TIMEOUT and code != 0
    finally:
        cq.cqsa_debug_set_fault(0)
        cq.cqsa_set_timeout_ms(0)
    assert torch.equal(cq.attention_paged(*args, **scales), want)
    _ok(cq)
