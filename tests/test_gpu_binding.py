"""The compiled functions behind the calls over a cache: the same results as the Python functions by themselves, which they leave everything to
that is out of the ordinary."""
import threading

import pytest
import torch

from tests import _seq as sq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cq():
    import exact_long_context_tcgen05_gb300 as m
    return m


class _Nothing:
    """Compiled functions that take nothing: the Python functions work alone."""

    def __getattr__(self, name):
        return lambda *a: None


def _step(cq, kind, dtype, strided=False, stream=None):
    """A prompt appended, read back, attended to whole and over selected pages; everything that comes out, and the caches."""
    d, page, hq, hkv, n = 64, 16, 6, 2, 150
    fused = sq.normal((n, hq + 2 * hkv, d), dtype, 3)
    q, k, v = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    if not strided:
        q, k, v = (x.contiguous() for x in (q, k, v))
    pages = -(-n // page) + 1
    width, more = {"same": (d, None), "e4m3": (d, ()), "4bit": (d // 2, (d // 32,))}[kind]
    caches = [torch.zeros(pages, hkv, page, width, dtype=dtype if kind == "same" else torch.uint8, device="cuda") for _ in range(2)]
    scales = {} if kind == "same" else {x: torch.zeros(pages, hkv, page, *more, dtype=torch.uint8, device="cuda") for x in ("k_scale", "v_scale")}
    table = torch.arange(pages - 1, -1, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    cu, lens = torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.tensor([n], dtype=torch.int32, device="cuda")
    bounds = torch.zeros(pages, hkv, 2, d, dtype=torch.int8, device="cuda"), torch.zeros(pages, hkv, dtype=torch.uint8, device="cuda")
    turn = cq.rotary_table(n, 32)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    on = {"stream": stream}
    cq.kv_cache_write(k, v, *caches, table, cu, lens, **scales, **on)
    written = [c.clone() for c in caches]
    rq = cq.kv_cache_append(q, k, v, turn, *caches, table, cu, lens, **scales, **on)
    got = [*written, rq, *cq.kv_cache_read(*caches, table, cu, lens, n, dtype, **scales, **on)]
    got += cq.attention_paged(rq, *caches, table, cu, lens, n, n, return_lse=True, **scales, **on)
    got.append(cq.attention_paged(rq[-1:], *caches, table, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), lens, 1, n, scale=0.2, causal=False, **scales, **on))
    cq.kv_page_bounds(caches[0], table, cu, lens, *bounds, n, k_scale=scales.get("k_scale"), **on)
    got += cq.attention_selected(rq, *caches, table, cu, lens, *bounds, 4, n, return_lse=True, return_pages=True, **scales, **on)
    got.append(cq.attention_selected(rq, *caches, table, cu, lens, *bounds, 4, n, **scales, **on))
    torch.cuda.synchronize()
    return [*got, *caches, *scales.values(), *bounds]


@pytest.mark.parametrize("kind,dt", [("same", "f16"), ("same", "bf16"), ("e4m3", "f16"), ("4bit", "bf16")])
@pytest.mark.parametrize("strided", [False, True])
def test_same_as_python_alone(cq, kind, dt, strided, monkeypatch):
    fast = _step(cq, kind, sq.DT[dt], strided)
    other = _step(cq, kind, sq.DT[dt], strided, torch.cuda.Stream())
    monkeypatch.setattr(cq, "_fast", _Nothing())
    alone = _step(cq, kind, sq.DT[dt], strided)
    for a, b, c in zip(fast, alone, other):
        assert a.dtype == b.dtype and a.shape == b.shape and torch.equal(a, b) and torch.equal(a, c)


def test_what_it_leaves_to_python(cq):
    """None for what is to be copied, moved or refused, a status for what the library refuses, the caller's own tensors where it gives them."""
    d, page, hkv = 64, 16, 2
    q = sq.normal((1, 4, d), torch.float16, 3)
    k, v, kc, vc, table = sq.make_cache([40], hkv, d, page, torch.float16, 3)
    cu, lens = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([40], dtype=torch.int32, device="cuda")
    f = cq._compiled().attention_paged

    def call(**kw):
        a = dict(q=q, kc=kc, vc=vc, table=table, cu=cu, lens=lens, mq=1, mk=40, causal=True, scale=None, ks=None, vs=None, lse=False, out=None, ws=None) | kw
        return f(*a.values())

    want = cq.attention_paged(q, kc, vc, table, cu, lens, 1, 40)
    assert torch.equal(call(), want) and torch.equal(call(mq=2 ** 40, mk=2 ** 70), want)
    out = torch.empty_like(q)
    assert call(out=out) is out and torch.equal(out, want)
    odd = torch.cat([q.flatten(), q.flatten()[:1]])[1:].reshape(1, 4, d)
    for kw in (dict(q=q.cpu()), dict(q=odd), dict(q=q[..., ::2]), dict(q=q.float()), dict(q=q.bfloat16()), dict(q=q[0]), dict(kc=kc[:, :, ::2]), dict(kc=kc.cpu()),
               dict(vc=vc[:1]), dict(table=table.long()), dict(table=table[0]), dict(cu=cu[:1]), dict(lens=lens.cpu()), dict(mq=-1), dict(mk=1.5), dict(scale=1),
               dict(ks=torch.zeros(3)), dict(vs=torch.zeros(3)), dict(out=out.float()), dict(out=out[:, :2]), dict(ws=torch.zeros(4)), dict(q=None), dict(q=[1])):
        assert call(**kw) is None, kw
    assert f() is None and f(q) is None
    assert call(ws=torch.zeros(4, dtype=torch.uint8, device="cuda")) == cq.CQSA_ERR_INVALID and "workspace" in cq.last_error()
    with pytest.raises(cq.CqsaError):
        cq.attention_paged(q, kc, vc, table, cu, lens, 1, 40, workspace=torch.zeros(4, dtype=torch.uint8, device="cuda"))
    with pytest.raises(cq.CqsaError):
        cq.attention_paged(q, kc, vc, table, cu, lens, 1, 40, scale=float("nan"))


class _Undecided:
    def __bool__(self):
        raise TypeError("neither")


def test_errors_come_back_as_exceptions(cq):
    """A tensor without memory of its own (its address is asked for while the interpreter is free) and an argument that is neither true nor false: exceptions, and the next call
    works."""
    d, page, hkv = 64, 16, 2
    q = sq.normal((1, 4, d), torch.float16, 3)
    k, v, kc, vc, table = sq.make_cache([40], hkv, d, page, torch.float16, 3)
    cu, lens = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([40], dtype=torch.int32, device="cuda")
    want = cq.attention_paged(q, kc, vc, table, cu, lens, 1, 40)
    f = cq._compiled().attention_paged
    for _ in range(3):
        with pytest.raises(RuntimeError, match="storage"):  # (one of a batch that vmap goes over)
            torch.vmap(lambda c: f(q, c, c, table, cu, lens, 1, 40, True, None, None, None, False, None, None))(kc[None])
        with pytest.raises(TypeError, match="neither"):
            f(q, kc, vc, table, cu, lens, 1, 40, True, None, None, None, _Undecided(), None, None)
    done = []
    t = threading.Thread(target=lambda: done.append(1))  # (another thread gets its turn)
    t.start()
    t.join()
    assert done and torch.equal(cq.attention_paged(q, kc, vc, table, cu, lens, 1, 40), want)


def test_threads(cq):
    """Calls from several threads at once, each on its own stream."""
    d, page = 64, 16
    cu, lens = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([400], dtype=torch.int32, device="cuda")
    problems = [(sq.normal((1, 4, d), torch.float16, s), *sq.make_cache([400], 2, d, page, torch.float16, s)[2:]) for s in range(4)]
    want = [cq.attention_paged(q, kc, vc, table, cu, lens, 1, 400) for q, kc, vc, table in problems]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        q, kc, vc, table = problems[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            got = [cq.attention_paged(q, kc, vc, table, cu, lens, 1, 400) for _ in range(200)]
            torch.cuda.current_stream().synchronize()
        if not all(torch.equal(g, want[i]) for g in got):
            bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
