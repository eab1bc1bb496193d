"""What the calls over sequences refuse: every bad argument gives a status and a message before anything is launched
(no GPU is touched)."""
import pytest
import torch

FAKE = 0x1000


@pytest.fixture(scope="module")
def cq():
    import __graft_entry__
    __graft_entry__._builder().build()
    import exact_long_context_tcgen05_gb300 as m
    return m


def _refused(cq, f, status, word):
    with pytest.raises(cq.CqsaError) as e:
        f()
    assert e.value.status == status and word in str(e.value), str(e.value)


PACKED = dict(q=FAKE, k=FAKE, v=FAKE, q_stride=0, k_stride=0, v_stride=0, out=FAKE, lse=FAKE, cu_seqlens=FAKE, n_seqs=2, T=100,
              Hq=8, Hkv=2, d=64, causal=True, scale=0.0, dtype=0, stream=0)
SIZES = [(dict(Hq=7), -1, "multiple"), (dict(Hkv=0), -1, "positive"), (dict(n_seqs=0), -1, "positive"), (dict(T=-1), -1, "positive"),
         (dict(d=96), -2, "head dim"), (dict(dtype=2), -2, "dtype"), (dict(dtype=3), -2, "dtype"), (dict(scale=-1.0), -1, "scale"),
         (dict(scale=float("nan")), -1, "scale"), (dict(scale=float("inf")), -1, "scale"), (dict(Hq=130, Hkv=2), -2, "64 at most"),
         (dict(T=2 ** 30), -2, "too large")]
POINTERS = [(dict(q=0), -1, "non-null"), (dict(q=FAKE + 8), -1, "16-byte"), (dict(out=FAKE + 2), -1, "16-byte"),
            (dict(lse=FAKE + 2), -1, "4-byte"), (dict(cu_seqlens=0), -1, "cu_seqlens"), (dict(cu_seqlens=FAKE + 2), -1, "cu_seqlens"),
            (dict(q_stride=100), -1, "stride"), (dict(q_stride=516), -1, "stride"), (dict(q_stride=-512), -1, "stride"),
            (dict(q_stride=2 ** 40), -1, "stride")]


@pytest.mark.parametrize("change,status,word", SIZES + POINTERS + [(dict(v=0), -1, "non-null"), (dict(k_stride=64), -1, "stride")])
def test_packed_forward(cq, change, status, word):
    _refused(cq, lambda: cq.cqsa_attn_packed_fwd(**(PACKED | change)), status, word)


BACKWARD = dict({k: v for k, v in PACKED.items()}, dout=FAKE, dq=FAKE, dk=FAKE, dv=FAKE, workspace=FAKE, workspace_bytes=2 ** 30)


@pytest.mark.parametrize("change,status,word", SIZES + POINTERS + [
    (dict(dout=0), -1, "non-null"), (dict(dk=FAKE + 4), -1, "16-byte"), (dict(lse=0), -1, "non-null"), (dict(workspace=0), -1, "workspace"),
    (dict(workspace=FAKE + 4), -1, "workspace"), (dict(workspace_bytes=1000), -1, "workspace")])
def test_packed_backward(cq, change, status, word):
    _refused(cq, lambda: cq.cqsa_attn_packed_bwd(**(BACKWARD | change)), status, word)


CACHE = dict(k=FAKE, v=FAKE, k_stride=0, v_stride=0, k_cache=FAKE, v_cache=FAKE, k_scale=0, v_scale=0, block_table=FAKE, max_pages=4,
             cu_seqlens=FAKE, kv_lens=FAKE, n_seqs=2, T=10, Hkv=2, d=64, page_size=16, n_pages=9, dtype=0, cache_dtype=0, stream=0)
PAGES = [(dict(k_cache=0), -1, "non-null"), (dict(v_cache=FAKE + 8), -1, "16-byte"), (dict(block_table=0), -1, "non-null"),
         (dict(block_table=FAKE + 2), -1, "4-byte"), (dict(page_size=8), -2, "page size"), (dict(page_size=48), -2, "page size"),
         (dict(page_size=512), -2, "page size"), (dict(n_pages=0), -1, "positive"), (dict(max_pages=0), -1, "positive"),
         (dict(max_pages=2 ** 27, page_size=16), -2, "too many"), (dict(n_pages=2 ** 30), -2, "too large"), (dict(cache_dtype=1), -2, "cache_dtype"),
         (dict(cache_dtype=2), -2, "cache_dtype"), (dict(cache_dtype=3), -1, "k_scale"),
         (dict(cache_dtype=3, k_scale=FAKE, v_scale=FAKE + 8), -1, "16-byte"), (dict(kv_lens=0), -1, "kv_lens"),
         (dict(cu_seqlens=FAKE + 1), -1, "cu_seqlens")]
CACHE_SIZES = [(dict(Hkv=0), -1, "positive"), (dict(n_seqs=0), -1, "positive"), (dict(T=-1), -1, "positive"), (dict(d=96), -2, "head dim"),
               (dict(dtype=2), -2, "dtype")]


@pytest.mark.parametrize("change,status,word", CACHE_SIZES + PAGES + [(dict(k=0), -1, "non-null"), (dict(v=FAKE + 4), -1, "16-byte"),
                                                                      (dict(k_stride=129), -1, "stride"), (dict(v_stride=8), -1, "stride")])
def test_cache_write(cq, change, status, word):
    _refused(cq, lambda: cq.cqsa_kv_cache_write(**(CACHE | change)), status, word)


@pytest.mark.parametrize("change,status,word", CACHE_SIZES + PAGES + [(dict(k=0), -1, "non-null"), (dict(v=FAKE + 4), -1, "16-byte")])
def test_cache_read(cq, change, status, word):
    a = {k: v for k, v in (CACHE | change).items() if k not in ("k_stride", "v_stride")}
    _refused(cq, lambda: cq.cqsa_kv_cache_read(**a), status, word)


PAGED = dict({k: v for k, v in CACHE.items() if k not in ("k", "v", "k_stride", "v_stride", "stream")}, q=FAKE, q_stride=0, out=FAKE,
             lse=0, max_q_len=1, max_kv_len=100, Hq=8, causal=True, scale=0.0, workspace=FAKE, workspace_bytes=2 ** 30, stream=0)


@pytest.mark.parametrize("change,status,word", SIZES + POINTERS + PAGES + [
    (dict(max_q_len=-1), -1, "max_q_len"), (dict(max_kv_len=-1), -1, "max_kv_len"), (dict(workspace=0), -1, "workspace"),
    (dict(workspace_bytes=16), -1, "workspace"), (dict(workspace=FAKE + 4), -1, "workspace")])
def test_paged(cq, change, status, word):
    _refused(cq, lambda: cq.cqsa_attn_paged_fwd(**(PAGED | change)), status, word)


def test_workspace_sizes(cq):
    assert cq.cqsa_attn_packed_bwd_workspace_size(3, 1000, 8, 2, 64) >= 1000 * 8 * (64 * 4 + 8)
    for bad in ((3, 0, 8, 2, 64), (3, 10, 0, 2, 64), (3, 10, 8, 2, 96), (3, 2 ** 30, 8, 2, 64), (0, 10, 8, 2, 64), (3, 10, 8, 0, 64)):
        assert cq.cqsa_attn_packed_bwd_workspace_size(*bad) == 0
    assert cq.cqsa_attn_paged_workspace_size(4, 4, 8, 2, 128, 16, 1, 1000, 0, 0) > 0
    assert cq.cqsa_attn_paged_workspace_size(4, 0, 8, 2, 128, 16, 1, 1000, 0, 0) == 0
    assert cq.cqsa_attn_paged_workspace_size(4, 4, 7, 2, 128, 16, 1, 1000, 0, 0) == 0


def test_torch_calls_refuse_shapes(cq):
    """The torch conveniences check shapes, types and devices before they take an address."""
    q, k, cu = torch.zeros(10, 4, 64, dtype=torch.float16), torch.zeros(10, 2, 64, dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
    for f in (lambda: cq._packed(q, k, k, cu),  # not on a GPU
              lambda: cq._tokens("q", q, 5, 64, q), lambda: cq._tokens("q", q.float(), 4, 64, q),
              lambda: cq._ints("cu", cu.long(), (2,), q.device), lambda: cq._ints("cu", cu, (3,), q.device),
              lambda: cq._out(torch.zeros(9, 4, 64, dtype=torch.float16), q), lambda: cq._out(q.transpose(0, 1).reshape(10, 4, 64)[:, ::2], q)):
        with pytest.raises(ValueError):
            f()
    t, stride = cq._tokens("q", torch.zeros(10, 8, 64, dtype=torch.float16)[:, 2:6], 4, 64, q)
    assert stride == 512 and t.stride(0) == 512
    t, stride = cq._tokens("q", torch.zeros(4, 10, 64, dtype=torch.float16).transpose(0, 1), 4, 64, q)
    assert stride == 256 and t.is_contiguous()
