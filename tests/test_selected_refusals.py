"""What the bounds of pages and the attention over selected pages refuse, before anything is launched (no GPU is touched)."""
import pytest

from tests.test_seq_refusals import CACHE, CACHE_SIZES, FAKE, PAGED, PAGES, POINTERS, SIZES, _refused, cq  # noqa: F401  (cq: the fixture)

BOUNDS = dict({k: v for k, v in CACHE.items() if k not in ("k", "v", "k_stride", "v_stride", "v_cache", "v_scale")}, bounds=FAKE, bounds_exp=FAKE, max_q_len=1)
KEYS = [(c, s, w) for c, s, w in PAGES if not {"v_cache", "v_scale"} & set(c)]


@pytest.mark.parametrize("change,status,word", CACHE_SIZES + KEYS + [
    (dict(bounds=0), -1, "bounds"), (dict(bounds=FAKE + 8), -1, "bounds"), (dict(bounds_exp=0), -1, "bounds"), (dict(max_q_len=-1), -1, "max_q_len"),
    (dict(cache_dtype=4), -1, "k_scale"), (dict(cache_dtype=4, k_scale=FAKE + 8), -1, "16-byte"), (dict(n_seqs=2 ** 30), -2, "too large")])
def test_bounds(cq, change, status, word):  # noqa: F811
    _refused(cq, lambda: cq.cqsa_kv_page_bounds(**(BOUNDS | change)), status, word)


SELECTED = dict({k: v for k, v in PAGED.items() if k not in ("max_q_len", "causal")}, pages=FAKE, bounds=FAKE, bounds_exp=FAKE, n_select=4)


@pytest.mark.parametrize("change,status,word", SIZES + POINTERS + PAGES + [
    (dict(bounds=0), -1, "bounds"), (dict(bounds=FAKE + 8), -1, "bounds"), (dict(bounds_exp=0), -1, "bounds"), (dict(pages=FAKE + 2), -1, "4-byte"),
    (dict(n_select=0), -1, "n_select"), (dict(n_select=-3), -1, "n_select"), (dict(n_select=2 ** 20 + 1), -1, "n_select"), (dict(max_kv_len=-1), -1, "max_kv_len"),
    (dict(Hq=66), -2, "32 at most"), (dict(T=2 ** 20, n_select=2 ** 14), -2, "too large"), (dict(workspace=0), -1, "workspace"),
    (dict(workspace_bytes=16), -1, "workspace"), (dict(workspace=FAKE + 4), -1, "workspace")])
def test_selected(cq, change, status, word):  # noqa: F811
    _refused(cq, lambda: cq.cqsa_attn_selected_fwd(**(SELECTED | change)), status, word)


def test_workspace_sizes(cq):  # noqa: F811
    size = cq.cqsa_attn_selected_workspace_size
    assert size(4, 8, 2, 128, 16, 8, 1000, 0, 0) > 4 * 2 * (63 + 8) * 4
    assert size(0, 8, 2, 128, 16, 8, 1000, 0, 0) == 0
    for bad in ((4, 7, 2, 128, 16, 8, 1000, 0, 0), (4, 8, 2, 96, 16, 8, 1000, 0, 0), (4, 8, 2, 128, 24, 8, 1000, 0, 0), (4, 8, 2, 128, 16, 0, 1000, 0, 0),
                (4, 8, 2, 128, 16, 8, -1, 0, 0), (4, 99, 1, 128, 16, 8, 1000, 0, 0)):
        assert size(*bad) == 0
    # scores of many tokens are held 64 MiB at a time
    assert size(2048, 32, 8, 128, 16, 8, 1 << 20, 0, 0) < (64 << 20) + 2 * 2048 * 8 * 8 * 4 + (64 << 20)
