"""What appending with the rotation and the 4-bit cache refuse, before anything is launched (no GPU is touched)."""
import pytest
import torch

from tests.test_seq_refusals import CACHE, CACHE_SIZES, FAKE, PAGES, _refused, cq  # noqa: F401  (cq: the fixture)

APPEND = dict({k: v for k, v in CACHE.items()}, q=FAKE, q_stride=0, q_out=FAKE, cos_sin=FAKE, max_pos=100, rot_dim=64, interleaved=False, Hq=4)


@pytest.mark.parametrize("change,status,word", CACHE_SIZES + PAGES + [
    (dict(k=0), -1, "non-null"), (dict(v=FAKE + 4), -1, "16-byte"), (dict(k_stride=129), -1, "stride"), (dict(v_stride=8), -1, "stride"),
    (dict(q=0), -1, "non-null"), (dict(q_out=0), -1, "non-null"), (dict(q_out=FAKE + 8), -1, "16-byte"), (dict(q_stride=260), -1, "stride"),
    (dict(q_stride=512), -1, "end to end"), (dict(Hq=-1), -1, "heads"), (dict(Hq=2 ** 30), -1, "heads"), (dict(T=2 ** 29), -1, "heads"), (dict(rot_dim=0), -1, "rot_dim"),
    (dict(rot_dim=24), -1, "rot_dim"), (dict(rot_dim=80), -1, "rot_dim"), (dict(rot_dim=-16), -1, "rot_dim"), (dict(max_pos=0), -1, "max_pos"),
    (dict(max_pos=2 ** 31), -1, "max_pos"), (dict(cos_sin=0), -1, "cos_sin"), (dict(cos_sin=FAKE + 4), -1, "cos_sin"),
    (dict(cache_dtype=4), -1, "k_scale"), (dict(cache_dtype=4, k_scale=FAKE, v_scale=FAKE + 8), -1, "16-byte"), (dict(cache_dtype=5), -2, "cache_dtype")])
def test_append(cq, change, status, word):  # noqa: F811
    _refused(cq, lambda: cq.cqsa_kv_cache_append(**(APPEND | change)), status, word)


@pytest.mark.parametrize("change,status,word", [(dict(cache_dtype=4), -1, "k_scale"), (dict(cache_dtype=4, k_scale=FAKE, v_scale=0), -1, "v_scale"),
                                                (dict(cache_dtype=4, k_scale=FAKE + 1, v_scale=FAKE), -1, "16-byte")])
def test_4bit_cache(cq, change, status, word):  # noqa: F811
    _refused(cq, lambda: cq.cqsa_kv_cache_write(**(CACHE | change)), status, word)
    _refused(cq, lambda: cq.cqsa_kv_cache_read(**{k: v for k, v in (CACHE | change).items() if k not in ("k_stride", "v_stride")}), status, word)


def test_kinds_and_scales(cq):  # noqa: F811
    """A byte cache is e4m3 or 4-bit by its scales' shape; scales of another shape, type or place are refused."""
    byte = torch.zeros(3, 2, 16, 64, dtype=torch.uint8)
    three, four = torch.zeros(3, 2, 16, dtype=torch.uint8), torch.zeros(3, 2, 16, 4, dtype=torch.uint8)
    assert cq._kind(byte, three, torch.float16) == (cq.CQSA_E4M3, 64) and cq._kind(byte, four, torch.float16) == (cq.CQSA_INT4, 128)
    assert cq._kind(byte.half(), None, torch.float16) == (cq.CQSA_F16, 64)
    for f in (lambda: cq._kind(byte.half(), None, torch.bfloat16), lambda: cq._scale("k_scale", None, byte.shape, cq.CQSA_INT4, 128, byte.device),
              lambda: cq._scale("k_scale", four[..., :2], byte.shape, cq.CQSA_INT4, 128, byte.device),
              lambda: cq._scale("k_scale", four.int(), byte.shape, cq.CQSA_INT4, 128, byte.device),
              lambda: cq._scale("k_scale", four, byte.shape, cq.CQSA_INT4, 64, byte.device),
              lambda: cq._scale("k_scale", four, byte.shape, cq.CQSA_F16, 64, byte.device)):
        with pytest.raises(ValueError):
            f()


def test_rotary_table(cq):  # noqa: F811
    t = cq.rotary_table(5, 4, base=100.0, device="cpu")
    a = torch.arange(5, dtype=torch.float64)[:, None] * torch.tensor([1.0, 0.1], dtype=torch.float64)
    assert t.dtype == torch.float32 and torch.equal(t, torch.cat([a.cos(), a.sin()], -1).float())
    assert torch.equal(cq.rotary_table(5, 4, inv_freq=[1.0, 0.1], device="cpu"), t)
    far = cq.rotary_table(2 ** 20 + 1, 2, inv_freq=[1.0], device="cpu")[-1].double()
    import math
    assert abs(far[0] - math.cos(2 ** 20)) < 2.0 ** -24 and abs(far[1] - math.sin(2 ** 20)) < 2.0 ** -24
    for f in (lambda: cq.rotary_table(4, 3, device="cpu"), lambda: cq.rotary_table(4, 4, inv_freq=[1.0], device="cpu")):
        with pytest.raises(ValueError):
            f()
