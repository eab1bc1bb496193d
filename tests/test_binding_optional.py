"""The compiled torch functions make calls quicker and are nothing that a call needs: without them, and without torch at the build, everything else is there."""
import os
import sys
import sysconfig
import warnings

import pytest

import exact_long_context_tcgen05_gb300 as cq
from exact_long_context_tcgen05_gb300 import build

torch = pytest.importorskip("torch")


@pytest.fixture
def absent(tmp_path, monkeypatch):
    """No binding for this torch and interpreter."""
    monkeypatch.setattr(cq, "_PKG", str(tmp_path))
    monkeypatch.setattr(cq, "_fast", None)


def test_calls_without_the_binding(absent):
    """Each call looks at its arguments itself (and here refuses tensors that are on no GPU) after one warning."""
    q, cache = torch.zeros(1, 2, 64, dtype=torch.float16), torch.zeros(2, 2, 16, 64, dtype=torch.float16)
    table, cu, lens = torch.zeros(1, 2, dtype=torch.int32), torch.tensor([0, 1], dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    bounds = torch.zeros(2, 2, 2, 64, dtype=torch.int8), torch.zeros(2, 2, dtype=torch.uint8)
    calls = (lambda: cq.kv_cache_write(q, q, cache, cache, table, cu, lens), lambda: cq.kv_cache_read(cache, cache, table, cu, lens, 1, torch.float16),
             lambda: cq.kv_cache_append(q, q, q, torch.zeros(4, 64), cache, cache, table, cu, lens),
             lambda: cq.attention_paged(q, cache, cache, table, cu, lens, 1, 1), lambda: cq.kv_page_bounds(cache, table, cu, lens, *bounds, 1),
             lambda: cq.attention_selected(q, cache, cache, table, cu, lens, *bounds, 1, 1))
    with warnings.catch_warnings(record=True) as seen:
        warnings.simplefilter("always")
        for call in calls:
            with pytest.raises(ValueError, match="CUDA"):
                call()
    assert len(seen) == 1 and "binding" in str(seen[0].message)


def test_a_binding_for_each_torch_and_interpreter():
    name = os.path.basename(build.binding_path())
    assert torch.__version__ in name and name.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert build.binding_path() == cq._binding_path()


def test_library_without_torch(monkeypatch):
    build.build()
    monkeypatch.setitem(sys.modules, "torch", None)  # (an import of it raises ImportError)
    assert build.build() == build.LIB and os.path.exists(build.LIB)


def test_library_without_a_host_compiler(monkeypatch, tmp_path, capfd):
    """A binding that does not compile is said so and leaves the library as it is, and no binding of older sources in its place."""
    build.build()
    (tmp_path / "cqsa_torch.so").write_bytes(b"older")
    os.utime(tmp_path / "cqsa_torch.so", (0, 0))
    monkeypatch.setattr(build, "binding_path", lambda: str(tmp_path / "cqsa_torch.so"))
    monkeypatch.setenv("CXX", "/bin/false")
    assert build.build() == build.LIB and os.path.exists(build.LIB) and not os.listdir(tmp_path)
    assert "binding" in capfd.readouterr().err
