"""build() on a machine without Python's headers: everything but the 8-bit expert calls (CPU only)."""
import os
import sys
import sysconfig

import pytest

torch = pytest.importorskip("torch")

from quantized_grouped_gemm_router_gb300 import build as B  # noqa: E402


@pytest.fixture
def no_headers(monkeypatch, tmp_path):
    """Neither the headers nor the module; the library as it is."""
    B.build()
    paths = dict(sysconfig.get_paths(), include=str(tmp_path / "include"))
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **kw: paths)
    monkeypatch.setattr(B, "MODULE_PATH", str(tmp_path / os.path.basename(B.MODULE_PATH)))


def test_the_library_is_built(no_headers):
    import quantized_grouped_gemm_router_gb300 as m
    with pytest.warns(UserWarning, match="Python.h"):
        assert B.build() == B.LIB_PATH
    assert not os.path.exists(B.MODULE_PATH)
    assert m.tile_rows() > 0


def test_no_old_module_stays(no_headers):
    """One that was built beside another library is not left to be loaded with this one."""
    with open(B.MODULE_PATH, "w"):
        pass
    os.utime(B.MODULE_PATH, (0, 0))
    with pytest.warns(UserWarning, match="Python.h"):
        B.build()
    assert not os.path.exists(B.MODULE_PATH)


def test_expert_calls_say_what_is_missing(monkeypatch):
    import quantized_grouped_gemm_router_gb300 as m
    from quantized_grouped_gemm_router_gb300 import experts
    B.build()
    monkeypatch.setattr(experts, "_native", experts._Unloaded())
    monkeypatch.setitem(sys.modules, "quantized_grouped_gemm_router_gb300._experts", None)  # as if it were not there
    for _ in range(2):
        with pytest.raises(ImportError, match="Python's headers"):
            m.expert_workspace(8)
    assert m.tile_rows() > 0
