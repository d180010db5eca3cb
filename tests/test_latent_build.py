"""When the library and the binding of the latent calls are built, and what a
latent call says where the binding is missing (no GPU needed)."""
import os

import pytest
import torch

from decode_attention_kv_gb300 import _build, kvd


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The build's files in a folder of their own, with one small kernel as the source."""
    src = tmp_path / "one.cu"
    src.write_text("__global__ void one(int* x) { *x = 1; }\n")
    monkeypatch.setattr(_build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(_build, "sources", lambda: [str(src)])
    monkeypatch.setattr(_build, "BINDING_ERROR", str(tmp_path / "objects" / "error"))
    monkeypatch.setattr(_build, "binding_path", lambda: str(tmp_path / "binding.so"))
    monkeypatch.setattr(_build, "BINDING_SRC", str(tmp_path / "binding.cpp"))
    monkeypatch.setattr(kvd, "_binding", None)
    return tmp_path


def test_the_library_links_without_the_binding(elsewhere, capsys):
    """Where the binding does not compile the build goes on, and a latent call
    raises what stopped it; once it compiles that is forgotten."""
    (elsewhere / "binding.cpp").write_text("#error no such headers\n")
    assert _build.build() == str(elsewhere / "lib.so")
    assert os.path.exists(elsewhere / "lib.so") and not os.path.exists(elsewhere / "binding.so")
    assert "no such headers" in capsys.readouterr().err
    assert _build.up_to_date() and not _build.binding_up_to_date()
    with pytest.raises(RuntimeError, match="no such headers"):
        kvd.verify_drafts(*[None] * 5)
    (elsewhere / "binding.cpp").write_text("int x;\n")
    _build.build()                          # the library is not linked again, the binding is
    assert _build.binding_up_to_date() and not os.path.exists(_build.BINDING_ERROR)


def test_no_binding_at_all(elsewhere):
    with pytest.raises(RuntimeError, match="build it first"):
        kvd.attend_latent(*[None] * 7)


@pytest.mark.parametrize("change", ["version", "abi", "python"])
def test_the_binding_goes_with_its_torch_and_python(monkeypatch, change):
    """Another torch, C++ ABI or Python: the library stays, the binding is built anew."""
    assert _build.up_to_date() and _build.binding_up_to_date()
    here = _build.binding_path()
    if change == "version":
        monkeypatch.setattr(torch, "__version__", "1.0.0")
    elif change == "abi":
        monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
    else:
        monkeypatch.setattr(_build.sysconfig, "get_config_var", lambda name: "cpython-30-none")
    assert _build.binding_path() != here
    assert _build.up_to_date() and not _build.binding_up_to_date()


def test_sources_of_the_library_and_of_the_binding(monkeypatch):
    """A newer kernel does not rebuild the binding, a newer binding source not the library."""
    time = os.path.getmtime
    later = {}
    monkeypatch.setattr(_build.os.path, "getmtime", lambda p: later.get(p, time(p)))
    later[_build.BINDING_SRC] = time(_build.LIB) + 1e6
    assert _build.up_to_date() and not _build.binding_up_to_date()
    later.clear()
    later[_build.sources()[-1]] = time(_build.LIB) + 1e6
    assert not _build.up_to_date() and _build.binding_up_to_date()
