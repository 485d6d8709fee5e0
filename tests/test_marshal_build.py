"""The library builds and its calls work where the C marshaller cannot be built or was built for another Python."""
import os
import sys
import sysconfig

import pytest

import paged_kv_looped_gb300 as rlt
from paged_kv_looped_gb300 import build as B


def hide(monkeypatch):
    """The package as if the module had not been built: nowhere to be found, not imported yet."""
    monkeypatch.setattr(rlt, "__path__", [])
    monkeypatch.delitem(sys.modules, "paged_kv_looped_gb300._marshal", raising=False)
    monkeypatch.setattr(rlt, "_bound", None)


def test_without_python_headers(monkeypatch, tmp_path):
    monkeypatch.setattr(B, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: {"include": str(tmp_path)})
    assert B.build_marshal() is None and not os.listdir(tmp_path)
    B.build()                                                   # (nothing else is out of date, so it only looks)
    assert B.up_to_date()


def test_without_a_c_compiler(monkeypatch, tmp_path):
    monkeypatch.setattr(B, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(B, "_host_cc", lambda: None)
    assert B.build_marshal() is None and not os.listdir(tmp_path)


def test_a_compile_error_is_one(monkeypatch, tmp_path):
    (tmp_path / "Python.h").write_text("#error not a header\n")
    monkeypatch.setattr(B, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: {"include": str(tmp_path)})
    with pytest.raises(RuntimeError, match="marshal.c"):
        B.build_marshal()


def test_the_module_is_this_pythons(monkeypatch, tmp_path):
    B.build()
    assert B.MARSHAL.endswith(sysconfig.get_config_var("EXT_SUFFIX")) and os.path.exists(B.MARSHAL)
    # the binding goes without it: no call is in the plain form
    hide(monkeypatch)
    m = rlt._plain()
    assert m is rlt._plain() and m.append(1, 2) is None and m.decode() is None and m.prefill(*range(14)) is None


@pytest.mark.gpu
def test_calls_without_the_module(cuda_device, monkeypatch):
    import torch
    from test_gpu_kv8_marshal import chain, inputs
    s = inputs(rlt)
    want = chain(rlt, s)
    hide(monkeypatch)
    got = chain(rlt, s)
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    assert rlt.rlt_get_device_error() == 0
