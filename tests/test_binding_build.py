"""The compiled way is used only where it was built for the library and the torch
that are loaded, and a build of older sources does not stay behind."""
import os
import subprocess
import sys
import types
import warnings

import pytest
import torch

import sparse_attention_attn_b200 as s2
from sparse_attention_attn_b200 import _lib, api, build
from tests.test_binding import NAMES

TORCH = f"{torch.version.__version__} {torch.version.git_version}"


def _fake(monkeypatch, **attrs):
    """A module in the place of _s2torch; the calls that reached it."""
    seen = []
    m = types.ModuleType("sparse_attention_attn_b200._s2torch")
    m.bind = lambda *a: seen.append(a)
    for n in NAMES:
        setattr(m, n, lambda *a: seen.append(a) or (1,))
    for k, v in attrs.items():
        setattr(m, k, v)
    monkeypatch.setitem(sys.modules, m.__name__, m)
    monkeypatch.setattr(s2, "_s2torch", m, raising=False)
    return seen


@pytest.mark.parametrize("attrs", [dict(), dict(header_hash="h0", torch_version=TORCH), dict(torch_version=TORCH),
                                   dict(header_hash="REAL", torch_version="2.0.0 abc"), dict(header_hash="REAL")])
def test_a_binding_of_another_build_is_not_called(monkeypatch, attrs):
    if attrs.get("header_hash") == "REAL":
        attrs["header_hash"] = _lib.load().s2attn_header_hash().decode()
    seen = _fake(monkeypatch, **attrs)
    b = api._Binding()
    with pytest.warns(RuntimeWarning, match="_s2torch.so was built for"):
        assert b.cache_plan(1, 2, 3) is None
    assert all(getattr(b, n)() is None for n in NAMES) and seen == []


def test_the_warning_as_an_error_comes_once(monkeypatch):
    seen = _fake(monkeypatch)
    b = api._Binding()
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(RuntimeWarning):
            b.cache_plan
        assert b.cache_plan(1) is None and b.qknorm_fwd() is None and seen == []


def test_a_binding_of_this_build_is_bound(monkeypatch):
    seen = _fake(monkeypatch, header_hash=_lib.load().s2attn_header_hash().decode(), torch_version=TORCH)
    assert api._Binding().cache_plan(5) == (1,)
    assert len(seen) == 2 and len(seen[0]) == 7 and all(seen[0]) and seen[1] == (5,)


def test_library_and_binding_name_the_header_they_were_built_with():
    assert _lib.load().s2attn_header_hash().decode() == build.header_hash()
    m = pytest.importorskip("sparse_attention_attn_b200._s2torch")
    assert (m.header_hash, m.torch_version) == (build.header_hash(), TORCH)
    assert build._torch_home()[1] == TORCH


@pytest.mark.parametrize("how", ["compiler fails", "no compiler", "no torch"])
def test_an_old_build_does_not_stay_behind(monkeypatch, tmp_path, capsys, how):
    so = tmp_path / "_s2torch.so"
    so.write_text("old")
    (tmp_path / "_s2torch.so.srchash").write_text("of older sources")
    monkeypatch.setattr(build, "BINDING", str(so))
    if how == "compiler fails":
        def fail(cmd, **kw):
            raise subprocess.CalledProcessError(1, cmd)
        monkeypatch.setattr(build.subprocess, "run", fail)
    elif how == "no compiler":
        monkeypatch.setattr(build.shutil, "which", lambda name: None)
    else:
        monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    build.build()  # (the library itself is up to date)
    assert os.listdir(tmp_path) == [] and "Python path serves alone" in capsys.readouterr().err


def test_an_up_to_date_build_stays(monkeypatch):
    if not os.path.exists(build.BINDING):
        pytest.skip("not built here")
    at = os.path.getmtime(build.BINDING)
    monkeypatch.setattr(build.shutil, "which", lambda name: None)  # no compiler is needed for it
    assert build.build_binding() == build.BINDING and os.path.getmtime(build.BINDING) == at
