"""The extension module of the argument checks is not loaded when it is older than what
it was built from: it reads the plans' structures, whose layout the header states."""
import os
import subprocess

import pytest

from split_kv_mla_gb300 import build as mla_build
from split_kv_mla_gb300 import mla


@pytest.mark.parametrize("newer", ["source", "header", None])
def test_an_old_binding_is_rebuilt(newer, tmp_path, monkeypatch):
    if not os.path.exists(mla_build.LIB):
        pytest.skip("library not built")
    mla.load()
    source = os.path.join(mla_build.CSRC, "mla_binding.cpp")
    deps = [source, *mla_build._headers()]
    monkeypatch.setattr(mla_build, "BUILD", str(tmp_path))
    monkeypatch.setattr(mla, "_binding", None)
    path = mla_build.binding_path()
    os.makedirs(os.path.dirname(path))
    open(path, "wb").close()            # no module, so that loading it fails
    newest = {"source": os.path.getmtime(source), None: max(map(os.path.getmtime, deps)) + 1,
              "header": max(map(os.path.getmtime, deps[1:]))}[newer]
    os.utime(path, (newest - (0 if newer is None else 1),) * 2)
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        return subprocess.CompletedProcess(cmd, 1, "", "not here")
    monkeypatch.setattr(mla_build.subprocess, "run", run)
    with pytest.raises(ImportError if newer is None else RuntimeError):
        mla._native()
    assert len(ran) == (0 if newer is None else 1)
    assert all(source in cmd for cmd in ran)
