"""The library without the extension that checks the arguments of some calls: built all the same, and the calls are checked in
Python."""
import os
import subprocess
import sysconfig

import pytest
import torch

from grok_gqa_attention_gb300 import build


@pytest.fixture
def tree(monkeypatch, tmp_path):
    """A build into an empty folder, with compilers that only leave their output; the commands that were run."""
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        headers = [cmd[i + 1] for i, x in enumerate(cmd) if x == "-I"]
        if "binding.cpp" in " ".join(cmd) and not any(os.path.exists(os.path.join(h, "Python.h")) for h in headers):
            return subprocess.CompletedProcess(cmd, 1, "", "fatal error: Python.h: No such file or directory")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libgrok_attn.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / os.path.basename(build.BINDING)))
    return ran


def _headers(monkeypatch, path):
    found = dict(sysconfig.get_paths(), include=str(path))
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda *a, **k: found)


def test_library_without_pythons_headers(monkeypatch, tmp_path, tree):
    """No Python.h: the library is built and up to date, and no older extension stays beside it."""
    _headers(monkeypatch, tmp_path / "nothing")
    open(build.BINDING, "w").close()
    assert build.build(force=True) == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    assert build.up_to_date()


def test_extension_comes_with_the_headers(monkeypatch, tmp_path, tree):
    """Once there is a Python.h, what was built without the extension is not up to date."""
    _headers(monkeypatch, tmp_path / "nothing")
    build.build(force=True)
    (tmp_path / "include").mkdir()
    (tmp_path / "include" / "Python.h").write_text("")
    _headers(monkeypatch, tmp_path / "include")
    assert not build.up_to_date()
    build.build()
    assert os.path.exists(build.BINDING) and build.up_to_date()


def test_errors_of_the_extensions_source_are_not_hidden(monkeypatch, tmp_path, tree):
    (tmp_path / "include").mkdir()
    (tmp_path / "include" / "Python.h").write_text("")
    _headers(monkeypatch, tmp_path / "include")
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **kw: subprocess.CompletedProcess(
        cmd, int("binding.cpp" in " ".join(cmd)), "", "error: expected ';'"))
    with pytest.raises(RuntimeError, match="binding.cpp"):
        build.build(force=True)


def test_calls_without_the_extension(monkeypatch, tmp_path):
    """Arguments are then checked in Python alone, and refused as with it."""
    import grok_gqa_attention_gb300 as G
    from grok_gqa_attention_gb300 import sparse
    build.build()
    monkeypatch.setattr(sparse, "_checked", None)
    monkeypatch.setattr(sparse.os.path, "exists", lambda p, real=os.path.exists: "_binding" not in p and real(p))
    q, pool = torch.zeros(2, 48, 128, dtype=torch.bfloat16), torch.zeros(4, 128, 8, 128, dtype=torch.bfloat16)
    table, one = torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    codes, scale = G.alloc_kv_bounds(4, "cpu")
    sel, ws = torch.zeros(2, 8, 2, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    for call in (lambda: G.kv_bounds_paged(pool, table, one, None, 1, codes, scale),
                 lambda: G.select_blocks_paged(q, codes, scale, table, one, 0, 0, torch.zeros(2, 8, 4), sel),
                 lambda: G.decode_sparse_paged(q, pool, pool, table, one, sel, ws, q),
                 lambda: G.decode_shared_paged(q, pool, pool, table, one, one, one[:1], ws, q)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_extension_is_of_this_interpreter(monkeypatch, tmp_path, tree):
    """It goes by the name that this Python gives its extensions: one that another Python built is neither loaded nor up to
    date."""
    from grok_gqa_attention_gb300 import sparse
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    assert os.path.basename(build.BINDING) == "_binding" + suffix
    (tmp_path / "include").mkdir()
    (tmp_path / "include" / "Python.h").write_text("")
    _headers(monkeypatch, tmp_path / "include")
    build.build(force=True)
    assert build.up_to_date()
    for other in ("_binding.so", "_binding.cpython-39-x86_64-linux-gnu.so"):
        os.replace(build.BINDING, tmp_path / other)
        assert not build.up_to_date()
        os.replace(tmp_path / other, build.BINDING)
    monkeypatch.undo()
    build.build()
    assert sparse._binding().__file__ == build.BINDING
