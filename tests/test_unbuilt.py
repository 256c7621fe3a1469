"""The package and its build where something they could use is not there (CPU)."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def unbuilt(tmp_path):
    """The package's sources without a built library."""
    to = tmp_path / "bit_quantized_mat_amd"
    to.mkdir()
    for f in os.listdir(os.path.join(ROOT, "bit_quantized_mat_amd")):
        if f.endswith(".py"):
            shutil.copy(os.path.join(ROOT, "bit_quantized_mat_amd", f), to)
    return tmp_path


def _python(code, cwd):
    return subprocess.run([sys.executable, "-c", code], cwd=cwd, capture_output=True, text=True, timeout=300)


def test_star_import_without_a_library(unbuilt):
    r = _python("from bit_quantized_mat_amd import *\n"
                "import bit_quantized_mat_amd as m\n"
                "for n in m.__all__: assert n in globals(), n\n"
                "assert MMVQ_MAX_COLS == 32\n"
                "for f in (paged_attention, kv_fork, KvCache, m.rope, library):\n"
                "    try: f() if f is library else f(None, None)\n"
                "    except RuntimeError as e: assert 'not built' in str(e), e\n"
                "    else: raise AssertionError(f)\n"
                "try: m.no_such_name\n"
                "except AttributeError: print('done')\n", unbuilt)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stderr


def test_names_come_with_the_library():
    import bit_quantized_mat_amd as m
    if not os.path.exists(m.library_path()):
        pytest.skip("not built")
    from bit_quantized_mat_amd import attention
    for n in m._ATTENTION:
        assert getattr(m, n) is getattr(attention, n)


@pytest.fixture
def bare_build(monkeypatch, tmp_path):
    """The build module with its compilations replaced and its own output folder."""
    from bit_quantized_mat_amd import build as b
    made = []
    monkeypatch.setattr(b, "_compile", lambda srcs, out, verbose: made.append(out))
    monkeypatch.setattr(b, "OBJ_DIR", str(tmp_path))
    monkeypatch.setattr(b, "BINDING_LIB", str(tmp_path / "_attention.so"))
    b.made = made
    return b


def test_build_without_a_host_compiler(bare_build, monkeypatch, capfd):
    # the C library needs hipcc alone; its Python binding is left out, loudly, and
    # one of an earlier build does not stay behind
    open(bare_build.BINDING_LIB, "w").close()
    monkeypatch.setattr(bare_build, "CXX", "no-such-compiler")
    assert bare_build.build() == bare_build.LIB
    assert bare_build.LIB in bare_build.made and bare_build.PROBE_LIB in bare_build.made
    assert not os.path.exists(bare_build.BINDING_LIB)
    assert "no-such-compiler" in capfd.readouterr().err


def test_build_without_torch(bare_build, monkeypatch, capfd):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert bare_build.build() == bare_build.LIB
    assert bare_build.LIB in bare_build.made
    assert "torch" in capfd.readouterr().err


def test_build_without_pythons_headers(bare_build, monkeypatch, capfd, tmp_path):
    import sysconfig
    paths = dict(sysconfig.get_paths(), include=str(tmp_path))
    monkeypatch.setattr(sysconfig, "get_paths", lambda: paths)
    assert bare_build.build() == bare_build.LIB
    assert "Python.h" in capfd.readouterr().err


def test_a_binding_that_does_not_compile_is_an_error(bare_build, monkeypatch, tmp_path):
    bad = tmp_path / "bad.cpp"
    bad.write_text("#error no\n")
    monkeypatch.setattr(bare_build, "BINDING_SRC", str(bad))
    if shutil.which(bare_build.CXX) is None:
        pytest.skip("no host compiler")
    with pytest.raises(subprocess.CalledProcessError):
        bare_build.build()
    assert bare_build.LIB in bare_build.made
