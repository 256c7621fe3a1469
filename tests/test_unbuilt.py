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
