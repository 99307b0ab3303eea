"""What is built and loaded where: the C library and the calls through ctypes need
neither torch's headers nor the compiled calls of the rollout step."""
import os
import subprocess
import sys

import pytest

from precision_rl_rollout_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def built():
    try:
        build.build()
    except RuntimeError as e:  # no nvcc on this machine
        pytest.skip(str(e))


def _python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)


def test_other_calls_do_without_the_compiled_ones(built):
    r = _python("from precision_rl_rollout_gb300 import binding as fb, build\n"
                "build.CALLS_STEM = '/nowhere/_calls'\n"
                "fb.load()\n"
                "assert fb.fp8rl_abi_version() > 0 and fb.fp8rl_gemm_workspace_bytes(64, 512, 512) >= 0\n"
                "assert fb.fp8rl_attn_paged_kernel_count(0, 1, 4, 2, 64, 100) == 0\n"
                "try:\n"
                "    fb.fp8rl_rope(None, None, None)\n"
                "except RuntimeError as e:\n"
                "    assert '/nowhere/_calls' in str(e) and 'build' in str(e)\n"
                "else:\n"
                "    raise SystemExit('a rollout call ran without its module')\n")
    assert r.returncode == 0, r.stderr


@pytest.fixture
def small(monkeypatch, tmp_path):
    """The build pointed at a folder of its own and two sources that compile at once."""
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    (csrc / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    (csrc / "calls.cpp").write_text("#error no torch here\n")
    for name, value in (("CSRC", csrc), ("BUILD_DIR", tmp_path / "objects"), ("LIB_PATH", tmp_path / "lib.so"),
                        ("CALLS_STEM", tmp_path / "_calls"), ("CALLS_SOURCE", csrc / "calls.cpp")):
        monkeypatch.setattr(build, name, str(value), raising=False)
    try:
        build._nvcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    return csrc


def test_the_library_is_built_where_the_calls_cannot_be(small):
    import ctypes
    open(build.calls_path(), "w").close()                     # of an earlier library: does not stay
    with pytest.warns(RuntimeWarning, match="no torch here"):
        path = build.build(force=True)
    assert path == build.LIB_PATH and ctypes.CDLL(path).one() == 1
    assert not os.path.exists(build.calls_path())
    # the library stands; only the calls are tried again
    when = os.path.getmtime(path)
    with pytest.warns(RuntimeWarning):
        build.build()
    assert os.path.getmtime(path) == when


def test_a_library_that_does_not_compile_is_an_error(small):
    (small / "one.cu").write_text("#error broken\n")
    with pytest.raises(RuntimeError, match="nvcc failed"):
        build.build(force=True)


def test_calls_built_for_another_torch_or_python_are_not_current(built, monkeypatch):
    import sysconfig
    import torch
    assert build.up_to_date()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "9.9.0")
        assert not build.up_to_date()
    with monkeypatch.context() as m:
        var = sysconfig.get_config_var
        m.setattr(sysconfig, "get_config_var", lambda n: "cpython-399-none" if n == "SOABI" else var(n))
        assert not build.up_to_date()
    assert build.up_to_date()
    # and are not loaded
    r = _python("import torch\n"
                "torch.__version__ = '9.9.0'\n"
                "from precision_rl_rollout_gb300 import binding as fb\n"
                "fb.load()\n"
                "try:\n"
                "    fb.load_calls()\n"
                "except RuntimeError as e:\n"
                "    assert '9.9.0' in str(e)\n"
                "else:\n"
                "    raise SystemExit('loaded')\n")
    assert r.returncode == 0, r.stderr


def test_tensor_memory_is_taken_before_the_next_kernel_is_let_in():
    """A kernel that allocates tensor memory after it has let its dependents in can find
    it taken by one of them, which holds it while it waits for the first to end: neither
    would.  Read from the sources: the allocation comes first in each such kernel."""
    import glob
    import re
    release = re.compile(r"pdl_wait_then_release\(|pdl_release_then_wait\(|grid_launch_dependents\(")
    seen = 0
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for kernel in re.split(r"\n(?:template[^\n]*\n)?__global__", text)[1:]:
            alloc = kernel.find("tmem_alloc(")
            if alloc < 0:
                continue
            seen += 1
            first = release.search(kernel)
            assert first is None or alloc < first.start(), (os.path.basename(path), kernel[:120])
    assert seen >= 7
