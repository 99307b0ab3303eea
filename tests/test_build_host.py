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
                "build.CALLS_PATH = '/nowhere/_calls.so'\n"
                "fb.load()\n"
                "assert fb.fp8rl_abi_version() > 0 and fb.fp8rl_gemm_workspace_bytes(64, 512, 512) >= 0\n"
                "assert fb.fp8rl_attn_paged_kernel_count(0, 1, 4, 2, 64, 100) == 0\n"
                "try:\n"
                "    fb.fp8rl_rope(None, None, None)\n"
                "except RuntimeError as e:\n"
                "    assert '_calls.so' in str(e) and 'build' in str(e)\n"
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
                        ("CALLS_PATH", tmp_path / "_calls.so"), ("CALLS_SOURCE", csrc / "calls.cpp")):
        monkeypatch.setattr(build, name, str(value), raising=False)
    try:
        build._nvcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    return csrc


def test_the_library_is_built_where_the_calls_cannot_be(small):
    import ctypes
    open(build.CALLS_PATH, "w").close()                     # of an earlier library: does not stay
    with pytest.warns(RuntimeWarning, match="no torch here"):
        path = build.build(force=True)
    assert path == build.LIB_PATH and ctypes.CDLL(path).one() == 1
    assert not os.path.exists(build.CALLS_PATH)
    # the library stands; only the calls are tried again
    when = os.path.getmtime(path)
    with pytest.warns(RuntimeWarning):
        build.build()
    assert os.path.getmtime(path) == when


def test_a_library_that_does_not_compile_is_an_error(small):
    (small / "one.cu").write_text("#error broken\n")
    with pytest.raises(RuntimeError, match="nvcc failed"):
        build.build(force=True)
