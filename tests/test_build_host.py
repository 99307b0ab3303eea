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
