"""The index arithmetic of the paged KV cache's kernels (csrc/qmm_kv.h and
csrc/qmm_attend_rows.h) and the rules of attention's launches
(csrc/qmm_attend_shape.h), next to and past the ends of 32 bits, built for the
host with AddressSanitizer and UndefinedBehaviorSanitizer and run by
tests/sanitize/kv_bounds_driver.cpp. CPU only."""

import os
import pathlib
import shutil
import subprocess

import pytest

from test_abi_sanitized import HIPCC, SAN_FLAGS

ROOT = pathlib.Path(__file__).resolve().parent.parent


@pytest.fixture(scope="session")
def driver(tmp_path_factory):
    if not shutil.which(HIPCC) and not os.path.exists(HIPCC):
        pytest.skip("no hipcc")
    exe = tmp_path_factory.mktemp("kv") / "kv_bounds_driver"
    obj = exe.with_suffix(".o")
    src = ROOT / "tests" / "sanitize" / "kv_bounds_driver.cpp"
    for cmd in ([HIPCC, "-std=c++17", "-O1", "-g", *SAN_FLAGS, "-x", "hip", "--cuda-host-only",
                 "-c", str(src), "-o", str(obj)],
                [HIPCC, *SAN_FLAGS, "-o", str(exe), str(obj)]):
        res = subprocess.run(cmd, capture_output=True, text=True)
        assert res.returncode == 0, res.stderr[-3000:]
    return exe


def run(exe, *args):
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    res = subprocess.run([str(exe), *map(str, args)], capture_output=True, text=True, env=env,
                         timeout=120)
    assert res.returncode == 0, f"{res.stdout}\n{res.stderr[-4000:]}"
    return res.stdout


def test_index_arithmetic(driver):
    assert "kv bounds passed" in run(driver)
