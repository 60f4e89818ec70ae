"""What is set up once per device (kernels' shared-memory limits), without a GPU."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_weight_gguf_gb300", "csrc")


def test_set_up_for_each_device_and_failures_are_not_kept(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "once_per_device")
    r = subprocess.run([gxx, "-std=c++17", "-Wall", "-Wextra", "-Werror", "-pthread", "-I", CSRC,
                        os.path.join(ROOT, "tests", "c", "once_per_device.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "all checks passed" in r.stdout, r.stdout


def test_no_launcher_sets_a_shared_memory_limit_for_one_device_only():
    """The limit of each launched kernel is set through allow_smem; the one direct call is the cluster
    count's, which is a query of the device that asks first."""
    direct = []
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            direct += [name] * len(re.findall(r"\bcudaFuncSetAttribute\(", f.read()))
    assert direct == ["qmm_internal.h", "qmm_mma_inst_q4k.cu"]
