"""What the library sets up once per device (kernel attributes, the workspace
pool, occupancy figures): a first attempt that fails, as for want of memory, must
not refuse the calls after it. The helper that keeps such values is compiled for
the host and run here; the library's sources keep none another way."""
import glob
import os
import shutil
import subprocess

import pytest

import gguf_quant_dequant_q4k_b200 as q4k

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(q4k.__file__), "csrc")
CUDA_INCLUDE = os.environ.get("CUDA_INCLUDE", "/usr/local/cuda/include")


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(CUDA_INCLUDE, "driver_types.h")),
                    reason="no C++ compiler or no CUDA headers")
def test_failed_attempts_are_tried_again(tmp_path):
    exe = os.path.join(tmp_path, "per_device_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread", "-I", CSRC, "-isystem", CUDA_INCLUDE,
                    os.path.join(HERE, "host", "per_device_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "per device ok" in r.stdout, r.stdout


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "q4k_moe_*.cu"))), ids=os.path.basename)
def test_no_first_status_is_kept(path):
    with open(path) as f:
        assert "once_flag" not in f.read()


def test_dense_calls_load_no_expert_kernels():
    """The set-up of every call's device info touches the dense kernels only: a
    program without experts neither waits for the others to load nor fails with them."""
    with open(os.path.join(CSRC, "q4k_api.cu")) as f:
        text = f.read()
    start = text.index("int current_device_info(")
    body = text[start:text.index("}  // namespace q4k", start)]
    assert "set_attributes" in body and "moe" not in body
