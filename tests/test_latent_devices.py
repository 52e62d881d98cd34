"""What the latent-row operators keep for each device and ask of their tensors' devices, without a GPU."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_mla_kv_gb300", "csrc")

ONCE = r"""
#include <stdio.h>
#include "device_once.cuh"
int main() {
  hs::DeviceOnce once, other;
  int calls = 0;
  cudaError_t next = cudaErrorMemoryAllocation;
  auto prepare = [&] { ++calls; return next; };
  auto say = [&](bool ok) { printf("%d %d\n", ok, calls); };
  say(once.ready(0, prepare) == cudaErrorMemoryAllocation);  // a failure is returned ...
  next = cudaSuccess;
  say(once.ready(0, prepare) == cudaSuccess);                // ... and tried again
  say(once.ready(0, prepare) == cudaSuccess);                // a success is kept,
  say(once.ready(1, prepare) == cudaSuccess);                // for its device only
  say(once.ready(63, prepare) == cudaSuccess);
  say(other.ready(0, prepare) == cudaSuccess);
  say(once.ready(-1, prepare) != cudaSuccess && once.ready(64, prepare) != cudaSuccess);
}
"""


def test_preparation_is_kept_for_each_device_and_only_when_it_succeeded(tmp_path):
    src = tmp_path / "once.cpp"
    src.write_text(ONCE)
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.check_call(["g++", "-std=c++17", "-I", CSRC, "-I", cuda, str(src), "-o", str(tmp_path / "once")])
    said = subprocess.check_output([str(tmp_path / "once")], text=True).split("\n")
    assert said[:7] == ["1 1", "1 2", "1 2", "1 3", "1 4", "1 5", "1 5"]


def test_no_kernel_is_prepared_once_for_a_process():
    """The shared-memory limit of a kernel belongs to a device."""
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        for part in text.split("static const cudaError_t")[1:]:
            assert "cudaFuncSetAttribute" not in part.split("}();")[0], name
