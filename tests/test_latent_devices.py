"""What the latent-row operators keep for each device and ask of their tensors' devices, without a GPU."""
import os
import subprocess
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

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


class StandIn(torch.Tensor):
    """A CPU tensor that says it is on CUDA device `on` (-1: on the CPU)."""
    __torch_function__ = torch._C._disabled_torch_function_impl
    on = 0
    is_cuda = property(lambda self: self.on >= 0)

    def get_device(self):
        return self.on


def stand_in(*shape, dtype=torch.bfloat16):
    return torch.Tensor._make_subclass(StandIn, torch.zeros(shape, dtype=dtype))


def calls():
    i32, f32 = torch.int32, torch.float32
    absorbed = dict(out=stand_in(2, 1, 512), lse=stand_in(2, 1, dtype=f32), status=stand_in(1, dtype=i32),
                    workspace=stand_in(64, dtype=torch.uint8))
    paged = dict(absorbed, out=stand_in(2, 1, 1, 512), lse=stand_in(2, 1, 1, dtype=f32))
    return {
        "append_rows": (dict(rows=stand_in(2, dtype=i32), latent=stand_in(2, 512), rope=stand_in(2, 64),
                             positions=stand_in(2, dtype=i32), rotation=stand_in(4, 64, dtype=f32), q_rope=stand_in(2, 1, 64),
                             q_out=stand_in(2, 1, 64), status=stand_in(1, dtype=i32)), {}),
        "attend_rows": (dict(rows=stand_in(2, 3, dtype=i32), q_latent=stand_in(2, 1, 512), q_rope=stand_in(2, 1, 64), **absorbed),
                        dict(scale=1.0)),
        "attend_pages": (dict(block_table=stand_in(2, 3, dtype=i32), ctx_len=stand_in(2, dtype=i32),
                              q_latent=stand_in(2, 1, 1, 512), q_rope=stand_in(2, 1, 1, 64), **paged), dict(scale=1.0)),
        "attend_expanded": (dict(q_nope=stand_in(2, 1, 128), q_rope=stand_in(2, 1, 64), k_nope=stand_in(3, 1, 128),
                                 k_rope=stand_in(3, 64), v=stand_in(3, 1, 128), cu_q=stand_in(2, dtype=i32),
                                 cu_k=stand_in(2, dtype=i32), out=stand_in(2, 1, 128), lse=stand_in(2, 1, dtype=f32),
                                 status=stand_in(1, dtype=i32)), dict(scale=1.0)),
    }


@pytest.mark.parametrize("name", ["append_rows", "attend_rows", "attend_pages", "attend_expanded"])
def test_tensors_of_another_device_are_refused_before_a_launch(name, monkeypatch):
    import sparse_mla_kv_gb300 as hs
    from sparse_mla_kv_gb300 import latent

    launched = []
    fake = SimpleNamespace(**{f"hs_{n}": lambda *a, n=n: launched.append(n) or 0 for n in calls()})
    current = [0]
    monkeypatch.setattr(latent, "_lib", lambda: fake)
    monkeypatch.setattr(latent, "_current_device", lambda: current[0])
    tensors, rest = calls()[name]
    rest["stream"] = SimpleNamespace(cuda_stream=0)
    if name != "attend_expanded":
        rest["pool"] = SimpleNamespace(handle=None)
    call = getattr(hs, name)
    call(**tensors, **rest)
    assert launched == [name]                    # all on the current device: it goes through
    for t, x in tensors.items():
        x.on = 1
        with pytest.raises(ValueError, match="device"):
            call(**tensors, **rest)
        x.on = -1
        with pytest.raises(TypeError):
            call(**tensors, **rest)
        x.on = 0
    current[0] = 1
    with pytest.raises(ValueError, match="current"):
        call(**tensors, **rest)
    for x in tensors.values():
        x.on = 1
    call(**tensors, **rest)
    current[0] = 0
    with pytest.raises(ValueError, match="current"):
        call(**tensors, **rest)
    assert launched == [name, name]
