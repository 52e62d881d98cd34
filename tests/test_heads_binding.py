"""The C boundary and the binding of the operators on pages of grouped heads and of read_rows, without a GPU: what is refused before a
device is touched, structures as the header has them, tensors of other devices."""
import ctypes
import os
import subprocess
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def hs():
    from sparse_mla_kv_gb300 import _build

    _build.build()
    import sparse_mla_kv_gb300

    return sparse_mla_kv_gb300


def test_structures_match_the_headers(hs, tmp_path):
    from sparse_mla_kv_gb300 import heads, latent

    pairs = (("hs_heads_append", heads.HeadsAppendC), ("hs_heads_read", heads.HeadsReadC), ("hs_heads_attend", heads.HeadsAttendC),
             ("hs_read_latent", latent.ReadLatentC))
    lines = []
    for c, py in pairs:
        lines.append(f'printf("{c} %zu\\n", sizeof({c}));')
        lines += [f'printf("{c}.{f} %zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "hs_heads.h"\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0; }\n")
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "layout")])
    said = dict(line.split() for line in subprocess.check_output([str(tmp_path / "layout")], text=True).splitlines())
    for c, py in pairs:
        assert int(said[c]) == ctypes.sizeof(py)
        for f, _ in py._fields_:
            assert int(said[f"{c}.{f}"]) == getattr(py, f).offset, (c, f)


def test_row_bytes(hs):
    assert hs.heads_row_bytes(1, 64) == 144 and hs.heads_row_bytes(8, 128) == 2064 and hs.heads_row_bytes(128, 128) == 32784
    for kv, dim in ((0, 64), (129, 64), (-1, 128), (4, 32), (4, 96), (4, 256), (4, 0)):
        with pytest.raises(ValueError):
            hs.heads_row_bytes(kv, dim)


def test_null_and_empty_arguments_are_refused_before_a_device_is_touched(hs):
    from sparse_mla_kv_gb300 import heads, latent

    L, M = heads._lib(), latent._lib()
    assert L.hs_append_heads(None, 0, None, None) == 1
    assert L.hs_append_heads(None, 0, ctypes.byref(heads.HeadsAppendC(kv_heads=1, head_dim=64)), None) == 1
    assert L.hs_read_heads(None, 0, None, None) == 1
    assert L.hs_read_heads(None, 0, ctypes.byref(heads.HeadsReadC(kv_heads=1, head_dim=64)), None) == 1
    assert L.hs_attend_heads(None, 0, None, None, 0, None) == 1
    assert L.hs_attend_heads(None, 0, ctypes.byref(heads.HeadsAttendC(kv_heads=1, head_dim=64, q_heads=1, scale=1.0)), None, 0, None) == 1
    assert M.hs_read_rows(None, 0, None, None) == 1
    assert M.hs_read_rows(None, 0, ctypes.byref(latent.ReadLatentC()), None) == 1


def test_cpu_tensors_and_wrong_shapes_raise(hs):
    pool = SimpleNamespace(handle=None, row_bytes=hs.heads_row_bytes(2, 64))
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    i = torch.zeros(2, dtype=torch.int32)
    table = torch.zeros((2, 3), dtype=torch.int32)
    for call in (lambda: hs.append_heads(pool, table, i, z(2, 2, 64), z(2, 2, 64)),
                 lambda: hs.read_heads(pool, table, None, None, 2, 64),
                 lambda: hs.attend_heads(pool, table, i, z(2, 2, 64), 1.0),
                 lambda: hs.read_rows(pool, i)):
        with pytest.raises(TypeError, match="CUDA"):
            call()
    with pytest.raises(ValueError):
        hs.append_heads(pool, table, i, z(2, 128), z(2, 2, 64))
    with pytest.raises(ValueError):
        hs.attend_heads(pool, table, i, z(2, 128), 1.0)


class StandIn(torch.Tensor):
    """A CPU tensor that says it is on CUDA device `on` (-1: on the CPU)."""
    __torch_function__ = torch._C._disabled_torch_function_impl
    on = 0
    is_cuda = property(lambda self: self.on >= 0)

    def get_device(self):
        return self.on


def stand_in(*shape, dtype=torch.bfloat16):
    return torch.Tensor._make_subclass(StandIn, torch.zeros(shape, dtype=dtype))


I32, F32 = torch.int32, torch.float32


def calls():
    tables = dict(block_table=stand_in(2, 3, dtype=I32))
    return {
        "append_heads": (dict(tables, ctx_len=stand_in(2, dtype=I32), k=stand_in(4, 2, 64), v=stand_in(4, 2, 64), cu=stand_in(3, dtype=I32),
                              status=stand_in(1, dtype=I32)), {}),
        "read_heads": (dict(tables, start=stand_in(2, dtype=I32), cu=stand_in(3, dtype=I32), k=stand_in(4, 2, 64), v=stand_in(4, 2, 64),
                            status=stand_in(1, dtype=I32)), dict(tokens=4, head_dim=64)),
        "attend_heads": (dict(tables, ctx_len=stand_in(2, dtype=I32), q=stand_in(4, 6, 64), cu_q=stand_in(3, dtype=I32),
                              out=stand_in(4, 6, 64), lse=stand_in(4, 6, dtype=F32), status=stand_in(1, dtype=I32),
                              workspace=stand_in(64, dtype=torch.uint8)), dict(scale=1.0)),
        "read_rows": (dict(rows=stand_in(4, dtype=I32), latent=stand_in(4, 512), rope=stand_in(4, 64), status=stand_in(1, dtype=I32)), {}),
    }


@pytest.fixture
def faked(hs, monkeypatch):
    """The library replaced by one that notes its calls, and a current device."""
    from sparse_mla_kv_gb300 import heads, latent

    launched, current = [], [0]
    fake = SimpleNamespace(**{f"hs_{n}": lambda *a, n=n: launched.append(n) or 0 for n in calls()})
    for module in (heads, latent):
        monkeypatch.setattr(module, "_lib", lambda: fake)
    monkeypatch.setattr(latent, "_current_device", lambda: current[0])
    return SimpleNamespace(launched=launched, current=current)


def arguments(hs, name):
    tensors, rest = calls()[name]
    return tensors, dict(rest, stream=SimpleNamespace(cuda_stream=0), pool=SimpleNamespace(handle=None, row_bytes=2 * 2 * 64 + 16))


@pytest.mark.parametrize("name", sorted(calls()))
def test_tensors_of_another_device_are_refused_before_a_launch(hs, faked, name):
    tensors, rest = arguments(hs, name)
    call = getattr(hs, name)
    call(**tensors, **rest)
    assert faked.launched == [name]              # all on the current device: it goes through
    for x in tensors.values():
        x.on = 1
        with pytest.raises(ValueError, match="device"):
            call(**tensors, **rest)
        x.on = -1
        with pytest.raises(TypeError):
            call(**tensors, **rest)
        x.on = 0
    faked.current[0] = 1
    with pytest.raises(ValueError, match="current"):
        call(**tensors, **rest)
    assert faked.launched == [name]


@pytest.mark.parametrize("name,change", [
    ("append_heads", dict(k=(4, 3, 64), v=(4, 3, 64))),          # not the pool's heads
    ("append_heads", dict(v=(4, 2, 128))), ("append_heads", dict(v=(3, 2, 64))), ("append_heads", dict(k=(4, 2, 32), v=(4, 2, 32))),
    ("append_heads", dict(cu=(2,))), ("append_heads", dict(cu=(4,))), ("append_heads", dict(ctx_len=(3,))),
    ("append_heads", dict(k=(3, 2, 64), v=(3, 2, 64), cu=None)),  # three tokens for two requests
    ("append_heads", dict(block_table=(6,))),
    ("read_heads", dict(k=(4, 2, 128))), ("read_heads", dict(k=(5, 2, 64))), ("read_heads", dict(start=(3,))), ("read_heads", dict(cu=(2,))),
    ("read_heads", dict(v=(4, 1, 64))), ("read_heads", dict(tokens=3, cu=None, k=(3, 2, 64), v=(3, 2, 64))),
    ("attend_heads", dict(out=(4, 6, 128))), ("attend_heads", dict(out=(4, 5, 64))), ("attend_heads", dict(lse=(4, 5))),
    ("attend_heads", dict(q=(4, 6, 96), out=(4, 6, 96))), ("attend_heads", dict(cu_q=(4,))), ("attend_heads", dict(ctx_len=(1,))),
    ("read_rows", dict(latent=(4, 511))), ("read_rows", dict(rope=(3, 64))), ("read_rows", dict(latent=(5, 512))),
])
def test_wrong_shapes_are_refused_before_a_launch(hs, faked, name, change):
    tensors, rest = arguments(hs, name)
    for key, shape in change.items():
        if key in rest:
            rest[key] = shape
        else:
            tensors[key] = shape and stand_in(*shape, dtype=tensors[key].dtype)
    with pytest.raises((ValueError, TypeError)):
        getattr(hs, name)(**tensors, **rest)
    assert faked.launched == []


@pytest.mark.parametrize("name,change", [
    ("append_heads", dict(k=F32)), ("append_heads", dict(k=torch.int8, v=torch.int8)), ("append_heads", dict(ctx_len=torch.int64)),
    ("append_heads", dict(block_table=torch.int64)), ("append_heads", dict(cu=torch.int64)), ("append_heads", dict(status=torch.int64)),
    ("read_heads", dict(k=F32)), ("read_heads", dict(k=torch.float64, v=torch.float64)), ("read_heads", dict(start=torch.int64)),
    ("attend_heads", dict(q=F32, out=F32)), ("attend_heads", dict(out=torch.float16)), ("attend_heads", dict(lse=torch.bfloat16)),
    ("attend_heads", dict(workspace=F32)), ("attend_heads", dict(cu_q=torch.int64)),
    ("read_rows", dict(rows=torch.int64)), ("read_rows", dict(rope=F32)), ("read_rows", dict(latent=torch.int8)),
])
def test_wrong_types_are_refused_before_a_launch(hs, faked, name, change):
    tensors, rest = arguments(hs, name)
    for key, dtype in change.items():
        tensors[key] = stand_in(*tensors[key].shape, dtype=dtype)
    with pytest.raises((ValueError, TypeError)):
        getattr(hs, name)(**tensors, **rest)
    assert faked.launched == []


def test_tensors_that_are_not_contiguous_where_they_must_be_are_refused(hs, faked):
    tensors, rest = arguments(hs, "attend_heads")
    for key, bad in (("q", stand_in(4, 64, 6).transpose(1, 2)), ("block_table", stand_in(3, 2, dtype=I32).t()),
                     ("lse", stand_in(6, 4, dtype=F32).t()), ("ctx_len", stand_in(4, dtype=I32)[::2])):
        with pytest.raises((ValueError, TypeError)):
            hs.attend_heads(**dict(tensors, **{key: bad}), **rest)
    assert faked.launched == []
