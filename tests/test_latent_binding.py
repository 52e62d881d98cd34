"""The latent-row operators' C boundary and binding, without a GPU."""
import ctypes
import os
import subprocess

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def hs():
    from sparse_mla_kv_gb300 import _build

    _build.build()
    import sparse_mla_kv_gb300

    return sparse_mla_kv_gb300


def test_structures_match_the_header(hs, tmp_path):
    from sparse_mla_kv_gb300 import latent

    lines = []
    for c, py in (("hs_append", latent.AppendC), ("hs_attend", latent.AttendC), ("hs_expanded", latent.ExpandedC)):
        lines.append(f'printf("{c} %zu\\n", sizeof({c}));')
        lines += [f'printf("{c}.{f} %zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "hs_latent.h"\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0; }\n")
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), "-I", cuda, str(src), "-o", str(tmp_path / "layout")])
    said = dict(line.split() for line in subprocess.check_output([str(tmp_path / "layout")], text=True).splitlines())
    for c, py in (("hs_append", latent.AppendC), ("hs_attend", latent.AttendC), ("hs_expanded", latent.ExpandedC)):
        assert int(said[c]) == ctypes.sizeof(py)
        for f, _ in py._fields_:
            assert int(said[f"{c}.{f}"]) == getattr(py, f).offset, (c, f)


def test_null_and_empty_arguments_are_refused_before_a_device_is_touched(hs):
    from sparse_mla_kv_gb300 import latent

    L = latent._lib()
    assert L.hs_append_rows(None, 0, None, None) == 1
    assert L.hs_append_rows(None, 0, ctypes.byref(latent.AppendC()), None) == 1
    assert L.hs_attend_rows(None, 0, None, 1, 1, None, None, 0, None) == 1
    assert L.hs_attend_rows(None, 0, None, -1, 1, ctypes.byref(latent.AttendC()), None, 0, None) == 1
    assert L.hs_attend_pages(None, 0, None, None, 1, 0, 1, ctypes.byref(latent.AttendC()), None, 0, None) == 1
    assert L.hs_attend_expanded(None, None) == 1
    for bad in (dict(heads=0), dict(heads=1025), dict(seqs=-1), dict(q_tokens=-1), dict(k_tokens=2 ** 31), dict(scale=float("nan"))):
        a = latent.ExpandedC(seqs=1, heads=1, q_tokens=1, k_tokens=1, scale=1.0)
        for f, x in bad.items():
            setattr(a, f, x)
        assert L.hs_attend_expanded(ctypes.byref(a), None) == 1, bad
    assert L.hs_attend_expanded(ctypes.byref(latent.ExpandedC(seqs=1, heads=1, q_tokens=1, k_tokens=1, scale=1.0)), None) == 1
    assert L.hs_attend_expanded(ctypes.byref(latent.ExpandedC(seqs=0, heads=1, scale=1.0)), None) == 0  # nothing to do


def test_cpu_tensors_and_wrong_shapes_raise(hs):
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        hs.attend_expanded(z(2, 1, 128), z(2, 1, 64), z(2, 1, 128), z(2, 64), z(2, 1, 128), i, i, 1.0)
    with pytest.raises(ValueError):
        hs.attend_expanded(z(2, 128), z(2, 1, 64), z(2, 1, 128), z(2, 64), z(2, 1, 128), i, i, 1.0)
    with pytest.raises(TypeError):
        hs.append_rows(None, i, z(2, 512), z(2, 64), i, torch.zeros(4, 64))
    with pytest.raises(TypeError):
        hs.append_rows(None, i, z(2, 512).to(torch.int16), z(2, 64), i, torch.zeros(4, 64))
    with pytest.raises(ValueError):
        hs.attend_rows(None, i, z(2, 1, 512), z(2, 1, 64), 1.0)
    with pytest.raises(TypeError):
        hs.attend_rows(None, i[None], z(1, 1, 512), z(1, 1, 64), 1.0)
    with pytest.raises(ValueError):
        hs.attend_pages(None, i[None], i, z(1, 1, 512), z(1, 1, 64), 1.0)
