"""The binding's compiled half is for one Python and one torch, and what cannot be built or loaded of it is left
out: every call then takes the Python half."""
import os
import sysconfig

import pytest
import torch

from gqa_attention_paged_b200 import binding, build


@pytest.fixture
def fresh(monkeypatch, tmp_path):
    """The binding as it is before its first call, with no compiled half."""
    for name in ("_lib", "_fast", "_fast_off"):
        monkeypatch.setattr(binding, name, None)
    monkeypatch.setattr(build, "FASTCALL", str(tmp_path / "_fastcall.so"))


def python_half_serves():
    lib = binding.load()
    assert binding._fast is None and binding._fast_off
    assert lib.gqa_pick_splits(1, 8, 16, 16, 0) == 1
    p, i32 = binding.new_fp4_pool(4, 2, 16, 64, "cpu"), torch.zeros(3, 4, dtype=torch.int32)
    q, ws = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(1 << 12, dtype=torch.uint8)
    for _ in range(2):
        with pytest.raises(ValueError, match="CUDA"):
            binding.gqa_paged_decode(q, p, p, i32, i32[:, 0], 0.1, out=q, workspace=ws, want_lse=False)


def test_name():
    name = os.path.basename(build.FASTCALL)
    assert torch.__version__ in name and name.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    binding.load()
    assert binding._fast is not None and binding._fast_off is None
    assert binding._fast.__spec__.loader.path == build.FASTCALL


def test_no_compiler(fresh, monkeypatch, capsys):
    monkeypatch.setattr(build, "CXX", "/nonexistent/g++")
    assert "/nonexistent/g++" in build.build_fastcall()
    python_half_serves()
    assert "/nonexistent/g++" in binding._fast_off
    # the library's own build is none the worse for it
    assert build.build() == build.LIB
    assert "left out" in capsys.readouterr().err


def test_sources_that_do_not_compile(fresh, monkeypatch, tmp_path):
    monkeypatch.setattr(build, "_torch_include", lambda: str(tmp_path))  # no ATen/dlpack.h
    assert "dlpack.h" in build.build_fastcall()
    assert not os.listdir(tmp_path)
    python_half_serves()


def test_a_file_that_does_not_load(fresh):
    with open(build.FASTCALL, "wb") as f:
        f.write(b"not a shared object")
    python_half_serves()


def test_a_missing_one_is_built(fresh):
    binding.load()
    assert binding._fast is not None and os.path.exists(build.FASTCALL)
    assert not build._fastcall_stale()
