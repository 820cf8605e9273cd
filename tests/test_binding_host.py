"""What the Python binding says about a library that is not the one it was written for."""
import ctypes
import subprocess

import pytest

from matrix_optimizer_muon_amd import _binding as B


def other_library(tmp_path, monkeypatch, names, version):
    src = "".join(f"int {n}(void) {{ return {version if n == 'dmuon_abi_version' else 0}; }}\n" for n in names)
    (tmp_path / "lib.c").write_text(src)
    path = str(tmp_path / "lib.so")
    subprocess.run(["gcc", "-shared", "-fPIC", str(tmp_path / "lib.c"), "-o", path], check=True)
    monkeypatch.setattr(B, "LIB_PATH", path)
    monkeypatch.setattr(B, "_lib", None)
    return path


@pytest.mark.parametrize("names,version,says", [
    ([n for n in B.EXPORTED if "ckpt8" not in n and "linear_ce" not in n and "embedding" not in n], B.ABI_VERSION, "lacks"),   # before the training gradients
    (B.EXPORTED[:4], B.ABI_VERSION, "lacks"), (["other"], 0, "lacks"),
    (B.EXPORTED, B.ABI_VERSION - 1, f"has ABI {B.ABI_VERSION - 1}"), (["dmuon_abi_version"], B.ABI_VERSION + 1, f"has ABI {B.ABI_VERSION + 1}")])
def test_another_library_is_named_and_not_kept(tmp_path, monkeypatch, names, version, says):
    path = other_library(tmp_path, monkeypatch, names, version)
    for _ in range(2):
        with pytest.raises(RuntimeError) as e:
            B.lib()
        assert path in str(e.value) and says in str(e.value) and "rebuild" in str(e.value)


def test_a_library_that_is_whole_is_taken(tmp_path, monkeypatch):
    path = other_library(tmp_path, monkeypatch, B.EXPORTED, B.ABI_VERSION)
    assert B.lib()._name == path
    assert B.lib().dmuon_last_error.restype is ctypes.c_char_p
