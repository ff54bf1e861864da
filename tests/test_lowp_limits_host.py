"""Host-side limits of the microscaled 4-bit and 8-bit KV cache entry points
(no GPU needed)."""
import sys

import pytest
import torch

import weight_only_int4_quantize_b200 as w4
from tests.test_lowp_host import A, B, lib  # noqa: F401
from weight_only_int4_quantize_b200 import build


@pytest.mark.parametrize("big", [(1 << 31) - 1, (1 << 31) - 257, (1 << 31) - 300, (1 << 31) - 383])
def test_linear_sizes_that_overflow_the_tile_arithmetic(lib, big):  # noqa: F811
    """A tile of 384 tokens reaches past the last one, and the rows that it
    counts there have to be 32-bit numbers."""
    assert lib.w4_fp4_linear(A, A, None, big, A, A, None, 8, 128, 0, B, 0, None) == 2


def test_values_without_a_truth_value(lib):  # noqa: F811
    """The error of asking for it reaches the caller before anything runs."""
    with pytest.raises(RuntimeError, match="ambiguous"):
        w4.fp4_quantize(torch.zeros(1, 128, dtype=torch.bfloat16), "mx", values=torch.ones(2))


def test_library_builds_where_torch_is_missing(tmp_path, monkeypatch, capsys):
    """libw4.so needs no torch: a user of the C ABI alone can build it.  The
    tensor front end is left out, and said to be."""
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libw4.so"))
    monkeypatch.setattr(build, "TENSORS", str(tmp_path / "_tensors.so"))
    ran = []

    def run(cmd, check):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build() == str(tmp_path / "libw4.so")
    assert ran and not any("tensors.cpp" in a for cmd in ran for a in cmd)
    assert "_tensors" in capsys.readouterr().err


def test_extension_that_cannot_be_loaded_says_why(lib, monkeypatch):  # noqa: F811
    """Built, but against another torch: not reported as missing."""
    class Broken:
        def find_spec(self, name, path=None, target=None):
            if name.endswith("._tensors"):
                raise ImportError("undefined symbol: of_another_torch")

    name = w4.__name__ + "._tensors"
    monkeypatch.setattr(w4, "_TENSORS", None)
    monkeypatch.delattr(w4, "_tensors", raising=False)
    monkeypatch.delitem(sys.modules, name, raising=False)
    monkeypatch.setattr(sys, "meta_path", [Broken(), *sys.meta_path])
    with pytest.raises(RuntimeError, match="no fallback") as e:
        w4.fp4_quantize(torch.zeros(1, 128, dtype=torch.bfloat16))
    assert "of_another_torch" in str(e.value) and "missing" not in str(e.value)
