"""The wrappers' host-side shortcut without a GPU: it is used with the torch it was
compiled against alone."""
import importlib
import os
import sys
import types

import pytest
import torch


@pytest.fixture(scope="module")
def ops():
    from rmsnorm_fp8_quantization_gb300 import _build
    _build.build()
    from rmsnorm_fp8_quantization_gb300 import ops as o
    return o


def test_it_says_what_it_was_compiled_against(ops):
    from rmsnorm_fp8_quantization_gb300 import _build
    assert ops._fast is not None and ops._fast.built_for == _build.torch_tag()
    assert torch.__version__ in _build.torch_tag() and _build.fastcall_up_to_date()


@pytest.mark.parametrize("built_for", [None, "2.0.0 0123"])
def test_one_compiled_against_another_torch_is_not_used(ops, monkeypatch, built_for):
    def never(*a):
        raise AssertionError("used")
    other = types.ModuleType("rmsnorm_fp8_quantization_gb300._fastcall")
    other.setup = never
    if built_for is not None:
        other.built_for = built_for
    import rmsnorm_fp8_quantization_gb300 as package
    monkeypatch.setitem(sys.modules, other.__name__, other)
    monkeypatch.setattr(package, "_fastcall", other, raising=False)
    assert ops._shortcut() is None


def test_it_is_compiled_again_for_another_torch(ops, monkeypatch, tmp_path):
    from rmsnorm_fp8_quantization_gb300 import _build
    calls = []
    monkeypatch.setattr(_build, "build_fastcall", lambda: calls.append(1))
    monkeypatch.setattr(_build, "up_to_date", lambda: True)
    assert _build.build() == _build.LIB and calls == []
    stamp = tmp_path / "stamp"
    stamp.write_text("2.0.0 0123")
    monkeypatch.setattr(_build, "FAST_STAMP", str(stamp))
    assert _build.build() == _build.LIB and calls == [1]
    monkeypatch.setattr(_build, "FAST_STAMP", str(tmp_path / "none"))
    assert _build.build() == _build.LIB and calls == [1, 1]
    assert importlib.machinery.EXTENSION_SUFFIXES[0] in os.path.basename(_build.FAST)


@pytest.mark.parametrize("missing", ["toolkit", "compiler", "room"])
def test_a_build_without_it_goes_on(ops, monkeypatch, tmp_path, capsys, missing):
    """The library is there, the shortcut is not, and nothing can compile it."""
    from rmsnorm_fp8_quantization_gb300 import _build

    def refuse(*a, **k):
        raise OSError("read-only") if missing == "room" else RuntimeError("nvcc not found")
    monkeypatch.setattr(_build, "up_to_date", lambda: True)
    monkeypatch.setattr(_build, "FAST", str(tmp_path / "_fastcall.so"))
    monkeypatch.setattr(_build, "FAST_STAMP", str(tmp_path / "stamp"))
    if missing == "toolkit":
        monkeypatch.setattr(_build, "_nvcc", refuse)
    elif missing == "compiler":
        monkeypatch.setattr(_build.shutil, "which", lambda n: None)
    else:
        monkeypatch.setattr(_build.subprocess, "run", refuse)
    assert _build.build() == _build.LIB
    assert "not built" in capsys.readouterr().err and not list(tmp_path.iterdir())


def test_numbers_beyond_a_float_are_left_to_the_wrapper(ops):
    """The shortcut says that it is not its call, with no exception set; the wrapper raises."""
    fast = ops._fast
    q, k = torch.zeros(2, 3, 4, 64), torch.zeros(2, 3, 2, 64)
    f, pos = torch.zeros(32, dtype=torch.float64), torch.zeros(2, 3, dtype=torch.int64)
    for mscale in (10 ** 400, -10 ** 400, 1e300):
        assert fast.rope(0, q, k, f, pos, 0, mscale) is None
    b = torch.zeros(2, 4, 64)
    cache = torch.zeros(2, 16, 4, 64)
    i = torch.zeros(2, dtype=torch.int32)
    assert fast.append(b, b, cache, cache, i, i, i, b, f, 0, 10 ** 400, None, None) is None
