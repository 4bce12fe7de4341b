"""The binding's host side: what it imports, asks torch for and remembers (no GPU)."""
import os
import subprocess
import sys
import types

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def lib():
    from exact_attention_14_gb300 import _build
    _build.build()


def test_plans_need_no_torch():
    """The package and its host-only functions, where torch cannot be imported at all."""
    code = """
import sys
sys.modules["torch"] = None                       # an import of torch raises
import exact_attention_14_gb300 as ea
assert ea.attn_decode_num_splits(4, 8, 4096) >= 1
assert ea.attn_fwd_num_units(1, 4, 4, 512, 512, 128, True) >= 1
assert ea.attn_kv_tiles(0, 256, 512, 512, 128, 1) >= 1
f, mag = ea.attn_rope_frequencies(64, 10000.0)
assert len(f) == 32 and mag == 1.0
assert ea.attn_status_string(0) == "ATTN_OK"
try:
    ea.rope(None, None, None, None)
except ImportError:
    print("ok")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr


def test_torch_comes_with_the_first_call_that_needs_it():
    code = """
import sys
import exact_attention_14_gb300 as ea
assert "torch" not in sys.modules
ea.attn_rope_frequencies(64, 10000.0)
assert "torch" not in sys.modules
try:
    ea.rope([], None, None, None)
except TypeError as e:
    assert "torch.Tensor" in str(e)
import torch
assert ea.torch is torch
m = ea.tree_mask_words(torch.ones(1, 2, 2, dtype=torch.bool))
print(m.flatten().tolist())
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "[3, 3]", r.stderr


def test_current_stream_without_torch_internals(monkeypatch):
    """Where torch does not have its internal call, its public ones give the same handle."""
    import torch

    import exact_attention_14_gb300 as ea
    ea.tree_mask_words(torch.ones(1, 1, 1, dtype=torch.bool))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: types.SimpleNamespace(cuda_stream=1000 + d))
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        monkeypatch.delattr(torch._C, name, raising=False)
    assert ea._stream_ptr(None) == 1003
    assert ea._on(torch.device("cuda", 3)) is ea._HERE
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 2000 + d, raising=False)
    assert ea._stream_ptr(None) == 2003


def test_a_workspace_size_of_zero_is_not_remembered(monkeypatch):
    """A device that did not answer once, or a shape that was refused, does not stay at 0 bytes."""
    import exact_attention_14_gb300 as ea
    sizes = [0, 0, 4096, 8192]
    asked = []

    def size(*a):
        asked.append(a)
        return sizes[len(asked) - 1]
    monkeypatch.setattr(ea, "load", lambda: types.SimpleNamespace(attn_decode_tree_workspace_size=size))
    args = (6, 2, 5, 96, 0, 77)
    assert [ea._tree_workspace(*args) for _ in range(4)] == [0, 0, 4096, 4096]
    assert len(asked) == 3
