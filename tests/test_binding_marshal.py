"""The binding's checking module (csrc/marshal.cpp): who needs it, and when it is built again."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    from mixture_experts_layer_pft_gb300 import build

    build.build()
    return build


def test_the_layer_s_calls_do_not_need_it():
    """Without the module the library loads and the layer's calls are answered; a call that needs it says what is missing."""
    code = """
import sys
sys.modules["mixture_experts_layer_pft_gb300._marshal"] = None  # importing it raises ImportError
import torch
from mixture_experts_layer_pft_gb300 import binding as B
assert B.workspace_size(B.MOE_OP_ALL, 64, 64, 4, 2, 64, torch.bfloat16) > 0
assert B.lib().moe_dispatch(None, None, -1, 2, 64, 1, None, None, 0, None) == B.MOE_ERR_INVALID_ARG
x = torch.zeros(4, 16)
try:
    B.moe_add_rmsnorm(x, None, torch.ones(16), 1e-6, None, x.clone(), None, None, None, x)
except RuntimeError as e:
    assert "_marshal" in str(e) and "build" in str(e), e
else:
    raise SystemExit("not refused")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def commands(build, monkeypatch):
    """What build() would run, without running it."""
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    build.build()
    return ran


def test_it_is_built_again_for_another_torch_or_python(built, monkeypatch):
    import torch

    key = built.MARSHAL_KEY
    monkeypatch.setattr(built, "MARSHAL_KEY", key + ".test")  # what is written here is not the tree's
    try:
        commands(built, monkeypatch)
        assert commands(built, monkeypatch) == []  # built for this torch and this Python
        monkeypatch.setattr(torch, "__version__", "0.0.1")
        ran = commands(built, monkeypatch)
        assert len(ran) == 1 and any(a.endswith("marshal.cpp") for a in ran[0])
        assert commands(built, monkeypatch) == []
        monkeypatch.setattr(sys, "version", "another")
        assert len(commands(built, monkeypatch)) == 1
    finally:
        if os.path.exists(key + ".test"):
            os.remove(key + ".test")
