"""The wrappers are imported, and an optimiser steps, in a program without numpy."""

import os
import subprocess
import sys

CODE = """
import contextlib, sys, warnings
sys.modules["numpy"] = None
warnings.simplefilter("ignore")
import torch
from moe_layer_router_amd import layer as L, lib

class P(torch.Tensor):
    is_cuda = True

seen = []
L._on = lambda *a: contextlib.nullcontext()
lib.moe_adamw = lambda table, options: seen.append([(r.param, r.grad, r.grad_dtype) for r in table])
p = [torch.zeros(8).as_subclass(P), torch.zeros(16).as_subclass(P)]
g = [torch.ones(8), torch.ones(16).to(torch.bfloat16)]
L.AdamW(p).step(g, 1e-3)
assert seen == [[(a.data_ptr(), b.data_ptr(), t) for a, b, t in zip(p, g, (lib.MOE_DTYPE_F32, lib.MOE_DTYPE_BF16))]]
print("stepped")
"""


def test_without_numpy():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CODE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "stepped" in r.stdout, r.stderr[-2000:]
