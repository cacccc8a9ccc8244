"""What the layer operators refuse beyond the sizes and pointers of test_layers_abi.py, and what their binding takes from
torch (CPU only: no call here enqueues work)."""
from __future__ import annotations

import math
import os
import subprocess
import sys

import pytest
import torch

import gated_deltanet_linear_17_b200 as gdn
from gated_deltanet_linear_17_b200 import _binding as B
from test_layers_abi import _attn, lib  # noqa: F401 (a fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), 3e38, 2.4e38])
def test_attn_refuses_a_scale_that_is_no_number(lib, scale):  # noqa: F811
    """Taken as a scale these give rows of NaN, and a NaN is neither positive nor the default's sign."""
    assert _attn(lib, scale=scale) == B.GDN_ERR_BAD_SHAPE
    assert _attn(lib, scale=scale, B=0) == B.GDN_ERR_BAD_SHAPE


@pytest.mark.parametrize("scale", [0.0, -1.0, float("-inf"), 1e-45, 2.3e38])
def test_attn_takes_other_scales(lib, scale):  # noqa: F811
    assert _attn(lib, scale=scale, B=0) == B.GDN_OK


def test_package_imports_without_torch_s_private_functions():
    """A torch that has renamed them, or is built without CUDA, still imports the package; the public ones serve."""
    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import gated_deltanet_linear_17_b200 as gdn
from gated_deltanet_linear_17_b200 import _layers
assert _layers._current_device is torch.cuda.current_device
assert _layers._current_stream is _layers._stream_handle
try:
    gdn.rms_norm(torch.zeros(2, 8), torch.zeros(8))
except RuntimeError as e:
    assert "CUDA device" in str(e)
else:
    raise SystemExit("a host tensor was taken")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT, timeout=600)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("original_max", [1, 4, 6, 7, 40, 4096, 1 << 20])
@pytest.mark.parametrize("rotary", [2, 8, 64, 128])
def test_yarn_divides_every_slow_angle(original_max, rotary):
    """An angle that turns at most beta_slow times over original_max positions is divided by the factor, the first too;
    one that turns at least beta_fast times is kept; the others lie between."""
    plain, _ = gdn.rope_inv_freq(rotary, device="cpu")
    yarn, _ = gdn.rope_inv_freq(rotary, scaling="yarn", factor=8.0, original_max=original_max, device="cpu")
    turns = original_max * 10000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / rotary) / (2 * math.pi)
    ratio = yarn.double() / plain.double()
    assert torch.allclose(ratio[turns <= 1.0], torch.tensor(0.125, dtype=torch.float64), rtol=2.0 ** -22)
    assert torch.allclose(ratio[turns >= 32.0], torch.tensor(1.0, dtype=torch.float64), rtol=2.0 ** -22)
    assert ((ratio >= 0.125 - 1e-6) & (ratio <= 1 + 1e-6)).all()
