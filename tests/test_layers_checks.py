"""What the layer operators refuse beyond the sizes and pointers of test_layers_abi.py, and what their binding takes from
torch (CPU only: no call here enqueues work)."""
from __future__ import annotations

import pytest

from gated_deltanet_linear_17_b200 import _binding as B
from test_layers_abi import _attn, lib  # noqa: F401 (a fixture)


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), 3e38, 2.4e38])
def test_attn_refuses_a_scale_that_is_no_number(lib, scale):  # noqa: F811
    """Taken as a scale these give rows of NaN, and a NaN is neither positive nor the default's sign."""
    assert _attn(lib, scale=scale) == B.GDN_ERR_BAD_SHAPE
    assert _attn(lib, scale=scale, B=0) == B.GDN_ERR_BAD_SHAPE


@pytest.mark.parametrize("scale", [0.0, -1.0, float("-inf"), 1e-45, 2.3e38])
def test_attn_takes_other_scales(lib, scale):  # noqa: F811
    assert _attn(lib, scale=scale, B=0) == B.GDN_OK
