"""The layer operators (include/gdn_layers.h) refuse bad arguments before touching a GPU, and the parts
of the binding that need none (CPU only: no call here enqueues work)."""
from __future__ import annotations

import ctypes
import math
import os

import pytest
import torch

import gated_deltanet_linear_17_b200 as gdn
from gated_deltanet_linear_17_b200 import _binding as B
from gated_deltanet_linear_17_b200 import _layers

M = 1 << 24  # fake, disjoint, 16-byte aligned addresses (never dereferenced)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        pytest.skip("libgdn.so not built")
    return _layers._layers_lib()


def _vp(x):
    return None if x is None else ctypes.c_void_p(x)


def _norm(lib, **over):
    a = dict(x=1 * M, residual=None, gate=None, weight=4 * M, eps=1e-6, offset=0.0, out=5 * M, residual_out=None,
             scales=None, rows=4, width=256, act=1, wdt=1, quant=0)
    a.update(over)
    return lib.gdn_rms_norm(_vp(a["x"]), _vp(a["residual"]), _vp(a["gate"]), _vp(a["weight"]), a["eps"], a["offset"],
                            _vp(a["out"]), _vp(a["residual_out"]), _vp(a["scales"]), a["rows"], a["width"], a["act"],
                            a["wdt"], a["quant"], None)


@pytest.mark.parametrize("over, code", [
    (dict(rows=-1), B.GDN_ERR_BAD_SHAPE),
    (dict(width=0), B.GDN_ERR_BAD_SHAPE),
    (dict(act=3), B.GDN_ERR_BAD_SHAPE),
    (dict(quant=3), B.GDN_ERR_BAD_SHAPE),
    (dict(quant=-1), B.GDN_ERR_BAD_SHAPE),
    (dict(act=1, wdt=2), B.GDN_ERR_BAD_SHAPE),               # a weight in the other 16-bit type
    (dict(width=32769), B.GDN_ERR_UNSUPPORTED),
    (dict(rows=1 << 31), B.GDN_ERR_UNSUPPORTED),
    (dict(rows=0), B.GDN_OK),
    (dict(rows=0, x=None), B.GDN_OK),
    (dict(x=None), B.GDN_ERR_NULL_ARG),
    (dict(weight=None), B.GDN_ERR_NULL_ARG),
    (dict(out=None), B.GDN_ERR_NULL_ARG),
    (dict(residual=2 * M), B.GDN_ERR_NULL_ARG),              # a residual without its output
    (dict(residual_out=2 * M), B.GDN_ERR_BAD_SHAPE),         # and the other way round
    (dict(quant=1), B.GDN_ERR_NULL_ARG),                     # 8 bits without scales
    (dict(scales=6 * M), B.GDN_ERR_BAD_SHAPE),               # scales without 8 bits
    (dict(x=M + 8), B.GDN_ERR_ALIGNMENT),
    (dict(weight=4 * M + 2), B.GDN_ERR_ALIGNMENT),
    (dict(quant=1, scales=6 * M + 2), B.GDN_ERR_ALIGNMENT),
    (dict(out=M + 16), B.GDN_ERR_OVERLAP),                   # out on x, but not x itself
    (dict(quant=1, scales=6 * M, out=M), B.GDN_ERR_OVERLAP),  # 8 bits cannot go in place
    (dict(gate=5 * M), B.GDN_ERR_OVERLAP),
    (dict(out=4 * M), B.GDN_ERR_OVERLAP),                    # on the weight
    (dict(residual=2 * M, residual_out=M), B.GDN_ERR_OVERLAP),   # the residual's output on x
    (dict(residual=2 * M, residual_out=5 * M), B.GDN_ERR_OVERLAP),  # on out
    (dict(residual=2 * M, residual_out=2 * M + 16), B.GDN_ERR_OVERLAP),
    (dict(quant=2, scales=5 * M + 512), B.GDN_ERR_OVERLAP),
    (dict(residual=2 * M, residual_out=2 * M, out=2 * M), B.GDN_ERR_OVERLAP),
    (dict(x=2 * M, residual=2 * M, residual_out=2 * M), B.GDN_ERR_OVERLAP),  # x is the residual: not in place
])
def test_norm_refusals(lib, over, code):
    assert _norm(lib, **over) == code


def _rope(lib, **over):
    a = dict(q=1 * M, k=2 * M, v=None, positions=3 * M, freq=4 * M, slots=None, mscale=1.0, q_out=5 * M, k_out=6 * M,
             kc=None, vc=None, T=3, Hq=4, Hkv=2, D=64, rotary=32, inter=0, rows=0, act=1)
    a.update(over)
    return lib.gdn_rope_fwd(_vp(a["q"]), _vp(a["k"]), _vp(a["v"]), _vp(a["positions"]), _vp(a["freq"]),
                            _vp(a["slots"]), a["mscale"], _vp(a["q_out"]), _vp(a["k_out"]), _vp(a["kc"]),
                            _vp(a["vc"]), a["T"], a["Hq"], a["Hkv"], a["D"], a["rotary"], a["inter"], a["rows"],
                            a["act"], None)


CACHE = dict(v=7 * M, slots=8 * M, kc=9 * M, vc=10 * M, rows=64, k_out=None)


@pytest.mark.parametrize("over, code", [
    (dict(T=-1), B.GDN_ERR_BAD_SHAPE),
    (dict(Hq=0), B.GDN_ERR_BAD_SHAPE),
    (dict(Hkv=0), B.GDN_ERR_BAD_SHAPE),
    (dict(rotary=31), B.GDN_ERR_BAD_SHAPE),
    (dict(rotary=66), B.GDN_ERR_BAD_SHAPE),
    (dict(rotary=-2), B.GDN_ERR_BAD_SHAPE),
    (dict(act=7), B.GDN_ERR_BAD_SHAPE),
    (dict(D=60), B.GDN_ERR_UNSUPPORTED),
    (dict(D=264), B.GDN_ERR_UNSUPPORTED),
    (dict(T=1 << 31), B.GDN_ERR_UNSUPPORTED),
    (dict(CACHE, rows=1 << 31), B.GDN_ERR_UNSUPPORTED),
    (dict(T=0), B.GDN_OK),
    (dict(q=None), B.GDN_ERR_NULL_ARG),
    (dict(positions=None), B.GDN_ERR_NULL_ARG),
    (dict(freq=None), B.GDN_ERR_NULL_ARG),
    (dict(k_out=None), B.GDN_ERR_NULL_ARG),                  # nowhere for the keys to go
    (dict(CACHE, v=None), B.GDN_ERR_NULL_ARG),
    (dict(CACHE, slots=None), B.GDN_ERR_NULL_ARG),
    (dict(CACHE, vc=None), B.GDN_ERR_NULL_ARG),
    (dict(v=7 * M), B.GDN_ERR_BAD_SHAPE),                    # values without a cache
    (dict(slots=7 * M), B.GDN_ERR_BAD_SHAPE),
    (dict(q=M + 4), B.GDN_ERR_ALIGNMENT),
    (dict(CACHE, kc=9 * M + 8), B.GDN_ERR_ALIGNMENT),
    (dict(positions=3 * M + 2), B.GDN_ERR_ALIGNMENT),
    (dict(q_out=M + 16), B.GDN_ERR_OVERLAP),
    (dict(q_out=2 * M), B.GDN_ERR_OVERLAP),                  # on k
    (dict(k_out=5 * M), B.GDN_ERR_OVERLAP),                  # on q_out
    (dict(CACHE, kc=7 * M), B.GDN_ERR_OVERLAP),              # the cache on v
    (dict(CACHE, vc=9 * M + 64), B.GDN_ERR_OVERLAP),         # the caches on one another
    (dict(k=M, q_out=M), B.GDN_ERR_OVERLAP),                 # q in place while k reads it
])
def test_rope_refusals(lib, over, code):
    assert _rope(lib, **over) == code


def _attn(lib, **over):
    a = dict(q=1 * M, k=2 * M, v=3 * M, table=4 * M, lens=5 * M, scale=0.0, out=6 * M, lse=7 * M, B=2, Hq=4, Hkv=2,
             D=64, P=8, page=16, max_pages=4, max_seqlen=0, act=1, ws=None, wsb=0)
    a.update(over)
    return lib.gdn_paged_attn_fwd(_vp(a["q"]), _vp(a["k"]), _vp(a["v"]), _vp(a["table"]), _vp(a["lens"]), a["scale"],
                                  _vp(a["out"]), _vp(a["lse"]), a["B"], a["Hq"], a["Hkv"], a["D"], a["P"], a["page"],
                                  a["max_pages"], a["max_seqlen"], a["act"], _vp(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("over, code", [
    (dict(B=-1), B.GDN_ERR_BAD_SHAPE),
    (dict(Hq=3), B.GDN_ERR_BAD_SHAPE),
    (dict(Hkv=0), B.GDN_ERR_BAD_SHAPE),
    (dict(page=0), B.GDN_ERR_BAD_SHAPE),
    (dict(max_pages=-1), B.GDN_ERR_BAD_SHAPE),
    (dict(max_seqlen=-1), B.GDN_ERR_BAD_SHAPE),
    (dict(P=-1), B.GDN_ERR_BAD_SHAPE),
    (dict(act=4), B.GDN_ERR_BAD_SHAPE),
    (dict(act=0), B.GDN_ERR_UNSUPPORTED),                    # fp32
    (dict(D=80), B.GDN_ERR_UNSUPPORTED),
    (dict(P=1 << 28), B.GDN_ERR_UNSUPPORTED),                # 2^32 cache rows
    (dict(max_pages=1 << 28), B.GDN_ERR_UNSUPPORTED),
    (dict(B=0), B.GDN_OK),
    (dict(q=None), B.GDN_ERR_NULL_ARG),
    (dict(k=None), B.GDN_ERR_NULL_ARG),
    (dict(table=None), B.GDN_ERR_NULL_ARG),
    (dict(lens=None), B.GDN_ERR_NULL_ARG),
    (dict(out=None), B.GDN_ERR_NULL_ARG),
    (dict(q=M + 2), B.GDN_ERR_ALIGNMENT),
    (dict(lens=5 * M + 1), B.GDN_ERR_ALIGNMENT),
    (dict(out=M), B.GDN_ERR_OVERLAP),                        # on q
    (dict(out=2 * M), B.GDN_ERR_OVERLAP),
    (dict(lse=6 * M), B.GDN_ERR_OVERLAP),
    (dict(page=256, max_pages=256, ws=8 * M, wsb=16), B.GDN_ERR_WORKSPACE),
    (dict(page=256, max_pages=256, ws=8 * M + 8, wsb=1 << 30), B.GDN_ERR_ALIGNMENT),
    (dict(page=256, max_pages=256, ws=3 * M, wsb=1 << 30), B.GDN_ERR_OVERLAP),  # the workspace on the values
])
def test_attn_refusals(lib, over, code):
    assert _attn(lib, **over) == code


def test_attn_workspace_bytes(lib):
    assert gdn.paged_attn_workspace_bytes(0, 8, 2, 128, 16, 64) == 0
    assert gdn.paged_attn_workspace_bytes(1, 7, 2, 128, 16, 64) == 0         # refused sizes
    long = gdn.paged_attn_workspace_bytes(1, 8, 2, 128, 16, 8192)
    assert long > 0 and long == gdn.paged_attn_workspace_bytes(1, 8, 2, 128, 16, 8192, 1 << 17)
    # a hint beyond the table is the table's own capacity; a short one needs no more than the capacity
    assert gdn.paged_attn_workspace_bytes(1, 8, 2, 128, 16, 8192, 1 << 30) == long
    assert gdn.paged_attn_workspace_bytes(1, 8, 2, 128, 16, 8192, 1) <= long


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(RuntimeError):
        gdn.rms_norm(x, x[0])
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(RuntimeError):
        gdn.rope_fwd(q, q, torch.zeros(2, dtype=torch.int32), torch.zeros(8))
    with pytest.raises(RuntimeError):
        gdn.paged_attn_fwd(q, q[None], q[None], torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError):
        gdn.rms_norm([1.0], x[0])


def test_inv_freq():
    f, m = gdn.rope_inv_freq(64, base=10000.0, device="cpu")
    want = torch.tensor([10000.0 ** (-2 * i / 64) for i in range(32)], dtype=torch.float64)
    assert f.dtype == torch.float32 and f.shape == (32,) and m == 1.0
    assert torch.equal(f, want.float())
    lin, m = gdn.rope_inv_freq(64, scaling="linear", factor=4.0, device="cpu")
    assert torch.equal(lin, (want / 4).float()) and m == 1.0
    ntk, m = gdn.rope_inv_freq(64, scaling="ntk", factor=4.0, device="cpu")
    assert m == 1.0 and ntk[0] == 1.0                                        # the fastest angle is kept
    assert abs(ntk[-1].item() / (want[-1].item() / 4) - 1) < 1e-6             # the slowest divided by the factor
    yarn, m = gdn.rope_inv_freq(64, scaling="yarn", factor=4.0, original_max=4096, device="cpu")
    assert m == 0.1 * math.log(4.0) + 1.0
    turns = 4096 * want / (2 * math.pi)
    ratio = yarn.double() / want
    # beyond a whole index (the ramp's ends are rounded outwards) of beta_fast and beta_slow turns
    one = (want[1] / want[0]).item()
    assert torch.allclose(ratio[turns > 32 / one], torch.tensor(1.0, dtype=torch.float64), atol=1e-6)
    assert torch.allclose(ratio[turns < 1 * one], torch.tensor(0.25, dtype=torch.float64), atol=1e-6)
    assert (ratio[1:] <= ratio[:-1] + 1e-7).all()
    same, m = gdn.rope_inv_freq(64, scaling="yarn", factor=1.0, device="cpu")
    assert torch.allclose(same.double(), want, rtol=1e-6) and m == 1.0
    for bad in (dict(rotary=7), dict(rotary=0), dict(rotary=64, scaling="other"), dict(rotary=64, base=1.0),
                dict(rotary=64, factor=0.5), dict(rotary=64, beta_fast=1.0, beta_slow=2.0)):
        with pytest.raises(ValueError):
            gdn.rope_inv_freq(device="cpu", **bad)
