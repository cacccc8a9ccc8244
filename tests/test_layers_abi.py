"""The layer operators (include/gdn_layers.h) refuse bad arguments before touching a GPU, and the parts
of the binding that need none (CPU only: no call here enqueues work)."""
from __future__ import annotations

import ctypes
import math
import os
import random

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
    (dict(width=32776), B.GDN_ERR_UNSUPPORTED),
    (dict(width=32761), B.GDN_ERR_UNSUPPORTED),               # no whole number of blocks, and no room for one more
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


# ------------------------------------------------------------------ how the paged attention cuts its work


def _split(lib, lens, heads, D, capacity, ctas):
    cap = 4 * (len(lens) * heads + ctas)
    rows = (ctypes.c_int32 * (7 * cap))()
    n = lib.gdn_testing_attn_split((ctypes.c_int32 * len(lens))(*lens), len(lens), heads, D, ctypes.c_int64(capacity),
                                   ctas, rows, cap)
    assert n >= 0
    return [tuple(rows[7 * i:7 * i + 7]) for i in range(n)]


def _check_split(lib, lens, heads, D, capacity, ctas):
    pieces = _split(lib, lens, heads, D, capacity, ctas)
    keys, places, begun = {}, set(), {}
    for cta, b, group, k0, k1, place, count in pieces:
        assert 0 <= cta < ctas and 0 <= k0 <= max(k0, k1)
        keys.setdefault((b, group), []).append((k0, k1, cta, place, count))
        if place < 2:                                     # one result a place
            assert (cta, place) not in places
            places.add((cta, place))
        if count:
            assert place == 1 and cta not in begun
            begun[cta] = (b, group, count)
    assert set(keys) == {(b, g) for b in range(len(lens)) for g in range(heads)}
    for (b, group), parts in keys.items():
        n = lens[b] if 0 <= lens[b] <= capacity else 0
        at = 0
        for k0, k1, *_ in parts:                          # every key once, in order
            if k1 > k0:
                assert k0 == at
                at = k1
        assert at == n
        if len(parts) == 1:
            assert parts[0][3] == 2 and parts[0][4] == 0
        else:                                             # neighbouring CTAs, found from the first
            first = parts[0][2]
            assert [p[2] for p in parts] == list(range(first, first + len(parts)))
            assert [p[3] for p in parts] == [1] + [0] * (len(parts) - 1)
            assert begun[first] == (b, group, len(parts))
    total = max(1, sum(k1 - k0 for _, _, _, k0, k1, _, _ in pieces if k1 > k0))
    return pieces, total


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attn_split_covers_every_key_once(lib, D):
    r = random.Random(D)
    _check_split(lib, [0], 1, D, 0, 2)
    _check_split(lib, [131072], 2, D, 131072, 296)
    _check_split(lib, [1] * 500, 3, D, 64, 444)
    _check_split(lib, [-5, 70, 4097, 64], 5, D, 4096, 148)  # refused lengths: one piece without keys
    _check_split(lib, [1 << 30, 17], 1, D, 1 << 30, 296)    # a list beyond 2^22 places
    for _ in range(150):
        B = r.choice([1, 2, 7, 33, 200])
        longest = r.choice([1, 63, 64, 65, 1000, 20000])
        lens = [r.choice([0, 1, 64, r.randint(0, longest)]) for _ in range(B)]
        _check_split(lib, lens, r.choice([1, 2, 8, 12]), D, 20000, r.choice([2, 3, 148, 296, 444]))


def test_attn_split_is_even(lib):
    """No CTA takes more than a unit of keys over the mean of an even batch."""
    pieces, total = _check_split(lib, [16384] * 16, 2, 256, 16384, 296)
    work = [0] * 296
    for cta, _, _, k0, k1, _, _ in pieces:
        work[cta] += max(0, k1 - k0)
    assert max(work) <= total / 296 + 64


@pytest.mark.parametrize("cluster", [1, 2, 4, 8])
def test_attn_cluster_covers_every_key_once(lib, cluster):
    k0, k1 = ctypes.c_int32(), ctypes.c_int32()
    for n in list(range(0, 300)) + [2047, 2048, 2049, (1 << 30) - 1, 1 << 30]:
        at = 0
        for rank in range(cluster):
            assert lib.gdn_testing_attn_cluster(n, cluster, rank, ctypes.byref(k0), ctypes.byref(k1)) == 0
            assert k0.value <= k1.value <= n
            if k1.value > k0.value:
                assert k0.value == at and k0.value % 16 == 0
                at = k1.value
        assert at == n


def test_attn_rows_stay_in_the_cache(lib):
    """The cache row of every key, and -1 for every page outside the cache, whatever the table holds."""
    r = random.Random(0)
    for page_size in (1, 2, 7, 16, 17, 24, 64, 100, 1 << 20):
        P = min(1000, ((1 << 31) - 1) // page_size)
        pages = [r.choice([0, P - 1, r.randrange(P), -1, P, P + 1, (1 << 31) - 1, -(1 << 31)]) for _ in range(40)]
        table = (ctypes.c_int32 * 40)(*pages)
        js = {0, 40 * page_size - 1} | {r.randrange(40 * page_size) for _ in range(300)}
        js |= {p * page_size + d for p in range(1, 40) for d in (-1, 0)}
        for j in js:
            row = lib.gdn_testing_attn_row(table, j, page_size, P)
            page = pages[j // page_size]
            assert row == (page * page_size + j % page_size if 0 <= page < P else -1)
            assert row < P * page_size


@pytest.mark.parametrize("rows", [(1 << 31) - 1, (1 << 31) - 31])
def test_norm_refuses_rows_whose_numbers_would_wrap(lib, rows):
    """Eight rows of four columns share a warp; the numbers of those behind the last row have to fit too."""
    assert _norm(lib, x=1 << 40, weight=1 << 50, out=1 << 45, rows=rows, width=1) == B.GDN_ERR_UNSUPPORTED


def test_attn_workspace_of_many_sequences_without_pages(lib):
    """More pairs than clusters are launched for, and a table without columns: still a list with CTAs."""
    none = gdn.paged_attn_workspace_bytes(1 << 24, 1, 1, 64, 16, 0)
    assert none > 0 and none == gdn.paged_attn_workspace_bytes(1 << 24, 1, 1, 64, 16, 4)
