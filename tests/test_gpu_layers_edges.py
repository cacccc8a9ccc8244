"""The layer operators on the GPU where two calls meet and where the arithmetic is at its limits: host threads that
call one operator at once, and inputs whose sizes lie far apart.  Formulas and tolerances are those of
test_gpu_layers.py; what a test adds to them stands in its docstring."""
from __future__ import annotations

import ctypes
import threading

import pytest
import torch

import gated_deltanet_linear_17_b200 as gdn
from gated_deltanet_linear_17_b200 import _layers
from test_gpu_layers import BF16, F16, F32, HALF, TINY, Paged, attn64, gen, norm64, randn, within

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ norm


@pytest.mark.parametrize("width, dtype", [(12288, BF16), (7000, BF16), (8192, F32), (5001, BF16)])
def test_norm_of_two_sizes_from_two_threads(width, dtype):
    """Two host threads in one instance of the kernel, one with a residual (more shared memory) and one without: neither
    takes the other's limit away between its setting and its launch.  The library is called directly, 20000 times from
    each thread; a limit of the call's own refused some 10 to 100 of them at 12288 columns."""
    lib = _layers._layers_lib()
    refused, outs, ins = [None, None], [None, None], [None, None]
    start = threading.Barrier(2)

    def work(i):
        g = gen(40 + i)
        x, r, w = randn(g, 1, width, dtype=dtype), randn(g, 1, width, dtype=dtype), randn(g, width, dtype=dtype)
        out, res = torch.empty_like(x), torch.empty_like(x)
        ins[i], outs[i] = (x, w, r if i else None), (out, res)
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        p = [ctypes.c_void_p(t.data_ptr()) for t in (x, r, w, out, res)]
        code = 1 if dtype == BF16 else 0
        args = (p[0], p[1] if i else None, None, p[2], 1e-6, 0.0, p[3], p[4] if i else None, None, 1, width, code,
                code, 0, ctypes.c_void_p(stream.cuda_stream))
        start.wait()
        refused[i] = sum(lib.gdn_rms_norm(*args) != 0 for _ in range(20000))
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert refused == [0, 0]
    for (x, w, r), (out, _) in zip(ins, outs):
        _, y = norm64(x, w, r, None, 1e-6, 0.0)
        within(out, y, (HALF[dtype] + 2.0 ** -17) * y.abs(), "out")


# ------------------------------------------------------------------ paged attention


def set_rows(c, b, k=None, v=None):
    """Sequence b's keys (values) [n, Hkv, D] into its list and its pages."""
    j = torch.arange(c.lens[b], device="cuda")
    rows = c.table[b].long()[j // c.page] * c.page + j % c.page
    for new, mine, cache in ((k, c.keys, c.k), (v, c.values, c.v)):
        if new is not None:
            mine[b] = new
            cache.view(-1, *cache.shape[2:])[rows] = new


@pytest.mark.parametrize("dtype, size", [(F16, 2000.0), (F16, 20000.0), (F16, 60000.0), (BF16, 1e8), (BF16, 1e15)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n, columns", [(1, None), (40, None), (3000, None), (3000, 100000)])
def test_attn_scores_of_extreme_size(dtype, size, D, n, columns):
    """Scores of up to some 10^31, of either sign.  Two keys (one, of a single key) share the largest score, every other
    lies below it by more than an exponential's range.  The two scores come of the same numbers by the same steps, so
    they are equal, their weights 1 and all others 0: out is the mean of the two values, off by its own rounding and one
    in fp32.  The magnitudes of a score add up to |lse|, and its D / 16 + 4 steps are good to 2^-22 each."""
    c = Paged([n, n], 1, D, 16, dtype, seed=int(size) % 97)
    top = sorted({min(7, n - 1), n * 5 // 6})
    q = torch.full((2, 3, D), size, device="cuda", dtype=dtype)
    for b, (high, low) in enumerate(((1.0, 0.0), (-0.5, -1.0))):
        k = torch.full((n, 1, D), low, device="cuda") * size
        k[top] = high * size
        set_rows(c, b, k=k.to(dtype))
    if columns:
        c = c.widened(columns)
    out, lse = gdn.paged_attn_fwd(q, c.k, c.v, c.table, c.seq_lens, output_lse=True)
    for b in range(2):
        o = c.values[b][top].double().mean(0).expand(3, D)
        _, l, _, _ = attn64(q[b], c.keys[b], c.values[b], D ** -0.5)
        within(out[b], o, (HALF[dtype] + 2.0 ** -24) * o.abs() + TINY[dtype], "out")
        within(lse[b], l, ((D / 16 + 4) * 2.0 ** -22 + 2.0 ** -20) * l.abs(), "lse")
