"""The layer operators on the GPU where two calls meet and where the arithmetic is at its limits: host threads that
call one operator at once, and inputs whose sizes lie far apart.  Formulas and tolerances are those of
test_gpu_layers.py; what a test adds to them stands in its docstring."""
from __future__ import annotations

import ctypes
import threading

import pytest
import torch

from gated_deltanet_linear_17_b200 import _layers
from test_gpu_layers import F32, BF16, gen, norm64, randn, within

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


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
