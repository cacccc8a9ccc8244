"""The layer operators on the GPU where two calls meet and where the arithmetic is at its limits: host threads that
call one operator at once, and inputs whose sizes lie far apart.  Formulas and tolerances are those of
test_gpu_layers.py; what a test adds to them stands in its docstring."""
from __future__ import annotations

import ctypes
import math
import threading

import pytest
import torch

import gated_deltanet_linear_17_b200 as gdn
from gated_deltanet_linear_17_b200 import _layers
from test_gpu_layers import BF16, F16, F32, HALF, TINY, Paged, attn64, gen, norm64, randn, rope64, within

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


@pytest.mark.parametrize("quant", ["row", "block"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("width", [128, 2048, 4096])
def test_norm_scales_are_rounded_once(width, dtype, quant):
    """Rows of one value in all places, weight and rstd 1: y is that value, and the scale is value / 448 rounded once.
    eps = 1 - value^2 makes rstd the root of 1 up to the rounding of the mean of equal squares, which a power of two
    as width leaves exact."""
    x = torch.tensor([0.0625, 0.125, 0.25, 0.375, 0.5, 0.625, 0.75, 0.875], device="cuda")
    for value in x.tolist():
        rows = torch.full((5, width), value, device="cuda", dtype=dtype)
        _, _, scales = gdn.rms_norm(rows, torch.ones(width, device="cuda", dtype=dtype), eps=1 - value * value, quant=quant)
        want = torch.tensor(value, dtype=torch.float64) / 448
        assert (scales == want.float().item()).all()


# ------------------------------------------------------------------ rope


@pytest.mark.parametrize("farthest", [50, 1 << 16, (1 << 31) - 1])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("mscale", [1.0, 1.3])
def test_rope_of_fp32_is_good_to_fp32(farthest, interleaved, mscale):
    """A factor is within 2^-24 of the exact one, and its product with mscale is rounded; the two products of an element
    are rounded once more each at most (relative: 2^-24 + 2^-24 + 2^-24 < 2^-22 of mscale (|a| + |b|)), and their sum.
    Frequencies of every size, among them some whose angles lie beside whole quarters of a turn; either sign of the
    position."""
    g = gen(farthest % 91)
    T, D = 3000, 128
    q, k = randn(g, T, 2, D, dtype=F32), randn(g, T, 1, D, dtype=F32)
    pos = torch.randint(-farthest, farthest, (T,), generator=g, device="cuda").to(torch.int32)
    f, _ = gdn.rope_inv_freq(D)
    f[::7] = math.pi / 2 ** torch.arange(10, device="cuda")
    f[3::11] = 9.7 * torch.rand(6, generator=g, device="cuda")
    got = gdn.rope_fwd(q, k, pos, f, interleaved=interleaved, mscale=mscale)
    for x, y in zip((q, k), got):
        want, size = rope64(x, pos, f, interleaved, mscale)
        within(y, want, 2.0 ** -22 * size + 2.0 ** -24 * want.abs(), "turned")


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


def shared(n, rows, D, dtype, seed, lens=None, columns=None):
    """`rows` sequences on the same pages, the first `lens[b]` keys of n each (all by default); values of one sign."""
    g = gen(seed)
    c = Paged([n], 1, D, 64, dtype, seed=seed, spare=0)
    set_rows(c, 0, v=(0.75 + 0.5 * torch.rand(n, 1, D, generator=g, device="cuda")).to(dtype))
    lens = [n] * rows if lens is None else lens
    table = c.table.expand(len(lens), -1).contiguous()
    if columns:
        wide = torch.full((len(lens), columns), -7, dtype=torch.int32, device="cuda")
        wide[:, :table.shape[1]] = table
        table = wide
    return c, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), randn(g, len(lens), 4, D, dtype=dtype)


def check_shared(c, table, lens, q, **kw):
    """All rows against 64 bits.  No more than 512 additions go to one accumulator, each cut off by up to 2^-23 of it: 2^-14
    more than check_attn allows."""
    dt, D = q.dtype, q.shape[2]
    out, lse = gdn.paged_attn_fwd(q, c.k, c.v, table, lens, output_lse=True, **kw)
    k, v = c.keys[0][:, 0].double(), c.values[0][:, 0].double()
    for b0 in range(0, q.shape[0], 50):
        qq, n = q[b0:b0 + 50].double(), lens[b0:b0 + 50]
        s = qq @ k.T * D ** -0.5
        s.masked_fill_(torch.arange(k.shape[0], device="cuda") >= n[:, None, None], -math.inf)
        e = (D / 16 + 4) * 2.0 ** -22 * (qq.abs() @ k.abs().T).amax(-1) * D ** -0.5
        l = torch.logsumexp(s, -1)
        p = torch.exp(s - l[..., None])
        o = p @ v
        tol = (2 * e[..., None] + 2.0 ** -13) * (p @ v.abs()) + HALF[dt] * o.abs() + TINY[dt]
        within(out[b0:b0 + 50], o, tol, f"out of rows {b0} on")
        within(lse[b0:b0 + 50], l, e + 2.0 ** -20 * (l.abs() + 1), "lse")
    return out, lse


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rows, hint", [(300, 0), (300, 1), (3, 1)])
def test_attn_sums_of_many_keys(D, dtype, rows, hint):
    """131072 keys a CTA and more, all values positive: what the tensor core cuts off of every addition adds up.  By the
    list, and by clusters whose hint is far too small."""
    c, table, lens, q = shared(131072 + 77, rows, D, dtype, D)
    a = check_shared(c, table, lens, q, max_seqlen=hint)
    again = gdn.paged_attn_fwd(q, c.k, c.v, table, lens, output_lse=True, max_seqlen=hint)
    assert torch.equal(a[0], again[0]) and torch.equal(a[1], again[1])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 12])
def test_attn_long_pieces_among_short_ones(D, group):
    """Lengths around whole pieces (8192 keys at D = 256, else 16384), several sequences a CTA: pieces that begin, end and
    lie within a CTA's part of the list, with sums carried on from piece to piece; queries of 1 and 12 heads."""
    some = [8192, 16383, 16385, 0, 16384, 1, 24640, 40000, 7000, 32769, 16320, 16448, 64, 49152, 0, 20001]
    lens = [some[(3 * i + i // 16) % 16] for i in range(500)]
    c, table, lens, _ = shared(50000, 0, D, BF16, D + 1, lens=lens)
    q = randn(gen(D), len(lens), group, D)
    keep = lens > 0
    out, lse = gdn.paged_attn_fwd(q, c.k, c.v, table, lens, output_lse=True)
    assert (out[~keep] == 0).all() and (lse[~keep] == -math.inf).all()
    check_shared(c, table[keep], lens[keep], q[keep])
    check_shared(c, table[keep], lens[keep], q[keep], max_seqlen=64)


@pytest.mark.parametrize("hint", [0, 1])
@pytest.mark.parametrize("D", [64, 256])
def test_attn_carried_sums_of_every_kind(D, hint):
    """Pieces without a weight (scores of -infinity), with all of it, with scores far below zero, and with a NaN or a bad
    page in one of them: of many rows on the same pages, so that a CTA has a sequence to itself."""
    n, copies = 40000, 60
    c = Paged([n] * 6, 1, D, 64, BF16, seed=3)
    q = 1 + 0.1 * randn(gen(4), 6, 2, D).abs()
    keys = [k.clone() for k in c.keys]
    keys[0][:18000] = -math.inf
    keys[1][8000:] = -math.inf
    keys[2][:] = -math.inf
    keys[3] = -200 - keys[3].abs()
    keys[5][20000, 0, 5] = math.nan
    for b, k in enumerate(keys):
        set_rows(c, b, k=k)
    c.table[4, 20000 // 64] = -1
    q, table, lens = q.repeat(copies, 1, 1), c.table.repeat(copies, 1), c.seq_lens.repeat(copies)
    out, lse = gdn.paged_attn_fwd(q, c.k, c.v, table, lens, output_lse=True, max_seqlen=hint)
    # where a sequence is cut differs from copy to copy, what comes out but in the last bits does not
    for b in range(6 * copies):
        if b % 6 not in (2, 4, 5):
            within(out[b], out[b % 6].double(), 2.0 ** -7 * out[b % 6].double().abs() + 2.0 ** -13, "a copy")
    assert (out[2::6] == 0).all() and (lse[2::6] == -math.inf).all()
    assert all(out[i::6].isnan().all() and lse[i::6].isnan().all() for i in (4, 5))
    for b, part in ((0, slice(18000, n)), (1, slice(0, 8000)), (3, slice(0, n))):
        o, l, av, e = attn64(q[b], c.keys[b][part], c.values[b][part], D ** -0.5)
        within(out[b], o, (2 * e[:, None] + 2.0 ** -13) * av + HALF[BF16] * o.abs(), f"out {b}")
        within(lse[b], l, e + 2.0 ** -20 * (l.abs() + 1), f"lse {b}")


@pytest.mark.parametrize("nats", [8, 12, 16, 18, 20])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D, n, group, columns", [(64, 16, 4, None), (128, 500, 1, None), (256, 700, 9, None),
                                                  (64, 3000, 9, 100000), (128, 3000, 4, 100000), (256, 3000, 1, 100000)])
def test_attn_keys_far_below_the_largest_score(nats, dtype, D, n, group, columns):
    """A key whose score lies `nats` above the others' and whose value is 0: the output consists of the others alone.
    Their weights are held to 2^-40 of the largest, each, in fp16; the rest of the tolerance is check_attn's."""
    g = gen(nats)
    c = Paged([n], 1, D, 16, dtype, seed=nats)
    q = randn(g, 1, 1, D, dtype=dtype).expand(1, group, D).contiguous()
    k, v = 0.05 * randn(g, n, 1, D, dtype=F32), 300 + 30 * randn(g, n, 1, D, dtype=F32)
    one = q[0, 0].float()
    k[n // 3] = one * (nats * D ** 0.5 / (one @ one))
    v[n // 3] = 0
    set_rows(c, 0, k=k.to(dtype), v=v.to(dtype))
    if columns:
        c = c.widened(columns)
    out, lse = gdn.paged_attn_fwd(q, c.k, c.v, c.table, c.seq_lens, output_lse=True)
    o, l, av, e = attn64(q[0], c.keys[0], c.values[0], D ** -0.5)
    held = 2.0 ** -40 * c.values[0][:, 0].double().abs().sum(0) if dtype == F16 else 0.0
    within(out[0], o, 2 * (e[:, None] + 2.0 ** -15) * av + HALF[dtype] * o.abs() + TINY[dtype] + held, "out")
    within(lse[0], l, e + 2.0 ** -20 * (l.abs() + 1), "lse")


@pytest.mark.parametrize("scale", [1e-50, 1e-46, 5e38, 1e300, 2.4e38])
def test_attn_refuses_scales_beyond_fp32(scale):
    """1e-50 is positive and finite, but 0 in fp32, which stands for the default."""
    c = Paged([30, 40], 2, 64, 16, BF16)
    with pytest.raises(ValueError, match="scale"):
        gdn.paged_attn_fwd(randn(gen(1), 2, 4, 64), c.k, c.v, c.table, c.seq_lens, scale=scale)


@pytest.mark.parametrize("scale", [1.5e-45, 1e-30, 2e38])
def test_attn_takes_scales_at_the_ends_of_fp32(scale):
    """The smallest: all scores 0, out the mean of the values.  The largest: the largest score takes all (they differ
    by far more than 2^-100 here)."""
    c = Paged([300], 1, 64, 16, BF16, seed=2)
    q = randn(gen(1), 1, 4, 64)
    out, lse = gdn.paged_attn_fwd(q, c.k, c.v, c.table, c.seq_lens, scale=scale, output_lse=True)
    s = torch.einsum("hd,nd->hn", q[0].double(), c.keys[0][:, 0].double())
    v = c.values[0][:, 0].double()
    want = v.mean(0).expand(4, 64) if scale < 1 else v[s.argmax(1)]
    within(out[0], want, HALF[BF16] * want.abs() + 2.0 ** -14 * v.abs().mean(0), "out")
    assert scale > 1 or (lse - math.log(300)).abs().max() < 2.0 ** -17


def test_sizes_beyond_32_bits_are_refused():
    """A width, head dimension or page count of 2^32 and something (8.6 GB of elements) is no smaller one."""
    n = (1 << 32) + 64
    x = torch.empty(n, device="cuda", dtype=BF16)
    few = torch.zeros(1, device="cuda", dtype=torch.int32)
    for call in (lambda: gdn.rms_norm(x, x), lambda: gdn.rms_norm(x, x, quant="block"),
                 lambda: gdn.rope_fwd(x.view(1, 1, n), x.view(1, 1, n), few, torch.ones(1, device="cuda")),
                 lambda: gdn.rope_fwd(x.view(1, n // 64, 64), x.view(1, n // 64, 64), few, torch.ones(1, device="cuda")),
                 lambda: gdn.paged_attn_fwd(x.view(1, 1, n), x.view(1, 1, 1, n), x.view(1, 1, 1, n), few.view(1, 1), few)):
        with pytest.raises((ValueError, RuntimeError)):
            call()


def test_calls_by_torch_s_public_functions(monkeypatch):
    """The device and the stream that a call runs on, where torch has no private functions for them."""
    g = gen(5)
    x, w = randn(g, 300, 256), randn(g, 256)
    want = gdn.rms_norm(x, w)[0]
    monkeypatch.setattr(_layers, "_current_device", torch.cuda.current_device)
    monkeypatch.setattr(_layers, "_current_stream", _layers._stream_handle)
    assert torch.equal(gdn.rms_norm(x, w)[0], want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert _layers._current_stream(0) == side.cuda_stream
        got = gdn.rms_norm(x, w)[0]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
