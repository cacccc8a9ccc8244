"""The layer operators on the GPU against their formulas in 64 bits: the norm, the rotary positions with
the write into a paged cache, the attention of one new token over it, and one decode step of all.

Tolerances, per element, from the arithmetic (u = 2^-24 is the fp32 unit roundoff):
  norm       y is a product of four fp32 factors.  The sum of squares of up to 32768 columns is 32
             sequential fused additions a lane at most and a tree of at most 20, all terms positive: 52 u, half
             of it in the root.  e^-g is 2^(-g log2 e): its argument is off by 2 u, relative, which is 2 |g| u of
             it, |g| < 8 in the tests, and the approximate exponential and reciprocal by 4 u each: 24 u.  With the
             products and the root: below 100 u < 2^-17, relative, plus the output's own rounding.  In 8 bits:
             half a step of e4m3, 2^-4 relative or 2^-10 below its normal range, in units of the scale.
  rope       the reduced angle is rounded to fp32 (|th| <= pi: 2^-23), the fast sine and cosine are within 2^-21.2
             (fp32 activations: 2^-24, both roundings in it), then two products and a sum: below
             2^-20 mscale (|a| + |b|), plus the output's rounding.
  attention  a score is a sum of D exact products accumulated in fp32 on the tensor core, in D / 16 steps
             whose inner additions may be cut off rather than rounded (2^-22 of the magnitudes each), scaled:
             e = (D / 16 + 4) 2^-22 scale sum |q k|.  A probability is then off by e + 2^-21 (exp2) + 2^-16
             (its two 16-bit parts) + as much of the maximum's, relative, and likewise the sum: out is
             within 2 (e + 2^-15) sum p |v| of the exact one, lse within e + 2^-20 |lse| + 2^-20.
"""
from __future__ import annotations

import math

import pytest
import torch

import gated_deltanet_linear_17_b200 as gdn

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}  # half a step of fp16's subnormals
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAN = float("nan")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=BF16):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def within(got, want, tol, what):
    assert got.shape == want.shape
    d = (got.double() - want).abs()
    assert torch.isfinite(got.double()).all(), f"{what}: not finite"
    over = d - tol
    i = int(over.argmax())
    assert over.max() <= 0, f"{what}: off by {d.flatten()[i]:.3e} where {tol.flatten()[i]:.3e} is allowed"


def guarded(shape, dtype, pad=64):
    """An uninitialised-looking tensor inside a larger one of a known pattern, and a check that nothing around it
    was written."""
    n = math.prod(shape)
    whole = torch.full((n + 2 * pad,), 72.0, device="cuda").to(dtype)
    whole[pad:pad + n] = NAN
    inner = whole[pad:pad + n].view(shape)

    def check():
        f = whole.float()
        assert (f[:pad] == 72).all() and (f[pad + n:] == 72).all(), "written outside the tensor"

    return inner, check


# ------------------------------------------------------------------ norm


def norm64(x, w, residual, gate, eps, offset):
    z = x.double() if residual is None else x.double() + residual.double()
    y = z / torch.sqrt((z * z).mean(-1, keepdim=True) + eps) * (w.double() + offset)
    return z, y if gate is None else y * gate.double() * torch.sigmoid(gate.double())


def check_norm(x, w, residual=None, gate=None, quant=None, eps=1e-6, offset=0.0):
    shape, width, dt = x.shape, x.shape[-1], x.dtype
    z, y = norm64(x, w, residual, gate, eps, offset)
    out, out_check = guarded(shape, dt if quant is None else torch.float8_e4m3fn)
    kw = dict(residual=residual, gate=gate, eps=eps, weight_offset=offset, quant=quant, out=out)
    if residual is not None:
        kw["residual_out"], res_check = guarded(shape, dt)
    if quant is not None:
        sshape = shape[:-1] if quant == "row" else (*shape[:-1], -(-width // 128))
        kw["scales"], sc_check = guarded(sshape, F32)
    got, res, scales = gdn.rms_norm(x, w, **kw)
    torch.cuda.synchronize()
    assert got is out
    out_check()
    if residual is None:
        assert res is None
    else:
        res_check()
        within(res, z, (HALF[dt] + 2.0 ** -24) * z.abs() + TINY[dt], "residual")
    rel = 2.0 ** -17
    if quant is None:
        assert scales is None
        within(got, y, (HALF[dt] + rel) * y.abs() + TINY[dt], "out")
        return
    sc_check()
    group = width if quant == "row" else 128
    pad = -width % group
    yp = torch.nn.functional.pad(y, (0, pad)).unflatten(-1, (-1, group))
    want = (yp.abs().amax(-1) / 448).clamp(min=2.0 ** -126)
    sc = scales.double() if quant == "block" else scales.double().unsqueeze(-1)
    within(sc, want, rel * want, "scales")
    step = want.unsqueeze(-1).expand_as(yp).flatten(-2)[..., :width]
    v = y / step
    tol = torch.maximum(2.0 ** -4 * v.abs(), torch.full_like(v, 2.0 ** -10)) + 2 * rel * v.abs()
    within(got.float(), v, tol, "out / scale")


WIDTHS = [1, 2, 7, 8, 64, 72, 120, 127, 128, 129, 136, 256, 257, 320, 1000, 1024, 1032, 1537, 2048, 4096, 5001, 8192,
          8193, 8200, 10240, 11111, 16384, 32759, 32760, 32768]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("quant", [None, "row", "block"])
def test_norm_widths(width, quant):
    g = gen(width)
    for i, dt in enumerate((BF16, F16, F32)):
        rows = 5 if i else 19
        x, r, z = (randn(g, rows, width, dtype=dt) for _ in range(3))
        w = (1 + 0.1 * randn(g, width, dtype=F32)).to(dt)
        check_norm(x, w, residual=r if i != 1 else None, gate=z if i != 0 else None, quant=quant)


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 4097])
@pytest.mark.parametrize("width", [128, 200, 131])
def test_norm_rows(rows, width):
    g = gen(rows)
    x, r, z = (randn(g, rows, width) for _ in range(3))
    w = randn(g, width, dtype=F32)                                # fp32 weights beside bf16 rows
    for quant in (None, "row", "block"):
        check_norm(x, w, residual=r, gate=z, quant=quant, offset=1.0, eps=1e-5)


def test_norm_of_heads():
    g = gen(3)
    x, z = randn(g, 37, 8, 128), randn(g, 37, 8, 128)
    check_norm(x, randn(g, 128), gate=z, quant="row")
    check_norm(x, randn(g, 128), gate=z)


def test_norm_zero_rows_and_empty():
    x = torch.zeros(6, 256, device="cuda", dtype=BF16)
    w = torch.ones(256, device="cuda", dtype=BF16)
    for quant in (None, "row", "block"):
        out, res, scales = gdn.rms_norm(x, w, residual=x, quant=quant)
        assert (out.float() == 0).all() and (res == 0).all()
        if scales is not None:
            assert (scales == 2.0 ** -126).all()
    out, res, scales = gdn.rms_norm(x[:0], w, residual=x[:0], quant="block")
    assert out.shape == (0, 256) and res.shape == (0, 256) and scales.shape == (0, 2)


@pytest.mark.parametrize("width", [128, 131, 2048])
@pytest.mark.parametrize("quant", [None, "row", "block"])
def test_norm_keeps_rows_apart(width, quant):
    """A row of NaN or infinities leaves its neighbours' bits as they were."""
    g = gen(5)
    x, z = randn(g, 9, width), randn(g, 9, width)
    w = randn(g, width)
    clean = gdn.rms_norm(x, w, gate=z, quant=quant)
    x2 = x.clone()
    x2[3, width // 2] = NAN
    x2[5, 0] = float("inf")
    dirty = gdn.rms_norm(x2, w, gate=z, quant=quant)
    keep = [i for i in range(9) if i not in (3, 5)]
    assert torch.equal(dirty[0].float()[keep], clean[0].float()[keep])
    assert dirty[0].float()[3].isnan().all() and dirty[0].float()[5, 0].isnan()
    if quant == "row":
        assert dirty[2][3].isnan()
    # a NaN of the gate stays in its element (and, in 8 bits, in its scale's group)
    z2 = z.clone()
    z2[4, 1] = NAN
    one = gdn.rms_norm(x, w, gate=z2, quant=quant)
    assert one[0].float()[4, 1].isnan()
    if quant is None:
        assert one[0].float()[4].isnan().sum() == 1
    elif quant == "block":
        assert one[2][4, 0].isnan() and not one[2][4, 1:].isnan().any()


def test_norm_in_place():
    g = gen(6)
    for width in (128, 131, 4096):
        x, r, w = randn(g, 33, width), randn(g, 33, width), randn(g, width)
        want = gdn.rms_norm(x, w, residual=r)
        xi, ri = x.clone(), r.clone()
        got = gdn.rms_norm(xi, w, residual=ri, out=xi, residual_out=ri)
        assert got[0] is xi and got[1] is ri
        assert torch.equal(xi, want[0]) and torch.equal(ri, want[1])


def test_norm_refusals():
    g = gen(7)
    x, w = randn(g, 4, 64), randn(g, 64)
    for bad in (dict(weight=w[:32]), dict(weight=w.half()), dict(residual=x[:2]), dict(residual=x.half()),
                dict(gate=x.t()), dict(quant="int8"), dict(residual_out=x), dict(scales=x),
                dict(out=x, quant="row")):
        with pytest.raises((ValueError, RuntimeError)):
            gdn.rms_norm(x, **{"weight": w, **bad})
    with pytest.raises(ValueError):
        gdn.rms_norm(x.t(), w[:4])                                # not contiguous
    with pytest.raises(ValueError):
        gdn.rms_norm(x.flatten()[1:129].view(2, 64), w)           # not aligned
    with pytest.raises(RuntimeError):
        gdn.rms_norm(x.double(), w.double())
    with pytest.raises(ValueError):
        gdn.rms_norm(randn(g, 1, 32776), randn(g, 32776))


def test_norm_many_rows():
    """Element offsets beyond 2^31: the last rows of a matrix of 2^31 + elements."""
    width, rows = 128, (1 << 24) + 5
    x = torch.empty(rows, width, device="cuda", dtype=BF16)
    x[-7:] = randn(gen(8), 7, width)
    x[:3] = randn(gen(9), 3, width)
    x[3:-7] = 1.0
    w = randn(gen(10), width)
    out, _, sc = gdn.rms_norm(x, w, quant="row")
    few, _, fs = gdn.rms_norm(torch.cat([x[:3], x[-7:]]), w, quant="row")
    assert torch.equal(out[-7:].float(), few[3:].float()) and torch.equal(sc[-7:], fs[3:])
    assert torch.equal(out[:3].float(), few[:3].float())


# ------------------------------------------------------------------ rope


def rope64(x, positions, f, interleaved, mscale):
    n = f.numel()
    a = positions.double()[:, None, None] * f.double()
    c, s = a.cos() * mscale, a.sin() * mscale
    y = x.double().clone()
    i = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    p, q = x[..., i[0]].double(), x[..., i[1]].double()
    y[..., i[0]], y[..., i[1]] = p * c - q * s, q * c + p * s
    size = torch.zeros_like(y)
    size[..., i[0]] = size[..., i[1]] = mscale * (p.abs() + q.abs())
    return y, size


def check_rope(T, Hq, Hkv, D, rotary, interleaved, dt, farthest, page=None, mscale=1.0, seed=0, in_place=False):
    g = gen(seed)
    q, k, v = randn(g, T, Hq, D, dtype=dt), randn(g, T, Hkv, D, dtype=dt), randn(g, T, Hkv, D, dtype=dt)
    pos = torch.randint(0, farthest, (T,), generator=g, device="cuda").to(torch.int32)
    pos[:1] = farthest - 1
    f, _ = gdn.rope_inv_freq(rotary) if rotary else (torch.empty(0, device="cuda"), 1.0)
    (wq, sq), (wk, sk) = rope64(q, pos, f, interleaved, mscale), rope64(k, pos, f, interleaved, mscale)
    tq, tk = (2.0 ** -20 * s + (HALF[dt] + 2.0 ** -20) * w.abs() * (s > 0) + TINY[dt] for w, s in ((wq, sq), (wk, sk)))
    q0, k0 = q.clone(), k.clone()
    q_out, qc = guarded((T, Hq, D), dt)
    k_out, kc = guarded((T, Hkv, D), dt)
    if in_place:
        q_out, k_out = q, k
    kw = dict(interleaved=interleaved, mscale=mscale, q_out=q_out, k_out=k_out)
    if page:
        P = -(-T // page) + 2
        caches = [guarded((P, page, Hkv, D), dt) for _ in range(2)]
        for c, _ in caches:
            c.fill_(5.0)
        slots = torch.randperm(P * page, generator=g, device="cuda")[:T].to(torch.int32)
        padding = torch.arange(T, device="cuda") % 5 == 3
        given = slots.clone()
        bad = torch.tensor([-1, P * page, -(1 << 31), (1 << 31) - 1], device="cuda", dtype=torch.int32)
        given[padding] = bad[torch.arange(int(padding.sum()), device="cuda") % 4]
        kw.update(v=v, k_cache=caches[0][0], v_cache=caches[1][0], slots=given)
    got_q, got_k = gdn.rope_fwd(q, k, pos, f, **kw)
    torch.cuda.synchronize()
    assert got_q is q_out and got_k is k_out
    within(q_out, wq, tq, "q")
    within(k_out, wk, tk, "k")
    if not in_place:
        qc(), kc()
        assert torch.equal(q, q0) and torch.equal(k, k0)
    if page:
        for (c, check), new in zip(caches, (k_out, v)):
            check()
            want = torch.full((P * page, Hkv, D), 5.0, device="cuda", dtype=dt)
            want[slots[~padding].long()] = new[~padding]
            assert torch.equal(c.view(P * page, Hkv, D), want)


@pytest.mark.parametrize("D, rotary", [(8, 2), (64, 64), (80, 20), (80, 80), (96, 24), (128, 32), (128, 46), (192, 2),
                                       (256, 64), (256, 256), (64, 0), (248, 240), (128, 16), (72, 70)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_heads(D, rotary, interleaved):
    for i, dt in enumerate((BF16, F16, F32)):
        check_rope(13, 6, 3, D, rotary, interleaved, dt, 5000, page=(4, None, 1)[i], mscale=1.0 if i else 1.25,
                   seed=D + i)


@pytest.mark.parametrize("T", [1, 2, 31, 257, 1500])
@pytest.mark.parametrize("Hq, Hkv", [(1, 1), (16, 2), (7, 7), (5, 3)])
def test_rope_tokens(T, Hq, Hkv):
    check_rope(T, Hq, Hkv, 128, 64, False, BF16, 1 << 20, page=16, seed=T)
    check_rope(T, Hq, Hkv, 64, 36, True, F16, 1 << 20, page=17, seed=T)
    check_rope(T, Hq, Hkv, 64, 36, False, F16, 1 << 20, seed=T)


@pytest.mark.parametrize("farthest", [1, 1 << 16, 1 << 24, (1 << 31) - 1])
def test_rope_far_positions(farthest):
    """The tolerance does not grow with the position."""
    check_rope(64, 2, 1, 128, 128, False, F32, farthest, seed=1)
    check_rope(64, 2, 1, 128, 128, True, F32, farthest, seed=2)


@pytest.mark.parametrize("rotary", [0, 20, 64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_in_place(rotary, interleaved):
    check_rope(99, 4, 2, 128, rotary, interleaved, BF16, 3000, page=8, in_place=True)


def test_rope_negative_positions_turn_back():
    """The turn by -p undoes the turn by p: a rotation's gradient is the call at the negated positions."""
    g = gen(1)
    q, k = randn(g, 50, 4, 64, dtype=F32), randn(g, 50, 2, 64, dtype=F32)
    pos = torch.randint(0, 100000, (50,), generator=g, device="cuda").to(torch.int32)
    f, _ = gdn.rope_inv_freq(64)
    a, b = gdn.rope_fwd(q, k, pos, f)
    c, d = gdn.rope_fwd(a, b, -pos, f)
    for got, want in ((c, q), (d, k)):
        pair = want.double().abs().unflatten(-1, (2, 32)).sum(-2, keepdim=True).expand(-1, -1, 2, -1).flatten(-2)
        within(got, want.double(), 2.0 ** -18 * pair, "back")


def test_rope_empty_and_refusals():
    g = gen(2)
    q, k, v = randn(g, 4, 2, 64), randn(g, 4, 1, 64), randn(g, 4, 1, 64)
    pos = torch.arange(4, device="cuda", dtype=torch.int32)
    f, _ = gdn.rope_inv_freq(64)
    a, b = gdn.rope_fwd(q[:0], k[:0], pos[:0], f)
    assert a.shape == (0, 2, 64) and b.shape == (0, 1, 64)
    cache = torch.zeros(2, 4, 1, 64, device="cuda", dtype=BF16)
    full = dict(v=v, k_cache=cache, v_cache=cache.clone(), slots=pos)
    out, none = gdn.rope_fwd(q, k, pos, f, **full)
    assert none is None and torch.equal(full["v_cache"].view(8, 1, 64)[:4], v)
    for bad in (dict(v=None), dict(slots=None), dict(k_cache=None), dict(slots=pos.long()), dict(v_cache=cache),
                dict(k_cache=cache.half()), dict(v=v[:2]), dict(q_out=k)):
        with pytest.raises((ValueError, RuntimeError)):
            gdn.rope_fwd(q, k, pos, f, **{**full, **bad})
    for args in ((q, k, pos.long(), f), (q, k, pos, f.double()), (q, k.half(), pos, f), (q, k[:2], pos, f),
                 (q.transpose(0, 1), k, pos, f), (q, k, pos, torch.cat([f, f])), (q[..., :60], k[..., :60], pos, f[:8])):
        with pytest.raises((ValueError, RuntimeError)):
            gdn.rope_fwd(*args)


# ------------------------------------------------------------------ paged attention


class Paged:
    """A paged cache of sequences of given lengths: pages in random order, NaN in every place behind a
    sequence's last key and on every spare page, and a table that is garbage behind the last page."""

    def __init__(self, lens, Hkv, D, page, dtype, seed=0, spare=3, columns=None):
        g = gen(seed)
        self.lens, self.page = lens, page
        need = [-(-n // page) for n in lens]
        self.max_pages = max(need + [0]) if columns is None else columns
        P = sum(need) + spare
        self.k = torch.full((P, page, Hkv, D), NAN, device="cuda", dtype=dtype)
        self.v = torch.full((P, page, Hkv, D), NAN, device="cuda", dtype=dtype)
        perm = torch.randperm(P, generator=g, device="cuda")
        garbage = torch.tensor([-1, P, (1 << 31) - 1, -(1 << 31)], dtype=torch.int64)
        table = garbage[torch.arange(len(lens) * self.max_pages) % 4].view(len(lens), self.max_pages)
        self.keys, self.values, at = [], [], 0
        for b, n in enumerate(lens):
            pages = perm[at:at + need[b]]
            at += need[b]
            table[b, :need[b]] = pages.cpu()
            kk, vv = randn(g, n, Hkv, D, dtype=dtype), randn(g, n, Hkv, D, dtype=dtype)
            rows = pages[torch.arange(n, device="cuda") // page] * page + torch.arange(n, device="cuda") % page
            self.k.view(-1, Hkv, D)[rows] = kk
            self.v.view(-1, Hkv, D)[rows] = vv
            self.keys.append(kk)
            self.values.append(vv)
        self.table = table.to(torch.int32).cuda()
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")


    def widened(self, capacity):
        """The same sequences in a table with room for `capacity` keys each: without a hint the work is then cut as for
        sequences of that length."""
        wide = Paged.__new__(Paged)
        wide.__dict__.update(self.__dict__)
        wide.max_pages = -(-capacity // self.page)
        wide.table = torch.full((len(self.lens), wide.max_pages), -7, dtype=torch.int32, device="cuda")
        wide.table[:, :self.max_pages] = self.table
        return wide


def attn64(q, keys, values, scale):
    """(out, lse, the tolerance's sum p |v| and e) of one sequence, in 64 bits."""
    Hq, D = q.shape
    n, Hkv, _ = keys.shape
    G = Hq // Hkv
    k, v = (t.double().repeat_interleave(G, dim=1) for t in (keys, values))
    s = torch.einsum("hd,nhd->hn", q.double(), k) * scale
    size = torch.einsum("hd,nhd->hn", q.double().abs(), k.abs()) * abs(scale)
    if n == 0:
        z = torch.zeros(Hq, D, dtype=torch.float64, device="cuda")
        return z, torch.full((Hq,), -math.inf, dtype=torch.float64, device="cuda"), z, z[:, 0]
    p = torch.softmax(s, dim=1)
    e = (D / 16 + 4) * 2.0 ** -22 * size.amax(1)
    return torch.einsum("hn,nhd->hd", p, v), torch.logsumexp(s, 1), torch.einsum("hn,nhd->hd", p, v.abs()), e


def check_attn(q, c, scale=None, skip=(), **kw):
    B, Hq, D = q.shape
    out, oc = guarded((B, Hq, D), q.dtype)
    lse, lc = guarded((B, Hq), F32)
    got = gdn.paged_attn_fwd(q, c.k, c.v, c.table, c.seq_lens, scale=scale, out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    assert got[0] is out and got[1] is lse
    oc(), lc()
    sc = scale if scale is not None else D ** -0.5
    for b in range(B):
        if b in skip:
            assert out[b].isnan().all() and lse[b].isnan().all()
            continue
        o, l, av, e = attn64(q[b], c.keys[b], c.values[b], sc)
        if c.lens[b] == 0:
            assert (out[b] == 0).all() and (lse[b] == -math.inf).all()
            continue
        tol = 2 * (e[:, None] + 2.0 ** -15) * av + HALF[q.dtype] * o.abs() + TINY[q.dtype]
        within(out[b], o, tol, f"out of sequence {b} ({c.lens[b]} keys)")
        within(lse[b], l, e + 2.0 ** -20 * (l.abs() + 1), f"lse of sequence {b}")
    return out, lse


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("page", [1, 16, 17, 64])
def test_attn_lengths(D, dtype, page):
    lens = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 255, 256, 257, 300, 511, 513, 777, 1025]
    c = Paged(lens, 2, D, page, dtype, seed=page)
    q = randn(gen(1), len(lens), 6, D, dtype=dtype)
    a = check_attn(q, c)
    # the hint changes how the work is split, not what comes out
    for hint in (1, 64, 1025, 1 << 20):
        check_attn(q, c, max_seqlen=hint)
    again = gdn.paged_attn_fwd(q, c.k, c.v, c.table, c.seq_lens, output_lse=True)
    assert torch.equal(a[0], again[0]) and torch.equal(a[1], again[1])   # run to run, bit for bit
    wide = c.widened(100000)
    assert gdn.paged_attn_workspace_bytes(len(lens), 6, 2, D, page, wide.max_pages) > 0
    a = check_attn(q, wide)                                               # cut by the list
    again = gdn.paged_attn_fwd(q, wide.k, wide.v, wide.table, wide.seq_lens, output_lse=True)
    assert torch.equal(a[0], again[0]) and torch.equal(a[1], again[1])


@pytest.mark.parametrize("Hkv, G", [(1, 1), (3, 2), (2, 7), (1, 8), (2, 9), (1, 16), (1, 17), (2, 24), (1, 40), (12, 1)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attn_heads(Hkv, G, D):
    lens = [700, 3, 0, 1290]
    c = Paged(lens, Hkv, D, 16, BF16, seed=G)
    q = randn(gen(2), len(lens), Hkv * G, D)
    check_attn(q, c)
    check_attn(q, c.widened(100000))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attn_many_short_sequences(D):
    """More pairs than CTAs, several of them one after the other in a CTA, empty ones among them."""
    lens = [(7 * i * i + 3 * i) % 150 if i % 5 else 0 for i in range(260)]
    c = Paged(lens, 3, D, 16, F16, seed=31)
    q = randn(gen(31), len(lens), 6, D, dtype=F16)
    check_attn(q, c)
    check_attn(q, c.widened(20000))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attn_long(D):
    """Long sequences among short ones, split over many CTAs; one head group alone."""
    lens = [40003, 5, 0, 9999]
    c = Paged(lens, 1, D, 32, BF16, seed=4)
    check_attn(randn(gen(3), len(lens), 4, D), c, max_seqlen=40003)
    check_attn(randn(gen(3), len(lens), 4, D), c, max_seqlen=100)
    one = Paged([70001], 1, D, 16, F16, seed=5)
    check_attn(randn(gen(4), 1, 2, D, dtype=F16), one)


def test_attn_wide_table():
    """A table of many more pages than any sequence has."""
    c = Paged([100, 33], 2, 128, 16, BF16, columns=5000)
    check_attn(randn(gen(5), 2, 8, 128), c)
    check_attn(randn(gen(5), 2, 8, 128), c, max_seqlen=100)


def test_attn_scores_of_every_size():
    """Scores up to the hundreds, one key that takes all the weight, equal scores, and other scales."""
    c = Paged([500, 64, 1], 1, 64, 16, F16, seed=6)
    q = randn(gen(6), 3, 4, 64, dtype=F16)
    check_attn(q, c, scale=4.0)
    check_attn(q, c, scale=0.001)
    check_attn(q * 0, c)                                          # every score 0: the mean of the values
    lens = c.lens
    c.k[c.table[0, 7].item(), 3] = 3 * q[0, 0]                     # one key along the query
    c.keys[0][7 * 16 + 3] = 3 * q[0, 0]
    assert lens[0] == 500
    check_attn(q, c, scale=2.0)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attn_scores_far_below_zero(D):
    """Scores of some -1000 for every key: what stands for the maximum of a part without keys must not be above them."""
    lens = [1, 70, 0, 300, 129, 64, 513, 2000, 5]
    c = Paged(lens, 1, D, 16, BF16, seed=21)
    q = 1 + 0.1 * randn(gen(21), len(lens), 3, D)
    for t in [c.k] + c.keys:
        t.copy_(-t.abs() - 2)
    for hint in (0, 2000, 64, 1 << 20):
        check_attn(q, c, scale=500.0 / D, max_seqlen=hint)
    check_attn(q, c.widened(100000), scale=500.0 / D)


def test_attn_infinite_scores():
    """Keys whose score is -infinity weigh nothing; a row of nothing else is a zero row, as a row without keys."""
    c = Paged([40, 40], 1, 64, 16, BF16, seed=7)
    q = randn(gen(7), 2, 2, 64).abs() + 0.5
    for b in range(2):
        for j in range(40):
            if b == 1 or j % 3 == 0:
                c.keys[b][j] = -math.inf
                c.k[c.table[b, j // 16].item(), j % 16] = -math.inf
    out, lse = gdn.paged_attn_fwd(q, c.k, c.v, c.table, c.seq_lens, output_lse=True)
    left = [j for j in range(40) if j % 3]
    o, l, av, e = attn64(q[0], c.keys[0][left], c.values[0][left], 0.125)
    within(out[0], o, 2 * (e[:, None] + 2.0 ** -15) * av + HALF[BF16] * o.abs(), "out")
    within(lse[0], l, e + 2.0 ** -20 * (l.abs() + 1), "lse")
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()


def test_attn_bad_rows_are_refused_alone():
    """A page outside the cache, a length beyond the table and a negative one: NaN for that sequence, nothing read out
    of bounds, the other sequences as ever."""
    lens = [200, 1000, 64, 64, 900, 30]
    c = Paged(lens, 2, 128, 16, BF16, seed=8)
    P = c.k.shape[0]
    c.table[0, 3] = P
    c.table[1, 60] = -1
    c.table[4, 0] = (1 << 31) - 1
    c.seq_lens[2] = c.max_pages * 16 + 1
    c.seq_lens[3] = -5
    q = randn(gen(8), len(lens), 8, 128)
    check_attn(q, c, skip=(0, 1, 2, 3, 4))
    check_attn(q, c, skip=(0, 1, 2, 3, 4), max_seqlen=64)
    wide = c.widened(100000)
    wide.seq_lens[2] = wide.max_pages * 16 + 1
    check_attn(q, wide, skip=(0, 1, 2, 3, 4))


def test_attn_no_pages():
    q = randn(gen(9), 3, 4, 64)
    empty = torch.empty(0, 16, 2, 64, device="cuda", dtype=BF16)
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    for table in (torch.empty(3, 0, dtype=torch.int32, device="cuda"),
                  torch.full((3, 7), -1, dtype=torch.int32, device="cuda")):
        out, lse = gdn.paged_attn_fwd(q, empty, empty, table, lens, output_lse=True)
        assert (out == 0).all() and (lse == -math.inf).all()
    out, lse = gdn.paged_attn_fwd(q[:0], empty, empty, table[:0], lens[:0])
    assert out.shape == (0, 4, 64) and lse is None


def test_attn_shared_pages_and_several_new_tokens():
    """Sequences that share pages (a common prefix), and three new tokens of one sequence as three rows."""
    c = Paged([333], 2, 128, 16, BF16, seed=10)
    c.table = c.table.expand(4, -1).contiguous()
    c.lens = [331, 332, 333, 160]
    c.seq_lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    c.keys, c.values = ([t[0][:n] for n in c.lens] for t in (c.keys, c.values))
    check_attn(randn(gen(10), 4, 8, 128), c)


def test_attn_offsets_beyond_32_bits():
    """A cache of more than 2^31 elements (4 GB of keys): pages at its end."""
    Hkv, D, page = 8, 256, 64
    P = (1 << 31) // (page * Hkv * D) + 40
    k = torch.zeros(P, page, Hkv, D, device="cuda", dtype=BF16)
    v = torch.zeros(P, page, Hkv, D, device="cuda", dtype=BF16)
    lens, g = [130, 64], gen(11)
    table = torch.tensor([[P - 1, 5, P - 30], [P - 2, -1, -1]], dtype=torch.int32, device="cuda")
    c = Paged.__new__(Paged)
    c.k, c.v, c.table, c.lens, c.max_pages, c.page = k, v, table, lens, 3, page
    c.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    c.keys, c.values = [], []
    for b, n in enumerate(lens):
        kk, vv = randn(g, n, Hkv, D), randn(g, n, Hkv, D)
        for i in range(-(-n // page)):
            m = min(page, n - i * page)
            k[table[b, i].item(), :m] = kk[i * page:i * page + m]
            v[table[b, i].item(), :m] = vv[i * page:i * page + m]
        c.keys.append(kk)
        c.values.append(vv)
    check_attn(randn(g, 2, 16, D), c)
    # the same rows written by rope_fwd
    n = lens[0]
    slots = (table[0, torch.arange(n, device="cuda") // page].long() * page + torch.arange(n, device="cuda") % page)
    f, _ = gdn.rope_inv_freq(64)
    gdn.rope_fwd(randn(g, n, 16, D), c.keys[0], torch.zeros(n, dtype=torch.int32, device="cuda"), f, v=c.values[0] * 2,
                 k_cache=k, v_cache=v, slots=slots.to(torch.int32))
    c.values[0] = c.values[0] * 2
    check_attn(randn(g, 2, 16, D), c)


def test_attn_refusals():
    c = Paged([30, 40], 2, 64, 16, BF16)
    q = randn(gen(12), 2, 4, 64)
    good = dict(q=q, k_cache=c.k, v_cache=c.v, block_table=c.table, seq_lens=c.seq_lens)
    long = torch.zeros(2, 4096, dtype=torch.int32, device="cuda")
    for bad in (dict(q=q.half()), dict(q=q.float()), dict(q=q[:, :3]), dict(v_cache=c.v[1:]), dict(k_cache=c.k.half()),
                dict(block_table=c.table.long()), dict(block_table=c.table[:1]), dict(seq_lens=c.seq_lens.long()),
                dict(seq_lens=c.seq_lens[:1]), dict(q=randn(gen(1), 2, 4, 80)), dict(max_seqlen=-1),
                dict(k_cache=c.k.transpose(1, 2), v_cache=c.v.transpose(1, 2)), dict(out=q),
                dict(lse=torch.zeros(2, 4, device="cuda", dtype=BF16)),
                dict(block_table=long, workspace=torch.zeros(64, device="cuda"))):
        with pytest.raises((ValueError, RuntimeError)):
            gdn.paged_attn_fwd(**{**good, **bad})


# ------------------------------------------------------------------ together


def decode_layer(x, residual, w, cache, table, pos, lens, slots, f, proj, hint, workspace=None):
    """One attention layer's decode step: norm, projections, rotary positions and cache write, attention, projection."""
    B = x.shape[0]
    h, residual, _ = gdn.rms_norm(x, w, residual=residual)
    q, k, v = (torch.matmul(h, m).view(B, -1, 128).contiguous() for m in proj[:3])
    q, _ = gdn.rope_fwd(q, k, pos, f, v=v, k_cache=cache[0], v_cache=cache[1], slots=slots)
    o, _ = gdn.paged_attn_fwd(q, cache[0], cache[1], table, lens, max_seqlen=hint, workspace=workspace)
    return torch.matmul(o.view(B, -1), proj[3]), residual, (q, k, v, o)


def test_decode_steps_of_a_hybrid_model():
    """A delta-rule layer (recurrent_fwd and its gated norm) and an attention layer over growing caches, several
    steps, each attention output against 64 bits on the keys and values of all steps so far."""
    g = gen(13)
    B, width, Hq, Hkv, page, steps = 3, 256, 4, 2, 4, 11
    proj = [randn(g, width, n * 128) * 0.06 for n in (Hq, Hkv, Hkv)] + [randn(g, Hq * 128, width) * 0.04]
    w = (1 + 0.1 * randn(g, width, dtype=F32)).to(BF16)
    wn = randn(g, 128)
    cache = [torch.full((16, page, Hkv, 128), NAN, device="cuda", dtype=BF16) for _ in range(2)]
    table = torch.randperm(16, generator=g, device="cuda")[:12].view(B, 4)[:, :3].contiguous().to(torch.int32)
    pool = torch.zeros(B, 2, 128, 128, device="cuda")
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    own = torch.arange(B, dtype=torch.int32, device="cuda")
    f, _ = gdn.rope_inv_freq(32)
    x, residual = randn(g, B, width), randn(g, B, width)
    keys, values = [], []
    for t in range(steps):
        pos = torch.full((B,), t, dtype=torch.int32, device="cuda")
        slots = table[:, t // page] * page + t % page
        x, residual, (q, k, v, o) = decode_layer(x, residual, w, cache, table, pos, pos + 1, slots, f, proj, 12)
        rk, _ = rope64(k, pos, f, False, 1.0)
        keys.append(rk.to(BF16))
        values.append(v)
        kk, vv = torch.stack(keys, 1), torch.stack(values, 1)
        got = cache[0][table[:, :t // page + 1].long()].flatten(1, 2)[:, :t + 1]
        assert (got.float() - kk.float()).abs().max() <= 2.0 ** -7 * kk.float().abs().max()  # a rounding of bf16
        assert torch.equal(cache[1][table[:, :t // page + 1].long()].flatten(1, 2)[:, :t + 1], vv)
        for b in range(B):
            want, _, av, e = attn64(q[b], got[b], vv[b], 128 ** -0.5)
            within(o[b], want, 2 * (e[:, None] + 2.0 ** -15) * av + HALF[BF16] * want.abs(), "attention")
        # the delta-rule layer of the same step, and its gated norm in 8 bits
        qd, kd, vd = (randn(g, B, 2, 128) for _ in range(3))
        od = gdn.recurrent_fwd(qd, kd, vd, -torch.rand(B, 2, generator=g, device="cuda"),
                               torch.rand(B, 2, generator=g, device="cuda").to(BF16), cu, pool, own, max_seqlen=1)
        check_norm(od, wn, gate=randn(g, B, 2, 128), quant="row")
    assert torch.isfinite(x.float()).all()


def test_prefill_output_norm():
    """chunk_fwd's output through the gated norm, 8 bits by head: the same values as a row of heads in blocks."""
    g = gen(14)
    T, Nv = 300, 4
    q, k, v, z = randn(g, T, 2, 128), randn(g, T, 2, 128), randn(g, T, Nv, 128), randn(g, T, Nv, 128)
    out, _ = gdn.chunk_fwd(q, k, v, -torch.rand(T, Nv, generator=g, device="cuda"),
                           torch.rand(T, Nv, generator=g, device="cuda").to(BF16),
                           torch.tensor([0, 100, T], dtype=torch.int32, device="cuda"))
    check_norm(out, randn(g, 128), gate=z, quant="row")


def test_layers_captured_and_replayed():
    """A captured decode step, replayed on new inputs, equals the eager one bit for bit; the pieces of two graphs with
    workspaces of their own do not mix."""
    g = gen(15)
    B, width, Hq, Hkv, page = 2, 128, 4, 1, 16
    proj = [randn(g, width, n * 128) * 0.06 for n in (Hq, Hkv, Hkv)] + [randn(g, Hq * 128, width) * 0.04]
    w = randn(g, width)
    c = [Paged([3999, 700], Hkv, 128, page, BF16, seed=s, columns=251) for s in (1, 2)]
    f, _ = gdn.rope_inv_freq(64)
    nbytes = gdn.paged_attn_workspace_bytes(B, Hq, Hkv, 128, page, 251, 4000)
    assert nbytes > 0
    graphs, outs, args = [], [], []
    for cc in c:
        lens = torch.tensor([4000, 701], dtype=torch.int32, device="cuda")
        pos = lens - 1
        last = (pos // page).long()
        # a fresh page where the sequence's new token starts one
        for b in range(B):
            if pos[b] % page == 0:
                cc.table[b, last[b]] = cc.k.shape[0] - 1
        slots = (cc.table[torch.arange(B, device="cuda"), last] * page + pos % page).to(torch.int32)
        x, r = randn(g, B, width), randn(g, B, width)
        ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        a = (x, r, w, (cc.k, cc.v), cc.table, pos, lens, slots, f, proj, 4000, ws)
        args.append(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for a in args:
            decode_layer(*a)
    torch.cuda.current_stream().wait_stream(side)
    for a in args:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            o = decode_layer(*a)
        graphs.append(gr)
        outs.append(o)
    for trial in range(3):
        for a in args:
            a[0].copy_(randn(g, B, width))
            a[1].copy_(randn(g, B, width))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for a, o in zip(args, outs):
            want = decode_layer(*a)
            assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])
            assert all(torch.equal(p, q) for p, q in zip(o[2], want[2]))
            assert torch.isfinite(o[0].float()).all()


def test_layers_on_another_stream():
    """``stream``: the work and the memory that the call allocates belong to that stream."""
    g = gen(16)
    s = torch.cuda.Stream()
    x, w = randn(g, 4096, 2048), randn(g, 2048)
    c = Paged([3000, 10], 2, 128, 16, BF16, seed=3)
    q, k = randn(g, 2, 8, 128), randn(g, 2, 2, 128)
    f, _ = gdn.rope_inv_freq(64)
    pos = torch.tensor([2999, 9], dtype=torch.int32, device="cuda")
    want = (gdn.rms_norm(x, w), gdn.rope_fwd(q, k, pos, f), gdn.paged_attn_fwd(q, c.k, c.v, c.table, c.seq_lens))
    torch.cuda.synchronize()
    for _ in range(5):
        s.wait_stream(torch.cuda.current_stream())
        got = (gdn.rms_norm(x, w, stream=s), gdn.rope_fwd(q, k, pos, f, stream=s),
               gdn.paged_attn_fwd(q, c.k, c.v, c.table, c.seq_lens, stream=s))
        torch.full((1 << 22,), 3.0, device="cuda")                # would reuse memory that the call gave up early
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(got[0][0], want[0][0])
        assert torch.equal(got[1][0], want[1][0]) and torch.equal(got[1][1], want[1][1])
        assert torch.equal(got[2][0], want[2][0])


def test_attn_allocates_its_own_workspace_in_the_library():
    """A C call without a workspace: allocated and freed on the stream."""
    from gated_deltanet_linear_17_b200 import _layers
    c = Paged([5000, 20], 2, 128, 16, BF16, seed=9)
    assert gdn.paged_attn_workspace_bytes(2, 8, 2, 128, 16, c.max_pages) > 0
    q = randn(gen(17), 2, 8, 128)
    want, _ = gdn.paged_attn_fwd(q, c.k, c.v, c.table, c.seq_lens)
    out = torch.empty_like(q)
    rc = _layers._layers_lib().gdn_paged_attn_fwd(
        q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), c.table.data_ptr(), c.seq_lens.data_ptr(), 0.0, out.data_ptr(),
        None, 2, 8, 2, 128, c.k.shape[0], 16, c.max_pages, 0, 1, None, 0, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and torch.equal(out, want)


@pytest.mark.parametrize("scale", [0.0, -0.5, NAN, float("inf")])
def test_attn_refuses_scales_that_are_not_positive(scale):
    """A scale at or below zero is the library's sign for its default; the binding lets none through as a value."""
    c = Paged([30, 40], 2, 64, 16, BF16)
    with pytest.raises(ValueError, match="scale"):
        gdn.paged_attn_fwd(randn(gen(18), 2, 4, 64), c.k, c.v, c.table, c.seq_lens, scale=scale)


@pytest.mark.parametrize("columns", [None, 4000])
def test_attn_nan_and_infinite_rows_stay_with_their_sequence(columns):
    """NaN in one sequence's keys or values, and an infinite value: that sequence alone is NaN (of the value, its
    column alone infinite or NaN), the next in the same list as if nothing were there."""
    c = Paged([130, 300, 1, 77], 2, 128, 16, BF16, seed=5)
    if columns:
        c = c.widened(columns)
    q = randn(gen(19), 4, 8, 128)
    want, want_lse = gdn.paged_attn_fwd(q, c.k, c.v, c.table, c.seq_lens, output_lse=True)
    place = lambda b, j: (int(c.table[b, j // 16]), j % 16)
    c.k[(*place(1, 200), 0)] = NAN              # head 0 of sequence 1
    c.v[(*place(0, 129), 1, 7)] = float("inf")  # column 7 of head 1 of sequence 0
    got, lse = gdn.paged_attn_fwd(q, c.k, c.v, c.table, c.seq_lens, output_lse=True)
    assert got[1, :4].isnan().all() and lse[1, :4].isnan().all()
    assert not got[0, 4:, 7].isfinite().any()   # the weight's second part may be below zero: infinity less infinity
    keep = torch.ones_like(got, dtype=torch.bool)
    keep[1, :4] = False
    keep[0, 4:, 7] = False
    assert torch.equal(got[keep], want[keep])
    lse[1, :4] = want_lse[1, :4]
    assert torch.equal(lse, want_lse)


def test_attn_one_workspace_for_calls_in_order():
    """Calls of different sizes behind one another on a stream may share a workspace, captured ones too."""
    cs = [Paged([9000, 5], 2, 128, 16, BF16, seed=6), Paged([700] * 40, 1, 64, 16, BF16, seed=7),
          Paged([3, 20000], 1, 256, 16, BF16, seed=8)]
    qs = [randn(gen(20), 2, 8, 128), randn(gen(21), 40, 24, 64), randn(gen(22), 2, 8, 256)]
    want = [gdn.paged_attn_fwd(q, c.k, c.v, c.table, c.seq_lens)[0] for q, c in zip(qs, cs)]
    ws = torch.empty(max(gdn.paged_attn_workspace_bytes(*q.shape[:2], c.k.shape[2], q.shape[2], 16, c.table.shape[1])
                         for q, c in zip(qs, cs)), dtype=torch.uint8, device="cuda")
    outs = [[torch.empty_like(q) for q in qs] for _ in range(4)]

    def run():
        for out in outs:
            for o, q, c in zip(out, qs, cs):
                gdn.paged_attn_fwd(q, c.k, c.v, c.table, c.seq_lens, out=o, workspace=ws)

    run()
    assert all(torch.equal(o, w) for out in outs for o, w in zip(out, want))
    for out in outs:
        for o in out:
            o.zero_()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        run()
    gr.replay()
    assert all(torch.equal(o, w) for out in outs for o, w in zip(out, want))


def test_layers_captured_with_copies_and_branches():
    """Launches that overlap their predecessor's end, in a graph whose predecessors are copies, fills and another
    branch's kernels: every one still waits for what it reads."""
    g = gen(23)
    B, Hq, Hkv, page, rows = 4, 8, 2, 16, 4096
    c = Paged([2500, 17, 900, 16], Hkv, 128, page, BF16, seed=9)
    f, _ = gdn.rope_inv_freq(128)
    lens = c.seq_lens
    pos = lens - 1
    slots = (c.table[torch.arange(B, device="cuda"), (pos // page).long()] * page + pos % page).to(torch.int32)
    w = randn(g, 1000)
    new = dict(x=randn(g, rows, 1000), q=randn(g, B, Hq, 128), k=randn(g, B, Hkv, 128), v=randn(g, B, Hkv, 128))
    held = {n: torch.zeros_like(t) for n, t in new.items()}
    side = torch.cuda.Stream()

    def step():
        for n in new:
            held[n].copy_(new[n])
        side.wait_stream(torch.cuda.current_stream())
        h, _, sc = gdn.rms_norm(held["x"], w, quant="row")
        with torch.cuda.stream(side):
            q, _ = gdn.rope_fwd(held["q"], held["k"], pos, f, v=held["v"], k_cache=c.k, v_cache=c.v, slots=slots)
            o, _ = gdn.paged_attn_fwd(q, c.k, c.v, c.table, lens)
            held["q"].zero_()
        held["x"].zero_()                              # behind the norm that read it
        h2, _, _ = gdn.rms_norm(held["x"], w)
        torch.cuda.current_stream().wait_stream(side)
        o2, _, _ = gdn.rms_norm(o, w[:128].contiguous())
        return h, sc, q, o, h2, o2

    step()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = step()
    for trial in range(3):
        for n in new:
            new[n].copy_(randn(g, *new[n].shape))
        gr.replay()
        torch.cuda.synchronize()
        got_now = [t.clone() for t in got]
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(got_now, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert not want[4].any() and torch.isfinite(want[3].float()).all()


@pytest.mark.parametrize("quant, scales", [(None, None), ("row", ()), ("block", (3,))])
def test_norm_of_one_row(quant, scales):
    """x [width]: the same as a matrix of one row; the scale of a row has no dimension."""
    g = gen(24)
    x, w = randn(g, 300), randn(g, 300)
    out, none, sc = gdn.rms_norm(x, w, quant=quant)
    want, _, wsc = gdn.rms_norm(x[None], w, quant=quant)
    assert out.shape == (300,) and none is None and torch.equal(out.view(torch.uint8), want[0].view(torch.uint8))
    assert sc is None if quant is None else sc.shape == scales and torch.equal(sc, wsc[0])


def test_layers_from_two_threads():
    """Two host threads, a stream and inputs each: the calls share nothing."""
    import threading

    f, _ = gdn.rope_inv_freq(64)
    sets = []
    for i in (0, 1):
        g = gen(25 + i)
        c = Paged([4000 + i, 33], 2, 128, 16, BF16, seed=10 + i)
        sets.append((c, randn(g, 2, 8, 128), randn(g, 2, 2, 128), randn(g, 64, 1000 + 24 * i), randn(g, 1000 + 24 * i),
                     torch.tensor([3999 + i, 32], dtype=torch.int32, device="cuda")))

    def step(c, q, k, x, w, pos):
        turned, _ = gdn.rope_fwd(q, k, pos, f)
        return (gdn.rms_norm(x, w, quant="row")[0].view(torch.uint8), turned,
                gdn.paged_attn_fwd(turned, c.k, c.v, c.table, c.seq_lens)[0])

    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    same = [0, 0]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                got = step(*sets[i])
                same[i] += all(torch.equal(a, b) for a, b in zip(got, want[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert same == [50, 50]
