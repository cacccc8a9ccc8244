"""ctypes binding of the layer operators (include/gdn_layers.h): the norm, the rotary positions with
the write into a paged cache, and the attention of one new token over that cache.

As in ``_binding``: shapes, types and devices are checked, torch supplies the device memory and the
stream, and every step of the computation runs in the library's CUDA kernels.  A call runs on its
tensors' device whatever the current device is, and on that device's current stream unless ``stream``
is given; memory that a call allocates belongs to the stream that it runs on.  The operators are forward
only: no gradient is recorded through them.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math

import torch

from . import _binding as _b

QUANT = {None: 0, "row": 1, "block": 2}
QUANT_GROUP = 128

_lib = None


def _layers_lib():
    global _lib
    if _lib is None:
        L = _b.lib()
        p, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        # x residual gate weight | eps offset | out residual_out scales | rows width | act weight quant | stream
        L.gdn_rms_norm.restype = ctypes.c_int
        L.gdn_rms_norm.argtypes = [p, p, p, p, f32, f32, p, p, p, i64, i32, i32, i32, i32, p]
        # q k v positions inv_freq slots | mscale | q_out k_out k_cache v_cache | T Hq Hkv D rotary interleaved |
        # cache_rows act stream
        L.gdn_rope_fwd.restype = ctypes.c_int
        L.gdn_rope_fwd.argtypes = [p, p, p, p, p, p, f32, p, p, p, p, i64, i32, i32, i32, i32, i32, i64, i32, p]
        L.gdn_paged_attn_workspace_bytes.restype = sz
        L.gdn_paged_attn_workspace_bytes.argtypes = [i32] * 7
        # q k_cache v_cache table lens | scale | out lse | B Hq Hkv D P page max_pages max_seqlen act | workspace
        L.gdn_paged_attn_fwd.restype = ctypes.c_int
        L.gdn_paged_attn_fwd.argtypes = [p, p, p, p, p, f32, p, p, i32, i32, i32, i32, i32, i32, i32, i32, i32, p, sz,
                                         p]
        _lib = L
    return _lib


_MOST = 0x7fffffff  # of the sizes that the library takes in 32 bits; ctypes would cut larger ones down


def _too_large(*sizes):
    return ValueError(f"a size of {max(sizes)} is beyond 2^31 - 1")


def _ptr(t):
    return None if t is None else t.data_ptr()


_Tensor, _f32, _i32 = torch.Tensor, torch.float32, torch.int32


def _need(t, name, dtype, shape, index):
    """``_binding._need`` (on CUDA device ``index``), with the comparisons of a good tensor kept cheap: a decode step's
    calls take a few microseconds."""
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == index
            and t.is_contiguous()):
        _b._need(t, name, dtype, shape, torch.device("cuda", index))


@contextlib.contextmanager
def _on(index, stream):
    """Device ``index`` and ``stream`` (or the device's current stream) as the current ones."""
    if stream is not None and stream.device.index != index:
        raise RuntimeError(f"the stream is on {stream.device}, the tensors on cuda:{index}")
    with torch.cuda.device(index), torch.cuda.stream(stream):
        yield


def _stream_handle(index):
    return torch.cuda.current_stream(index).cuda_stream


# The current device, and the current stream's handle on a device.  torch's private ones take a tenth of the public
# ones' time; a torch without them (built for the CPU alone, or of another version) has the public ones.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_handle)


def _tensor(t, name):
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    return t


def _cuda(t, name):
    """The index of the CUDA device that t lies on."""
    index = _tensor(t, name).get_device()
    if index < 0 or not t.is_cuda:
        raise RuntimeError(f"{name} must be on a CUDA device (got {t.device})")
    return index


def _act(t, name, types=_b.DTYPES):
    if t.dtype not in types:
        raise RuntimeError(f"{name} must be one of {[str(d) for d in types]} (got {t.dtype})")
    return t.dtype


def rms_norm(x, weight, residual=None, gate=None, eps=1e-6, weight_offset=0.0, quant=None, out=None,
             residual_out=None, scales=None, stream=None):
    """Root-mean-square norm through ``gdn_rms_norm``; returns (out, residual_out, scales).

    z = x + residual; y = z / sqrt(mean(z^2) + eps) * (weight + weight_offset); with a ``gate``,
    y *= gate * sigmoid(gate) (the gated norm of a delta-rule layer's output, of x [T, Nv, 128]).
    x [..., width], residual and gate of x's shape and type (bf16, fp16 or fp32), weight [width] of
    that type or fp32.  ``residual_out`` holds z in x's type (None without a residual).
    ``quant`` None gives y in x's type (scales None); "row" gives float8_e4m3fn with one fp32 scale per
    row, [...]; "block" one per row and 128 columns, [..., ceil(width / 128)]: y is about out * scale.
    ``out`` may be x (without ``quant``) and ``residual_out`` may be the residual: then they are
    updated in place."""
    dev = _cuda(x, "x")
    if stream is not None or dev != _current_device():
        with _on(dev, stream):
            return rms_norm(x, weight, residual, gate, eps, weight_offset, quant, out, residual_out, scales)
    if quant not in QUANT:
        raise ValueError(f"quant must be one of {list(QUANT)} (got {quant!r})")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be [..., width] with at least one column")
    act, shape = _act(x, "x"), x.shape
    width = shape[-1]
    if width > _MOST:
        raise _too_large(width)
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    wdt = _f32 if _tensor(weight, "weight").dtype is _f32 else act
    _need(weight, "weight", wdt, (width,), dev)
    if residual is not None:
        _need(residual, "residual", act, shape, dev)
    if gate is not None:
        _need(gate, "gate", act, shape, dev)
    if residual_out is not None:
        if residual is None:
            raise ValueError("residual_out needs a residual")
        _need(residual_out, "residual_out", act, shape, dev)
    odt = act if quant is None else torch.float8_e4m3fn
    if out is not None:
        _need(out, "out", odt, shape, dev)
    lead = shape[:-1]
    sshape = None if quant is None else lead if quant == "row" else (*lead, -(-width // QUANT_GROUP))
    if scales is not None:
        if quant is None:
            raise ValueError("scales need quant")
        _need(scales, "scales", _f32, sshape, dev)
    if out is None:
        out = torch.empty_like(x) if quant is None else torch.empty_like(x, dtype=odt)
    if residual is not None and residual_out is None:
        residual_out = torch.empty_like(x)
    if quant is not None and scales is None:
        scales = x.new_empty(sshape, dtype=_f32)
    rc = _layers_lib().gdn_rms_norm(x.data_ptr(), _ptr(residual), _ptr(gate), weight.data_ptr(), eps, weight_offset,
                                    out.data_ptr(), _ptr(residual_out), _ptr(scales), x.numel() // width, width,
                                    _b.DTYPES[act], _b.DTYPES[wdt], QUANT[quant], _current_stream(dev))
    if rc:
        _b._check(rc, "gdn_rms_norm")
    return out, residual_out, scales


def rope_inv_freq(rotary, base=10000.0, scaling=None, factor=1.0, original_max=4096, beta_fast=32.0, beta_slow=1.0,
                  device="cuda"):
    """The angles per position of ``rope_fwd``, fp32 [rotary / 2] on ``device``, and the factor of the
    turned columns (its ``mscale``); returns (inv_freq, mscale).

    ``scaling`` None: base^(-2i/rotary).  For contexts ``factor`` times longer than ``original_max``:
    "linear" divides every frequency by ``factor``; "ntk" raises the base by factor^(rotary/(rotary-2)),
    so that the slowest angle is divided by ``factor`` and the fastest kept; "yarn" (Peng et al. 2023)
    keeps angles that turn at least ``beta_fast`` times over ``original_max`` positions, divides those
    that turn at most ``beta_slow`` times, blends linearly in between, and gives mscale
    0.1 ln(factor) + 1.  Computed in 64 bits."""
    if rotary < 2 or rotary % 2:
        raise ValueError("rotary must be even and at least 2")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError("scaling must be None, 'linear', 'ntk' or 'yarn'")
    if not (base > 1.0 and factor >= 1.0 and original_max >= 1 and beta_fast > beta_slow > 0.0):
        raise ValueError("rope_inv_freq needs base > 1, factor >= 1, original_max >= 1 and beta_fast > beta_slow > 0")
    mscale = 1.0
    if scaling == "ntk" and rotary > 2:
        base = base * factor ** (rotary / (rotary - 2))
    i = torch.arange(0, rotary, 2, dtype=torch.float64)
    f = base ** (-i / rotary)
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        def place(turns):  # the (fractional) index of the angle that turns so often over original_max
            return rotary * math.log(original_max / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))

        low, high = max(math.floor(place(beta_fast)), 0), min(math.ceil(place(beta_slow)), rotary - 1)
        ramp = ((i / 2 - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
        if place(beta_slow) <= 0.0:  # no angle turns more often than that: the ramp ends before the first
            ramp = torch.ones_like(i)
        f = f * (1.0 - ramp) + f / factor * ramp
        mscale = 0.1 * math.log(factor) + 1.0
    return f.float().to(device), mscale


def rope_fwd(q, k, positions, inv_freq, v=None, k_cache=None, v_cache=None, slots=None, interleaved=False,
             mscale=1.0, q_out=None, k_out=None, stream=None):
    """Rotary positions of q and k, and the write into a paged cache, through ``gdn_rope_fwd``; returns
    (q_out, k_out).

    q [T, Hq, D], k [T, Hkv, D] of one type (bf16, fp16 or fp32), positions [T] int32, inv_freq fp32
    [rotary / 2] (``rope_inv_freq``).  The first ``rotary`` columns of a head turn in the pairs
    (i, rotary/2 + i), or (2i, 2i + 1) when ``interleaved``; the turned columns are multiplied by
    ``mscale``.  With ``k_cache`` and ``v_cache`` [P, page_size, Hkv, D], the turned keys and v [T, Hkv, D]
    also go to the cache rows ``slots`` [T] int32 (page * page_size + place in the page; a slot
    outside the cache marks a padding token, which is not written; slots have to differ), and the turned
    keys are returned only if ``k_out`` is given (else None).  ``q_out`` may be q, ``k_out`` may be k."""
    dev = _cuda(q, "q")
    if stream is not None or dev != _current_device():
        with _on(dev, stream):
            return rope_fwd(q, k, positions, inv_freq, v, k_cache, v_cache, slots, interleaved, mscale, q_out, k_out)
    if q.dim() != 3 or _tensor(k, "k").dim() != 3:
        raise ValueError("q must be [T, Hq, D] and k [T, Hkv, D]")
    act = _act(q, "q")
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    if Hq > _MOST or Hkv > _MOST or D > _MOST:
        raise _too_large(Hq, Hkv, D)
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    _need(k, "k", act, (T, Hkv, D), dev)
    _need(positions, "positions", _i32, (T,), dev)
    turned = _tensor(inv_freq, "inv_freq").shape
    if len(turned) != 1 or 2 * turned[0] > D:
        raise ValueError(f"inv_freq must be [rotary / 2] with rotary <= {D} (got {tuple(turned)})")
    _need(inv_freq, "inv_freq", _f32, turned, dev)
    rows = 0
    if (k_cache is None) != (v_cache is None) or (k_cache is None) != (slots is None) or \
            (k_cache is None) != (v is None):
        raise ValueError("k_cache, v_cache, slots and v belong together: give all or none")
    if k_cache is not None:
        cshape = _tensor(k_cache, "k_cache").shape
        if len(cshape) != 4:
            raise ValueError("k_cache and v_cache must be [P, page_size, Hkv, D]")
        cshape = (cshape[0], cshape[1], Hkv, D)
        _need(v, "v", act, (T, Hkv, D), dev)
        _need(k_cache, "k_cache", act, cshape, dev)
        _need(v_cache, "v_cache", act, cshape, dev)
        _need(slots, "slots", _i32, (T,), dev)
        rows = cshape[0] * cshape[1]
    if q_out is not None:
        _need(q_out, "q_out", act, (T, Hq, D), dev)
    if k_out is not None:
        _need(k_out, "k_out", act, (T, Hkv, D), dev)
    if q_out is None:
        q_out = torch.empty_like(q)
    if k_out is None and k_cache is None:
        k_out = torch.empty_like(k)
    rc = _layers_lib().gdn_rope_fwd(q.data_ptr(), k.data_ptr(), _ptr(v), positions.data_ptr(), inv_freq.data_ptr(),
                                    _ptr(slots), mscale, q_out.data_ptr(), _ptr(k_out), _ptr(k_cache), _ptr(v_cache),
                                    T, Hq, Hkv, D, 2 * turned[0], 1 if interleaved else 0, rows, _b.DTYPES[act],
                                    _current_stream(dev))
    if rc:
        _b._check(rc, "gdn_rope_fwd")
    return q_out, k_out


@functools.lru_cache(maxsize=1024)
def paged_attn_workspace_bytes(B, Hq, Hkv, D, page_size, max_pages, max_seqlen=0) -> int:
    """Bytes of workspace of ``paged_attn_fwd`` for these sizes (``gdn_paged_attn_workspace_bytes``)."""
    return int(_layers_lib().gdn_paged_attn_workspace_bytes(B, Hq, Hkv, D, page_size, max_pages, max_seqlen))


def paged_attn_fwd(q, k_cache, v_cache, block_table, seq_lens, scale=None, max_seqlen: int = 0, out=None, lse=None,
                   output_lse=False, workspace=None, stream=None):
    """Attention of one new token of each sequence over a paged cache, through ``gdn_paged_attn_fwd``;
    returns (out, lse).

    q [B, Hq, D] bf16 or fp16, D 64, 128 or 256; k_cache, v_cache [P, page_size, Hkv, D] of q's type, Hq a
    multiple of Hkv (query head h reads key/value head h // (Hq // Hkv)); block_table [B, max_pages]
    int32, the pages of each sequence in order (entries past its last page are not read); seq_lens [B]
    int32, the keys of each sequence, the new token's own among them.  ``scale`` is positive, in fp32's
    range (default 1/sqrt(D)).  ``max_seqlen`` is the longest length if known, else 0 (it sets how the work
    is split).  A length of 0 gives a zero row and lse -inf; a length beyond the table or a page outside the
    cache gives NaN for that sequence.
    ``lse`` [B, Hq] fp32 is written when given or when ``output_lse``.  ``workspace``: a device buffer
    of ``paged_attn_workspace_bytes`` bytes, allocated here when not given; calls that can overlap on
    the GPU, replayed graphs among them, need buffers of their own."""
    dev = _cuda(q, "q")
    if stream is not None or dev != _current_device():
        with _on(dev, stream):
            return paged_attn_fwd(q, k_cache, v_cache, block_table, seq_lens, scale, max_seqlen, out, lse, output_lse,
                                  workspace)
    act = _act(q, "q", (torch.bfloat16, torch.float16))
    cshape, tshape = _tensor(k_cache, "k_cache").shape, _tensor(block_table, "block_table").shape
    if q.dim() != 3 or len(cshape) != 4 or len(tshape) != 2:
        raise ValueError("q must be [B, Hq, D], the caches [P, page_size, Hkv, D] and block_table [B, max_pages]")
    B, Hq, D = q.shape
    P, page, Hkv, _ = cshape
    if Hkv < 1 or Hq < 1 or Hq % Hkv:
        raise ValueError(f"Hq ({Hq}) must be a multiple of Hkv ({Hkv})")
    if page < 1:
        raise ValueError("page_size must be at least 1")
    max_seqlen = min(int(max_seqlen), 0x7fffffff)
    if max_seqlen < 0:
        raise ValueError("max_seqlen must not be negative")
    if scale is not None and not 1.4e-45 <= scale <= 2.3e38:
        raise ValueError(f"scale must be positive and finite in fp32, at most 2.3e38 (got {scale})")
    max_pages = tshape[1]
    if B > _MOST or Hq > _MOST or D > _MOST or P > _MOST or page > _MOST or max_pages > _MOST:
        raise _too_large(B, Hq, D, P, page, max_pages)
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    _need(k_cache, "k_cache", act, (P, page, Hkv, D), dev)
    _need(v_cache, "v_cache", act, (P, page, Hkv, D), dev)
    _need(block_table, "block_table", _i32, (B, max_pages), dev)
    _need(seq_lens, "seq_lens", _i32, (B,), dev)
    if out is not None:
        _need(out, "out", act, (B, Hq, D), dev)
    if lse is not None:
        _need(lse, "lse", _f32, (B, Hq), dev)
    if workspace is not None:
        if _cuda(workspace, "workspace") != dev or not workspace.is_contiguous():
            raise RuntimeError(f"workspace must be a contiguous tensor on cuda:{dev}")
    if out is None:
        out = torch.empty_like(q)
    if lse is None and output_lse:
        lse = torch.empty(B, Hq, dtype=_f32, device=q.device)  # (sizes as a tuple take half a microsecond more)
    if workspace is None:
        nbytes = paged_attn_workspace_bytes(B, Hq, Hkv, D, page, max_pages, max_seqlen)
        if nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = _layers_lib().gdn_paged_attn_fwd(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
                                          seq_lens.data_ptr(), 0.0 if scale is None else scale, out.data_ptr(),
                                          _ptr(lse), B, Hq, Hkv, D, P, page, max_pages, max_seqlen, _b.DTYPES[act],
                                          _ptr(workspace), ws_bytes, _current_stream(dev))
    if rc:
        _b._check(rc, "gdn_paged_attn_fwd")
    return out, lse
