"""Cases of the serving operators that stand around the delta-rule layers of a hybrid model:

  rms_norm        the root-mean-square norm, with the residual's addition, the SiLU gate of a delta-rule layer's
                  output and an output in 8 bits with scales
  rope            rotary positions of q and k, with the new keys and values written into a paged cache
  paged_attn      attention of one new token of each sequence over that cache

Each case can be run in a plain form of elementary torch operations, or by the package's own entry points (``own``).
Types, sizes and the ragged lengths are in the case; everything random comes from the seed.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -126
BLOCK = 128


def listed():
    return [
        # one decode step's block norm: a handful of tokens, latency alone
        dict(name="norm_step", op="rms_norm", dtype="bf16", rows=8, width=2048, residual=True, gate=False, quant="none"),
        # the norm before a layer's 8-bit projections over a prefill: sum with the residual, one scale a token
        dict(name="norm_prefill_row8", op="rms_norm", dtype="bf16", rows=16384, width=4096, residual=True, gate=False,
             quant="row"),
        # the output norm of a one-layer delta-rule prefill (32768 tokens, 32 v-heads of 128), gated, scales by head
        dict(name="norm_heads_gated8", op="rms_norm", dtype="bf16", rows=32768 * 32, width=128, residual=False,
             gate=True, quant="block"),
        # a width that no vector load divides, in 32 bits
        dict(name="norm_odd", op="rms_norm", dtype="fp32", rows=4099, width=1537, residual=True, gate=True,
             quant="none"),
        # the new tokens of a decode batch: a quarter of the head turned, keys and values scattered over the pages
        dict(name="rope_step", op="rope", dtype="bf16", tokens=64, q_heads=16, kv_heads=2, head_dim=256, rotary=64,
             interleaved=False, farthest=32768, cache=True, page=16, scattered=True),
        # a prefill of 32768 tokens filling its pages in order
        dict(name="rope_prefill", op="rope", dtype="bf16", tokens=32768, q_heads=16, kv_heads=2, head_dim=256,
             rotary=64, interleaved=False, farthest=32768, cache=True, page=16, scattered=False),
        # the whole head in neighbouring pairs, far positions, an odd number of tokens, no cache
        dict(name="rope_far", op="rope", dtype="fp16", tokens=4099, q_heads=32, kv_heads=8, head_dim=128, rotary=128,
             interleaved=True, farthest=1 << 20, cache=False, page=16, scattered=False),
        # one short conversation
        dict(name="attn_short", op="paged_attn", dtype="bf16", batch=1, q_heads=16, kv_heads=2, head_dim=256, page=16,
             shortest=700, longest=700),
        # one very long one: all the parallelism is in the cache's length
        dict(name="attn_long", op="paged_attn", dtype="bf16", batch=1, q_heads=16, kv_heads=2, head_dim=256, page=16,
             shortest=131072, longest=131072),
        # every head its own keys, odd page size, empty and short sequences among the others
        dict(name="attn_ragged", op="paged_attn", dtype="fp16", batch=37, q_heads=12, kv_heads=12, head_dim=64,
             page=24, shortest=0, longest=5000),
        # a serving batch of ordinary lengths
        dict(name="attn_batch", op="paged_attn", dtype="bf16", batch=64, q_heads=32, kv_heads=8, head_dim=128,
             page=16, shortest=1, longest=8192),
        # a full serving batch of long lengths
        dict(name="attn_large", op="paged_attn", dtype="bf16", batch=256, q_heads=16, kv_heads=2, head_dim=256,
             page=64, shortest=1024, longest=16384),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("rms_norm", "rope", "paged_attn"))
    if op == "rms_norm":
        width = rng.choice((64, 128, 256, 2048, 4096, 5120, 8192, _log(rng, 33, 16384), _log(rng, 33, 16384) | 1))
        gate = rng.random() < 0.5
        return dict(op=op, dtype=rng.choice(("bf16", "bf16", "fp16", "fp32")),
                    rows=_log(rng, 1, max(1, (1 << 26) // width)), width=width, residual=not gate or rng.random() < 0.3,
                    gate=gate, quant=rng.choice(("none", "row", "block")))
    if op == "rope":
        head_dim = rng.choice((64, 80, 96, 128, 192, 256))
        kv_heads = rng.randint(1, 8)
        q_heads = kv_heads * rng.randint(1, 8)
        most = (1 << 27) // ((q_heads + 2 * kv_heads) * head_dim)
        return dict(op=op, dtype=rng.choice(("bf16", "bf16", "fp16", "fp32")), tokens=_log(rng, 1, most),
                    q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim,
                    rotary=rng.choice((head_dim, head_dim // 2, head_dim // 4, 2 * rng.randint(1, head_dim // 2))),
                    interleaved=rng.random() < 0.5, farthest=_log(rng, 16, 1 << 21), cache=rng.random() < 0.7,
                    page=rng.choice((1, 16, 24, 32, 64)), scattered=rng.random() < 0.5)
    head_dim = rng.choice((64, 128, 256))
    kv_heads = rng.randint(1, 12)
    batch = _log(rng, 1, 256)
    most = max(1, min(131072, (1 << 30) // (head_dim * kv_heads * batch)))
    longest = _log(rng, 1, most)
    return dict(op=op, dtype=rng.choice(("bf16", "fp16")), batch=batch, q_heads=kv_heads * rng.randint(1, 16),
                kv_heads=kv_heads, head_dim=head_dim, page=rng.choice((8, 16, 17, 24, 32, 64, 128)),
                shortest=rng.choice((0, 1, longest // 2, longest)), longest=longest)


def _lengths(case):
    """The lengths of the cache's sequences: the longest, the shortest, and between them what the sizes give."""
    r = random.Random(case["batch"] * 1000003 + case["longest"])
    n = [r.randint(case["shortest"], case["longest"]) for _ in range(case["batch"])]
    n[-1] = case["shortest"]
    n[0] = case["longest"]
    return n


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=dt if dt != torch.float32 else None)

    s = dict(case)
    if case["op"] == "rms_norm":
        shape = (case["rows"], case["width"])
        s["x"] = normal(*shape)
        s["residual_in"] = normal(*shape).mul_(3.0) if case["residual"] else None
        s["gate_in"] = normal(*shape) if case["gate"] else None
        s["weight"] = normal(case["width"]).mul_(0.1).add_(1.0)
        s["eps"] = 1e-6
    elif case["op"] == "rope":
        T, D = case["tokens"], case["head_dim"]
        s["q"] = normal(T, case["q_heads"], D)
        s["k"] = normal(T, case["kv_heads"], D)
        first = int(torch.randint(0, max(1, case["farthest"] - T + 1), (1,), generator=gen, device=dev))
        run = torch.arange(T, device=dev, dtype=torch.int64) + first
        some = torch.randint(0, case["farthest"], (T,), generator=gen, device=dev)
        s["positions"] = (some if case["scattered"] else run).to(torch.int32)
        half = torch.arange(0, case["rotary"], 2, device=dev, dtype=torch.float64) / case["rotary"]
        s["inv_freq"] = (10000.0 ** -half).float()
        s["mscale"] = 1.0 if case["farthest"] <= 32768 else 0.1 * math.log(case["farthest"] / 32768) + 1.0
        s["k_cache"] = s["v_cache"] = s["slots"] = s["v"] = None
        if case["cache"]:
            page = case["page"]
            pages = -(-T // page) + 3
            s["v"] = normal(T, case["kv_heads"], D)
            s["k_cache"] = normal(pages, page, case["kv_heads"], D)
            s["v_cache"] = normal(pages, page, case["kv_heads"], D)
            if case["scattered"]:
                s["slots"] = torch.randperm(pages * page, generator=gen, device=dev)[:T].to(torch.int32)
            else:
                t = torch.arange(T, device=dev)
                perm = torch.randperm(pages, generator=gen, device=dev)
                s["slots"] = (perm[t // page] * page + t % page).to(torch.int32)
    else:
        lens, page = _lengths(case), case["page"]
        need = [-(-n // page) for n in lens]
        total = sum(need) + 3
        s["q"] = normal(case["batch"], case["q_heads"], case["head_dim"])
        s["k_cache"] = normal(total, page, case["kv_heads"], case["head_dim"])
        s["v_cache"] = normal(total, page, case["kv_heads"], case["head_dim"])
        n = torch.tensor(lens, device=dev)
        p = torch.tensor(need, device=dev)
        perm = torch.randperm(total, generator=gen, device=dev)
        col = torch.arange(max(1, max(need)), device=dev)
        at = (torch.cumsum(p, 0) - p)[:, None] + col[None, :]
        s["block_table"] = torch.where(col[None, :] < p[:, None], perm[at.clamp(max=total - 1)], -1).to(torch.int32)
        s["seq_lens"] = n.to(torch.int32)
        s["scale"] = 1.0 / math.sqrt(case["head_dim"])
    return s


# ------------------------------------------------------------------ the operators in plain form


def _plain_norm(s):
    z = s["x"].float()
    if s["residual_in"] is not None:
        z = z + s["residual_in"].float()
    y = z * torch.rsqrt((z * z).mean(dim=-1, keepdim=True) + s["eps"]) * s["weight"].float()
    if s["gate_in"] is not None:
        g = s["gate_in"].float()
        y = y * (g / (1.0 + torch.exp(-g)))
    dt = s["x"].dtype
    got = {"residual": z.to(dt) if s["residual_in"] is not None else None}
    if s["quant"] == "none":
        got["out"] = y.to(dt)
        return got
    rows, width = y.shape
    size = width if s["quant"] == "row" else BLOCK
    groups = -(-width // size)
    padded = torch.zeros(rows, groups * size, device=y.device)
    padded[:, :width] = y
    padded = padded.view(rows, groups, size)
    scales = (padded.abs().amax(dim=-1) / E4M3_MAX).clamp(min=MIN_SCALE)
    q = (padded / scales[:, :, None]).view(rows, groups * size)[:, :width]
    got["out"] = q.to(torch.float8_e4m3fn)
    got["scales"] = scales.view(rows) if s["quant"] == "row" else scales
    return got


def _turn(x, cos, sin, interleaved):
    """x [T, H, D] with its first 2 n columns turned by the angles whose cosines are cos [T, n]."""
    n = cos.shape[1]
    c, d = cos[:, None, :], sin[:, None, :]
    y = x.float().clone()
    a, b = (x[:, :, 0:2 * n:2].float(), x[:, :, 1:2 * n:2].float()) if interleaved else \
        (x[:, :, :n].float(), x[:, :, n:2 * n].float())
    first, second = a * c - b * d, b * c + a * d
    if interleaved:
        y[:, :, 0:2 * n:2], y[:, :, 1:2 * n:2] = first, second
    else:
        y[:, :, :n], y[:, :, n:2 * n] = first, second
    return y.to(x.dtype)


def _plain_rope(s):
    angles = s["positions"].double()[:, None] * s["inv_freq"].double()[None, :]
    cos, sin = (torch.cos(angles) * s["mscale"]).float(), (torch.sin(angles) * s["mscale"]).float()
    q, k = _turn(s["q"], cos, sin, s["interleaved"]), _turn(s["k"], cos, sin, s["interleaved"])
    if s["k_cache"] is None:
        return {"q": q, "k": k}
    slots = s["slots"].long()
    s["k_cache"].view(-1, *k.shape[1:])[slots] = k
    s["v_cache"].view(-1, *k.shape[1:])[slots] = s["v"]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attn(s):
    B, Hq, D = s["q"].shape
    Hkv = s["k_cache"].shape[2]
    table = s["block_table"].clamp(min=0).long()
    k = s["k_cache"][table].float().view(B, -1, Hkv, D).permute(0, 2, 3, 1)       # [B, Hkv, D, L]
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    scores = torch.matmul(q, k) * s["scale"]                                      # [B, Hkv, G, L]
    del k
    L = scores.shape[-1]
    seen = torch.arange(L, device=q.device)[None, :] < s["seq_lens"][:, None]
    scores = scores.masked_fill(~seen[:, None, None, :], -math.inf)
    most = scores.amax(dim=-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp(scores - most)
    total = p.sum(dim=-1, keepdim=True)
    v = s["v_cache"][table].float().view(B, -1, Hkv, D).permute(0, 2, 1, 3)       # [B, Hkv, L, D]
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    lse = (torch.log(total) + most).view(B, Hq).masked_fill(s["seq_lens"][:, None] == 0, -math.inf)
    return {"out": o.view(B, Hq, D).to(s["q"].dtype), "lse": lse}


def run(state):
    s = state
    if own:
        import gated_deltanet_linear_17_b200 as gdn
        if s["op"] == "rms_norm":
            quant = None if s["quant"] == "none" else s["quant"]
            out, residual, scales = gdn.rms_norm(s["x"], s["weight"], residual=s["residual_in"], gate=s["gate_in"],
                                                 eps=s["eps"], quant=quant)
            got = {"residual": residual, "out": out}
            return got if quant is None else {**got, "scales": scales}
        if s["op"] == "rope":
            q, k = gdn.rope_fwd(s["q"], s["k"], s["positions"], s["inv_freq"], v=s["v"], k_cache=s["k_cache"],
                                v_cache=s["v_cache"], slots=s["slots"], interleaved=s["interleaved"],
                                mscale=s["mscale"])
            return {"q": q, "k": k} if s["k_cache"] is None else \
                {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        out, lse = gdn.paged_attn_fwd(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"],
                                      scale=s["scale"], max_seqlen=s["longest"], output_lse=True)
        return {"out": out, "lse": lse}
    return {"rms_norm": _plain_norm, "rope": _plain_rope, "paged_attn": _plain_attn}[s["op"]](s)


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "rms_norm":
        n = case["rows"] * case["width"]
        quant = case["quant"] != "none"
        scales = case["rows"] * (1 if case["quant"] == "row" else -(-case["width"] // BLOCK)) * 4 if quant else 0
        read = n * size * (1 + case["residual"] + case["gate"]) + case["width"] * size
        return {"bytes": read + n * (1 if quant else size) + n * size * case["residual"] + scales,
                "flops": n * (4 + case["residual"] + 5 * case["gate"] + 2 * quant)}
    if case["op"] == "rope":
        T, D = case["tokens"], case["head_dim"]
        kv = T * case["kv_heads"] * D * size
        moved = 2 * T * case["q_heads"] * D * size + 2 * kv + (2 * kv + 4 * T if case["cache"] else 0)
        return {"bytes": moved + 4 * T + 2 * case["rotary"],
                "flops": 3 * T * (case["q_heads"] + case["kv_heads"]) * case["rotary"]}
    lens, D = _lengths(case), case["head_dim"]
    rows = case["batch"] * case["q_heads"]
    pages = sum(-(-n // case["page"]) for n in lens)
    return {"bytes": sum(lens) * case["kv_heads"] * D * size * 2 + rows * D * size * 2 + rows * 4 + 4 * pages +
            4 * case["batch"], "flops": 4 * sum(lens) * case["q_heads"] * D}


# ------------------------------------------------------------------ the definitions in 64 bits


def _to_e4m3(v):
    """v rounded to the nearest value of 4 exponent and 3 mantissa bits, halves to even (|v| <= 448)."""
    exponent = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(exponent - 3.0)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_norm(s):
    out, residual, scales = [], [], []
    rows = s["x"].shape[0]
    part = max(1, (1 << 24) // s["width"])
    for r in range(0, rows, part):
        z = s["x"][r:r + part].double()
        if s["residual_in"] is not None:
            z += s["residual_in"][r:r + part].double()
            residual.append(z.clone())
        y = z / torch.sqrt(torch.sum(z ** 2, dim=1, keepdim=True) / s["width"] + s["eps"])
        y *= s["weight"].double()
        if s["gate_in"] is not None:
            g = s["gate_in"][r:r + part].double()
            y *= g * torch.sigmoid(g)
        if s["quant"] != "none":
            pieces = [y] if s["quant"] == "row" else list(torch.split(y, BLOCK, dim=1))
            sc = [torch.clamp(p.abs().max(dim=1, keepdim=True).values / E4M3_MAX, min=MIN_SCALE) for p in pieces]
            y = torch.cat([_to_e4m3(p / c) for p, c in zip(pieces, sc)], dim=1)
            scales.append(torch.cat(sc, dim=1))
        out.append(y)
    got = {"residual": torch.cat(residual) if residual else None, "out": torch.cat(out)}
    if scales:
        got["scales"] = torch.cat(scales)[:, 0] if s["quant"] == "row" else torch.cat(scales)
    return got


def _exact_rope(s):
    n = s["inv_freq"].numel()
    angle = torch.outer(s["positions"].double(), s["inv_freq"].double())
    turn = torch.polar(torch.full_like(angle, s["mscale"]), angle)[:, None, :]

    def turned(x):
        head, rest = x[..., :2 * n].double(), x[..., 2 * n:].double()
        pair = head.unflatten(-1, (n, 2)) if s["interleaved"] else head.unflatten(-1, (2, n)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        z = z if s["interleaved"] else z.transpose(-1, -2)
        return torch.cat([z.flatten(-2), rest], dim=-1)

    q, k = turned(s["q"]), turned(s["k"])
    if s["k_cache"] is None:
        return {"q": q, "k": k}
    caches = []
    for cache, new in ((s["k_cache"], k), (s["v_cache"], s["v"].double())):
        c = cache.double()
        c.flatten(0, 1).index_copy_(0, s["slots"].long(), new)
        caches.append(c)
    return {"q": q, "k_cache": caches[0], "v_cache": caches[1]}


def _exact_attn(s):
    B, Hq, D = s["q"].shape
    Hkv, page = s["k_cache"].shape[2], s["page"]
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(s)):
        if n == 0:
            continue
        pages = s["block_table"][b, :-(-n // page)].long()
        for h in range(Hkv):
            rows = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            k = s["k_cache"][pages, :, h].flatten(0, 1)[:n].double()
            v = s["v_cache"][pages, :, h].flatten(0, 1)[:n].double()
            scores = (s["q"][b, rows].double() @ k.T) * s["scale"]
            lse[b, rows] = torch.logsumexp(scores, dim=1)
            out[b, rows] = torch.softmax(scores, dim=1) @ v
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"rms_norm": _exact_norm, "rope": _exact_rope, "paged_attn": _exact_attn}[case["op"]](s)
