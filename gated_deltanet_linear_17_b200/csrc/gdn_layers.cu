// Host side of the layer operators (include/gdn_layers.h): argument checks and launches.
#include "gdn_layers.h"

#include <float.h>
#include <math.h>

#include <algorithm>

#include "gdn_testing.h"
#include "layers.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && na && nb && x < y + nb && y < x + na;
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

bool dtype_ok(int32_t t) { return t == GDN_DTYPE_FP32 || t == GDN_DTYPE_BF16 || t == GDN_DTYPE_FP16; }
size_t dtype_size(int32_t t) { return t == GDN_DTYPE_FP32 ? 4 : 2; }

struct Span {
    const void *p;
    size_t bytes;
};
// any of outs[] on any of ins[] or on another of outs[]
bool any_overlap(const Span *outs, int no, const Span *ins, int ni)
{
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j)
            if (overlap(outs[i].p, outs[i].bytes, ins[j].p, ins[j].bytes)) return true;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return true;
    }
    return false;
}

// sizes of the paged attention; max_len: the longest sequence that its plan is made for
int attn_sizes(int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t page_size, int32_t max_pages,
               int32_t max_seqlen, int64_t *max_len)
{
    if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || page_size <= 0 || max_pages < 0 || max_seqlen < 0)
        return GDN_ERR_BAD_SHAPE;
    const int64_t capacity = (int64_t)page_size * max_pages;
    const int64_t tiles = (int64_t)Hkv * ((Hq / Hkv + 15) / 16);
    if ((D != 64 && D != 128 && D != 256) || capacity > (int64_t(1) << 30) || Hq > 65535 || tiles > 65535 ||
        B >= (1 << 30))
        return GDN_ERR_UNSUPPORTED;
    *max_len = max_seqlen > 0 ? std::min<int64_t>(max_seqlen, capacity) : capacity;
    return GDN_OK;
}

// workspace of a plan's CTAs: begun, part_ml, part (none where clusters finish what they begin)
size_t attn_bytes(const gdn::AttnPlan &plan, int32_t D)
{
    return (size_t)plan.ctas * (sizeof(int4) + 32 * sizeof(float2) + 32 * D * sizeof(float));
}

}  // namespace

extern "C" {

int gdn_rms_norm(const void *x, const void *residual, const void *gate, const void *weight, float eps,
                 float weight_offset, void *out, void *residual_out, float *scales, int64_t rows, int32_t width,
                 int32_t act_dtype, int32_t weight_dtype, int32_t quant, void *stream)
{
    if (rows < 0 || width <= 0 || !dtype_ok(act_dtype) || quant < GDN_QUANT_NONE || quant > GDN_QUANT_BLOCK)
        return GDN_ERR_BAD_SHAPE;
    if (weight_dtype != act_dtype && weight_dtype != GDN_DTYPE_FP32) return GDN_ERR_BAD_SHAPE;
    // (a warp's rows are numbered in 32 bits, those behind the last among them)
    if (width > GDN_NORM_MAX_WIDTH - (width % 8 ? 8 : 0) || rows > (int64_t(1) << 31) - 32) return GDN_ERR_UNSUPPORTED;
    if (rows == 0) return GDN_OK;
    if (!x || !weight || !out || (residual && !residual_out) || (quant != GDN_QUANT_NONE && !scales))
        return GDN_ERR_NULL_ARG;
    if ((!residual && residual_out) || (quant == GDN_QUANT_NONE && scales)) return GDN_ERR_BAD_SHAPE;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(gate, 16) || !aligned(weight, 16) ||
        !aligned(out, 16) || !aligned(residual_out, 16) || !aligned(scales, 4))
        return GDN_ERR_ALIGNMENT;
    const size_t n = (size_t)rows * width, matrix = n * dtype_size(act_dtype);
    const int groups = quant == GDN_QUANT_BLOCK ? (width + GDN_QUANT_GROUP - 1) / GDN_QUANT_GROUP : 1;
    const Span outs[3] = {{out, quant == GDN_QUANT_NONE ? matrix : n}, {residual_out, matrix},
                          {scales, (size_t)rows * groups * sizeof(float)}};
    const Span weights = {weight, width * dtype_size(weight_dtype)};
    // each lane reads its elements of x (of the residual) before it writes them to out (to residual_out)
    const bool on_x = out == x && quant == GDN_QUANT_NONE, on_residual = residual_out == residual;
    const Span for_out[4] = {{on_x ? nullptr : x, matrix}, {residual, matrix}, {gate, matrix}, weights};
    const Span for_residual[4] = {{x, matrix}, {on_residual ? nullptr : residual, matrix}, {gate, matrix}, weights};
    const Span for_scales[4] = {{x, matrix}, {residual, matrix}, {gate, matrix}, weights};
    if (any_overlap(outs, 1, for_out, 4) || any_overlap(outs + 1, 1, for_residual, 4) ||
        any_overlap(outs + 2, 1, for_scales, 4) || any_overlap(outs, 3, nullptr, 0))
        return GDN_ERR_OVERLAP;
    gdn::NormParams p;
    p.x = x, p.residual = residual, p.gate = gate, p.weight = weight;
    p.out = out, p.residual_out = residual_out, p.scales = scales;
    p.eps = eps, p.weight_offset = weight_offset, p.inv_width = 1.0f / (float)width;
    p.rows = rows, p.width = width, p.quant = quant, p.weight_f32 = weight_dtype == GDN_DTYPE_FP32;
    return cuda_status(gdn::launch_rms_norm(p, act_dtype, (cudaStream_t)stream));
}

int gdn_rope_fwd(const void *q, const void *k, const void *v, const int32_t *positions, const float *inv_freq,
                 const int32_t *slots, float mscale, void *q_out, void *k_out, void *k_cache, void *v_cache,
                 int64_t T, int32_t Hq, int32_t Hkv, int32_t D, int32_t rotary, int32_t interleaved,
                 int64_t cache_rows, int32_t act_dtype, void *stream)
{
    if (T < 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || rotary < 0 || rotary > D || rotary % 2 != 0 || cache_rows < 0 ||
        !dtype_ok(act_dtype))
        return GDN_ERR_BAD_SHAPE;
    if (D % 8 != 0 || D > GDN_ROPE_MAX_DIM || T >= (int64_t(1) << 31) || cache_rows >= (int64_t(1) << 31) ||
        Hq > 65535 || Hkv > 65535)
        return GDN_ERR_UNSUPPORTED;
    if (T == 0) return GDN_OK;
    if (!q || !k || !positions || (rotary > 0 && !inv_freq) || !q_out) return GDN_ERR_NULL_ARG;
    const bool cache = k_cache || v_cache;
    if (cache ? !k_cache || !v_cache || !v || !slots : !k_out) return GDN_ERR_NULL_ARG;
    if (!cache && (v || slots || cache_rows)) return GDN_ERR_BAD_SHAPE;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) ||
        !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(positions, 4) || !aligned(inv_freq, 4) ||
        !aligned(slots, 4))
        return GDN_ERR_ALIGNMENT;
    const size_t es = dtype_size(act_dtype), nq = (size_t)T * Hq * D * es, nk = (size_t)T * Hkv * D * es,
                 nc = (size_t)cache_rows * Hkv * D * es;
    const Span outs[4] = {{q_out, nq}, {k_out, nk}, {k_cache, nc}, {v_cache, nc}};
    // a thread reads its whole unit of a head before it writes it, so a head may be turned in place
    const Span ins[6] = {{q_out == q ? nullptr : q, nq}, {k_out == k ? nullptr : k, nk}, {v, nk},
                         {positions, (size_t)T * 4}, {inv_freq, (size_t)rotary * 2},
                         {slots, (size_t)T * 4}};
    if (any_overlap(outs, 4, ins, 6)) return GDN_ERR_OVERLAP;
    if ((q_out == q && (overlap(q, nq, k, nk) || overlap(q, nq, k_cache, nc) || overlap(q, nq, v_cache, nc))) ||
        (k_out && k_out == k && (overlap(k, nk, q, nq) || overlap(k, nk, k_cache, nc) || overlap(k, nk, v_cache, nc))))
        return GDN_ERR_OVERLAP;
    gdn::RopeParams p;
    p.q = q, p.k = k, p.v = v, p.positions = positions, p.slots = slots, p.inv_freq = inv_freq;
    p.q_out = q_out, p.k_out = k_out, p.k_cache = k_cache, p.v_cache = v_cache, p.mscale = mscale;
    p.T = T, p.cache_rows = cache_rows, p.Hq = Hq, p.Hkv = Hkv, p.D = D, p.n = rotary / 2;
    return cuda_status(gdn::launch_rope(p, act_dtype, interleaved != 0, (cudaStream_t)stream));
}

size_t gdn_paged_attn_workspace_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t page_size,
                                      int32_t max_pages, int32_t max_seqlen)
{
    int64_t max_len = 0;
    if (attn_sizes(B, Hq, Hkv, D, page_size, max_pages, max_seqlen, &max_len) || B == 0) return 0;
    return attn_bytes(gdn::attn_plan(B, Hq, Hkv, D, max_len), D);
}

int gdn_paged_attn_fwd(const void *q, const void *k_cache, const void *v_cache, const int32_t *block_table,
                       const int32_t *seq_lens, float scale, void *out, float *lse, int32_t B, int32_t Hq,
                       int32_t Hkv, int32_t D, int32_t P, int32_t page_size, int32_t max_pages, int32_t max_seqlen,
                       int32_t act_dtype, void *workspace, size_t workspace_bytes, void *stream)
{
    int64_t max_len = 0;
    int rc = attn_sizes(B, Hq, Hkv, D, page_size, max_pages, max_seqlen, &max_len);
    if (rc) return rc;
    if (P < 0 || !dtype_ok(act_dtype)) return GDN_ERR_BAD_SHAPE;
    const float log2e = 1.44269504f;
    if (!(scale <= 0.f) && !(scale * log2e <= FLT_MAX)) return GDN_ERR_BAD_SHAPE;  // NaN among them
    if (act_dtype == GDN_DTYPE_FP32 || (int64_t)P * page_size >= (int64_t(1) << 31)) return GDN_ERR_UNSUPPORTED;
    if (B == 0) return GDN_OK;
    const bool keys = P > 0 && max_pages > 0;
    if (!q || !seq_lens || !out || (keys && (!k_cache || !v_cache)) || (max_pages > 0 && !block_table))
        return GDN_ERR_NULL_ARG;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
        !aligned(workspace, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(lse, 4))
        return GDN_ERR_ALIGNMENT;
    const gdn::AttnPlan plan = gdn::attn_plan(B, Hq, Hkv, D, max_len);
    const size_t need = attn_bytes(plan, D);
    if (workspace && workspace_bytes < need) return GDN_ERR_WORKSPACE;
    const size_t nq = (size_t)B * Hq * D * 2, nc = (size_t)P * page_size * Hkv * D * 2;
    const Span outs[3] = {{out, nq}, {lse, (size_t)B * Hq * 4}, {workspace, need}};
    const Span ins[5] = {{q, nq}, {k_cache, nc}, {v_cache, nc}, {block_table, (size_t)B * max_pages * 4},
                         {seq_lens, (size_t)B * 4}};
    if (any_overlap(outs, 3, ins, 5)) return GDN_ERR_OVERLAP;
    const cudaStream_t st = (cudaStream_t)stream;
    void *own = nullptr;
    if (need && !workspace) {
        if (cudaMallocAsync(&own, need, st) != cudaSuccess) return GDN_ERR_CUDA;
        workspace = own;
    }
    gdn::AttnParams p;
    // (without a page nothing is read of the caches, but the copies of absent keys name a mapped address)
    p.q = q, p.k = P > 0 ? k_cache : q, p.v = P > 0 ? v_cache : q, p.table = block_table, p.lens = seq_lens, p.out = out, p.lse = lse;
    p.begun = static_cast<int4 *>(workspace);
    p.part_ml = reinterpret_cast<float2 *>(p.begun + plan.ctas);
    p.part = reinterpret_cast<float *>(p.part_ml + 32 * (size_t)plan.ctas);
    p.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf((float)D)) * log2e;
    p.B = B, p.Hq = Hq, p.Hkv = Hkv, p.group = Hq / Hkv, p.row_tiles = (Hq / Hkv + 15) / 16;
    p.P = P, p.page_size = page_size, p.max_pages = max_pages, p.ctas = plan.ctas, p.direct = plan.direct;
    p.capacity = (long long)page_size * max_pages;
    p.by_page = gdn::FastDiv((uint32_t)page_size);
    rc = cuda_status(gdn::launch_paged_attn(p, D, act_dtype == GDN_DTYPE_FP16, st));
    if (own && cudaFreeAsync(own, st) != cudaSuccess && rc == GDN_OK) rc = GDN_ERR_CUDA;
    return rc;
}

int gdn_testing_attn_split(const int32_t *lens, int32_t B, int32_t heads, int32_t D, int64_t capacity, int32_t ctas,
                           int32_t *pieces, int32_t max_pieces)
{
    if (!lens || !pieces || B <= 0 || heads <= 0 || ctas <= 0 || capacity < 0 || (D != 64 && D != 128 && D != 256))
        return -1;
    int64_t total = 0;
    for (int b = 0; b < B; ++b) total += (int64_t)gdn::attn_places(D, lens[b], capacity) * heads;
    const int parts = (int)std::min<int64_t>(total, ctas);
    int count = 0, b = 0, group = 0, u0 = 0;
    for (int i = 0; i < parts; ++i) {
        int64_t at = gdn::attn_part_begin(total, i, parts);
        const int64_t end = gdn::attn_part_begin(total, i + 1, parts);
        while (at < end) {
            const int all = gdn::attn_places(D, lens[b], capacity), n = gdn::attn_refused(lens[b], capacity) ? 0 : lens[b];
            const int take = (int)std::min<int64_t>(all - u0, end - at);
            if (count >= max_pieces) return -1;
            const gdn::KeyRange k = gdn::attn_keys(D, u0, take, n);
            int32_t *r = pieces + 7 * (int64_t)count++;
            r[0] = i, r[1] = b, r[2] = group, r[3] = k.k0, r[4] = k.k1;
            r[5] = take == all ? 2 : u0 == 0;
            r[6] = take < all && u0 == 0 ? gdn::attn_part_of(total, at + all - 1, parts) - i + 1 : 0;
            at += take, u0 += take;
            if (u0 == all) {
                u0 = 0;
                if (++group == heads) group = 0, ++b;
            }
        }
    }
    return count;
}

int gdn_testing_attn_cluster(int32_t n, int32_t cluster, int32_t rank, int32_t *k0, int32_t *k1)
{
    if (n < 0 || cluster <= 0 || rank < 0 || rank >= cluster || !k0 || !k1) return -1;
    const gdn::KeyRange k = gdn::attn_cluster_keys(rank, cluster, n);
    *k0 = k.k0, *k1 = k.k1;
    return 0;
}

int gdn_testing_attn_row(const int32_t *pages, int32_t j, int32_t page_size, int32_t P)
{
    if (!pages || j < 0 || page_size <= 0 || P < 0) return -2;
    return gdn::attn_cache_row(pages, j, gdn::FastDiv((uint32_t)page_size), page_size, P);
}

}  // extern "C"
