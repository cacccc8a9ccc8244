// Attention of one new token of each sequence over a paged key/value cache (gdn_paged_attn_fwd):
//
//   s_j = scale q . k_j,  out = sum_j e^{s_j} v_j / sum_j e^{s_j},  lse = log sum_j e^{s_j}
//
// Every key and value is read once from HBM and used by the G = Hq / Hkv query heads of its head:
// G flops a byte of a 16-bit cache, so up to G of about 250 the cache's bytes bound it, and the matrix
// products (mma.sync: 16 query rows, zero-padded, against 8 keys or columns) only have to keep up.
//
// The split.  A CTA takes one piece of one sequence's keys for one key/value head and up to 16 of its
// query heads; its four warps take every fourth tile of 16 keys.  A warp is on its own until the end
// of the piece: its own ring of tiles in shared memory, filled by cp.async a few tiles ahead, its own
// running maximum, sum and output accumulators (fp32, in registers), no CTA barrier.  At the end the
// four partial results are joined through shared memory.  A sequence in one piece is then done;
// otherwise the piece's unnormalised sum, maximum and sum of exponentials go to the workspace, and a
// second kernel (started early by a programmatic dependency) joins the pieces in their order, so that
// the result does not depend on the order in which CTAs run.
//
// Roundings.  Scores, exponentials (base 2, the scale folded in), sums and outputs are fp32.  The
// probabilities enter their product with V as a pair of 16-bit numbers, p = hi + lo (16 bits or more of
// p in bf16, 22 in fp16): one rounded number would put an error as large as the output's own rounding
// into it, and the second product costs nothing beside the memory traffic.  The sum of exponentials
// takes them unrounded, so lse is good to fp32.
#include <algorithm>

#include "gdn_layers.h"
#include "layers.cuh"

namespace gdn {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kTile = 16;  // keys a warp takes at a time
constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;

template <int D>
struct Shape {
    static constexpr int kStages = D == 256 ? 3 : 4;
    static constexpr int kHalf = kTile * D * 2;      // bytes of a tile's keys (or values)
    static constexpr int kStage = 2 * kHalf;
    static constexpr int kRing = kStages * kStage;   // per warp
    static constexpr int kQ = 16 * D * 2;            // query rows, behind the rings
    static constexpr int kSmem = kWarps * kRing + kQ;
    static constexpr int kCtas = D == 256 ? 1 : D == 128 ? 1 : 2;
    static_assert(kWarps * kRing >= kWarps * 16 * D * 4, "the join of the warps fits into the rings");
};

// byte offset of 16-byte chunk c of row r in a tile of D-element rows: eight rows at one chunk lie in
// eight different bank groups
template <int D>
__device__ __forceinline__ uint32_t sw(int r, int c)
{
    return r * (D * 2) + ((c ^ (r & 7)) << 4);
}

template <bool F16>
__device__ __forceinline__ void mma(float *d, const uint32_t *a, uint32_t b0, uint32_t b1)
{
    if (F16) mma16816(d, a, b0, b1);
    else mma16816_bf16(d, a, b0, b1);
}

__device__ __forceinline__ float quad_max(float x)
{
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x)
{
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// the pieces of a sequence of n keys: keys a piece, and pieces (1 for n = 0)
__device__ __forceinline__ int2 pieces(int n, const AttnPlan &plan)
{
    const int least = ((n + plan.splits - 1) / plan.splits + 63) & ~63;
    const int chunk = max(plan.chunk, least);
    return make_int2(chunk, max(1, (n + chunk - 1) / chunk));
}
// a length outside the table's range stands for the whole sequence being refused
__device__ __forceinline__ bool bad_length(int n, const AttnParams &p)
{
    return n < 0 || n > (long long)p.max_pages * p.page_size;
}

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, Shape<D>::kCtas) paged_attn_kernel(const AttnParams p)
{
    using S = Shape<D>;
    extern __shared__ __align__(128) uint8_t smem[];
    asm volatile("griddepcontrol.launch_dependents;");
    const int b = (int)fast_div(blockIdx.x, p.by_splits), piece = blockIdx.x - b * p.plan.splits;
    const int hkv = blockIdx.y / p.row_tiles, tile_row0 = (blockIdx.y - hkv * p.row_tiles) * 16;
    const int rows = min(16, p.group - tile_row0);
    const int head0 = hkv * p.group + tile_row0;  // first query head of this CTA
    const int n_raw = p.lens[b];
    const bool bad = bad_length(n_raw, p);
    const int n = bad ? 0 : n_raw;
    const int2 pc = pieces(n, p.plan);
    if (piece >= pc.y) return;
    const int k0 = piece * pc.x, k1 = min(n, k0 + pc.x);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t ring = smem_addr(smem) + warp * S::kRing;
    const uint32_t qs = smem_addr(smem) + kWarps * S::kRing;
    const uint16_t *kc = static_cast<const uint16_t *>(p.k), *vc = static_cast<const uint16_t *>(p.v);

    // query rows to shared memory (rows past the group's zero)
    for (int i = tid; i < 16 * (D / 8); i += kThreads) {
        const int r = i / (D / 8), c = i % (D / 8);
        uint4 x = make_uint4(0, 0, 0, 0);
        if (r < rows)
            x = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) +
                                                ((long long)b * p.Hq + head0 + r) * D)[c];
        *reinterpret_cast<uint4 *>(smem + kWarps * S::kRing + sw<D>(r, c)) = x;
    }
    __syncthreads();

    // this warp's tiles: first + 16 (warp + 4 i)
    const int tiles = (k1 - k0 + kTile - 1) / kTile;
    const int mine = tiles > warp ? (tiles - warp + kWarps - 1) / kWarps : 0;
    const int32_t *table = p.table + (long long)b * p.max_pages;
    bool bad_page = false;
    // cache row of key (lane & 15) of tile i; -1 past the piece or on a page outside the cache
    auto cache_row = [&](int i) {
        const int j = k0 + kTile * (warp + kWarps * i) + (lane & 15);
        if (i >= mine || j >= k1) return -1;
        const int pg = (int)fast_div(j, p.by_page), page = table[pg];
        if ((unsigned)page >= (unsigned)p.P) {
            bad_page = true;
            return -1;
        }
        return page * p.page_size + (j - pg * p.page_size);
    };
    auto fetch = [&](int stage, int row) {
        const uint32_t dst = ring + stage * S::kStage;
#pragma unroll
        for (int i = 0; i < kTile * (D / 8) / 32; ++i) {
            const int id = lane + 32 * i, r = id / (D / 8), c = id % (D / 8);
            const int rr = __shfl_sync(0xffffffffu, row, r);
            const long long at = rr < 0 ? 0 : ((long long)rr * p.Hkv + hkv) * D + 8 * c;
            cp_async16(dst + sw<D>(r, c), kc + at, rr >= 0);
            cp_async16(dst + S::kHalf + sw<D>(r, c), vc + at, rr >= 0);
        }
    };

    float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    uint32_t qf[D < 256 ? D / 16 : 1][4];
    if (D < 256) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
            ldsm_x4(qs + sw<D>(lane & 15, 2 * k + (lane >> 4)), qf[k][0], qf[k][1], qf[k][2], qf[k][3]);
    }

#pragma unroll
    for (int i = 0; i < S::kStages - 1; ++i) {
        if (i < mine) fetch(i, cache_row(i));
        cp_async_commit();
    }
    int next_row = cache_row(S::kStages - 1);
    int stage = 0;
    for (int i = 0; i < mine; ++i) {
        cp_async_wait<S::kStages - 2>();
        __syncwarp();
        {
            const int ahead = i + S::kStages - 1;
            if (ahead < mine) fetch(stage == 0 ? S::kStages - 1 : stage - 1, next_row);
            cp_async_commit();
            next_row = cache_row(ahead + 1);
        }
        const uint32_t ks = ring + stage * S::kStage, vs = ks + S::kHalf;
        stage = stage + 1 == S::kStages ? 0 : stage + 1;

        // scores of 16 rows x 16 keys
        float s[2][4] = {};
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            uint32_t b0, b1, b2, b3, a[4];
            ldsm_x4(ks + sw<D>((lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)), b0, b1, b2, b3);
            if (D < 256) {
                mma<F16>(s[0], qf[k], b0, b1);
                mma<F16>(s[1], qf[k], b2, b3);
            } else {
                ldsm_x4(qs + sw<D>(lane & 15, 2 * k + (lane >> 4)), a[0], a[1], a[2], a[3]);
                mma<F16>(s[0], a, b0, b1);
                mma<F16>(s[1], a, b2, b3);
            }
        }
        const int left = k1 - (k0 + kTile * (warp + kWarps * i));  // keys of this tile (1 .. 16, or more)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int key = 8 * t + 2 * (lane & 3) + (e & 1);
                s[t][e] = key < left ? s[t][e] * p.scale_log2 : -INFINITY;
            }
        float alpha[2], ref[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float top =
                quad_max(fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1])));
            const float now = fmaxf(m[r], top);
            ref[r] = now == -INFINITY ? 0.f : now;  // every score -infinity so far: the exponentials are 0
            alpha[r] = exp2f(m[r] - ref[r]);
            m[r] = now;
            l[r] *= alpha[r];
        }
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
            for (int t = 0; t < D / 8; ++t) {
                o[t][0] *= alpha[0];
                o[t][1] *= alpha[0];
                o[t][2] *= alpha[1];
                o[t][3] *= alpha[1];
            }
        }
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float p0 = exp2f(s[t][2 * r] - ref[r]), p1 = exp2f(s[t][2 * r + 1] - ref[r]);
                l[r] += p0 + p1;
                split2<F16>(p0, p1, hi[2 * t + r], lo[2 * t + r]);
            }
#pragma unroll
        for (int t = 0; t < D / 16; ++t) {
            uint32_t b0, b1, b2, b3;
            ldsm_x4_t(vs + sw<D>((lane & 7) + (((lane >> 3) & 1) << 3), 2 * t + (lane >> 4)), b0, b1, b2, b3);
            mma<F16>(o[2 * t], hi, b0, b1);
            mma<F16>(o[2 * t + 1], hi, b2, b3);
            mma<F16>(o[2 * t], lo, b0, b1);
            mma<F16>(o[2 * t + 1], lo, b2, b3);
        }
    }
    cp_async_wait<0>();
    if (__any_sync(0xffffffffu, bad_page)) l[0] = l[1] = NAN;
    if (bad) l[0] = l[1] = NAN;

    // join the four warps
    __shared__ float wm[kWarps][16], wl[kWarps][16];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] = quad_sum(l[r]);
        if ((lane & 3) == 0) {
            wm[warp][lane / 4 + 8 * r] = m[r];
            wl[warp][lane / 4 + 8 * r] = l[r];
        }
    }
    __syncthreads();  // every warp is done with its ring
    float *os = reinterpret_cast<float *>(smem);
    float f[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = lane / 4 + 8 * r;
        const float top = fmaxf(fmaxf(wm[0][row], wm[1][row]), fmaxf(wm[2][row], wm[3][row]));
        f[r] = exp2f(m[r] - (top == -INFINITY ? 0.f : top));
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = lane / 4 + 8 * r;
        if (row >= rows) continue;
#pragma unroll
        for (int t = 0; t < D / 8; ++t)
            *reinterpret_cast<float2 *>(os + (warp * 16 + row) * D + 8 * t + 2 * (lane & 3)) =
                make_float2(o[t][2 * r] * f[r], o[t][2 * r + 1] * f[r]);
    }
    __syncthreads();
    for (int i = tid; i < rows * (D / 4); i += kThreads) {
        const int row = i / (D / 4), c = i % (D / 4);
        const float top = fmaxf(fmaxf(wm[0][row], wm[1][row]), fmaxf(wm[2][row], wm[3][row]));
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float4 y = reinterpret_cast<const float4 *>(os + (w * 16 + row) * D)[c];
            x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
            sum += wl[w][row] * exp2f(wm[w][row] - (top == -INFINITY ? 0.f : top));
        }
        const int head = head0 + row;
        if (pc.y == 1) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            uint16_t *out = static_cast<uint16_t *>(p.out) + ((long long)b * p.Hq + head) * D + 4 * c;
            *reinterpret_cast<uint2 *>(out) =
                make_uint2(pack2<F16>(x.x * inv, x.y * inv), pack2<F16>(x.z * inv, x.w * inv));
            if (p.lse && c == 0) p.lse[(long long)b * p.Hq + head] = sum == 0.f ? -INFINITY : kLn2 * (top + log2f(sum));
        } else {
            const long long at = ((long long)b * p.plan.splits + piece) * p.Hq + head;
            reinterpret_cast<float4 *>(p.part + at * D)[c] = x;
            if (c == 0) p.part_ml[at] = make_float2(top, sum);
        }
    }
}

// joins the pieces of one (sequence, query head); nothing to do where the sequence was one piece
template <int D, bool F16>
__global__ void __launch_bounds__(128) paged_attn_join_kernel(const AttnParams p)
{
    constexpr int kCols = D / 4, kGroups = 128 / kCols;  // threads along the columns, groups along the pieces
    __shared__ float weight[GDN_ATTN_MAX_SPLITS];
    __shared__ float red[2][4];
    __shared__ float4 part[kGroups][kCols];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int b = blockIdx.x, head = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
    const int n = p.lens[b];
    if (bad_length(n, p)) return;
    const int count = pieces(n, p.plan).y;
    if (count == 1) return;
    const long long at0 = (long long)b * p.plan.splits * p.Hq + head;
    float top = -INFINITY;
    for (int s = tid; s < count; s += 128) top = fmaxf(top, p.part_ml[at0 + (long long)s * p.Hq].x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    if (lane == 0) red[0][tid >> 5] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    float sum = 0.f;
    for (int s = tid; s < count; s += 128) {
        const float2 ml = p.part_ml[at0 + (long long)s * p.Hq];
        const float w = exp2f(ml.x - (top == -INFINITY ? 0.f : top));
        weight[s] = w;
        sum += w * ml.y;
    }
    sum = warp_sum(sum);
    if (lane == 0) red[1][tid >> 5] = sum;
    __syncthreads();
    sum = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
    const int c = tid % kCols, g = tid / kCols;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = g; s < count; s += kGroups) {
        const float4 y = reinterpret_cast<const float4 *>(p.part + (at0 + (long long)s * p.Hq) * D)[c];
        const float w = weight[s];
        x.x = fmaf(w, y.x, x.x), x.y = fmaf(w, y.y, x.y), x.z = fmaf(w, y.z, x.z), x.w = fmaf(w, y.w, x.w);
    }
    part[g][c] = x;
    __syncthreads();
    if (g != 0) return;
#pragma unroll
    for (int i = 1; i < kGroups; ++i) {
        const float4 y = part[i][c];
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint16_t *out = static_cast<uint16_t *>(p.out) + ((long long)b * p.Hq + head) * D + 4 * c;
    *reinterpret_cast<uint2 *>(out) = make_uint2(pack2<F16>(x.x * inv, x.y * inv), pack2<F16>(x.z * inv, x.w * inv));
    if (p.lse && c == 0) p.lse[(long long)b * p.Hq + head] = sum == 0.f ? -INFINITY : kLn2 * (top + log2f(sum));
}

template <int D, bool F16>
cudaError_t launch(const AttnParams &p, cudaStream_t st)
{
    using S = Shape<D>;
    const auto kern = paged_attn_kernel<D, F16>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)p.B * p.plan.splits, (unsigned)p.Hkv * p.row_tiles);
    kern<<<grid, kThreads, S::kSmem, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess || p.plan.splits == 1) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.B, (unsigned)p.Hq);
    cfg.blockDim = dim3(128);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_attn_join_kernel<D, F16>, p);
}

}  // namespace

AttnPlan attn_plan(int B, int Hq, int Hkv, int D, long long max_len)
{
    const long long rows = (Hq / Hkv + 15) / 16;
    const long long pairs = (long long)B * Hkv * rows, slots = 148 * (D == 64 ? 2 : 1);
    long long chunk = (max_len * pairs + slots - 1) / slots;
    if (pairs >= slots / 2) chunk = max_len * pairs / (8 * slots);
    chunk = std::max(chunk, 256LL);
    chunk = std::max(chunk, (max_len + GDN_ATTN_MAX_SPLITS - 1) / GDN_ATTN_MAX_SPLITS);
    chunk = (chunk + 63) / 64 * 64;
    const long long splits = std::max(1LL, (max_len + chunk - 1) / chunk);
    return AttnPlan{(int)splits, (int)chunk};
}

cudaError_t launch_paged_attn(const AttnParams &p, int D, bool f16, cudaStream_t st)
{
    switch (D) {
    case 64: return f16 ? launch<64, true>(p, st) : launch<64, false>(p, st);
    case 128: return f16 ? launch<128, true>(p, st) : launch<128, false>(p, st);
    default: return f16 ? launch<256, true>(p, st) : launch<256, false>(p, st);
    }
}

}  // namespace gdn
