// Declarations shared by the host entries of gdn_layers.h and their kernels.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

// n / d for 0 <= n < 2^31 by one 32 x 32 -> 64 multiplication.  With s = ceil(log2 d) - 1 and
// mul = ceil(2^(32 + s) / d) < 2^32 + 1, the error n (mul d - 2^(32 + s)) / (d 2^(32 + s)) is below
// n / 2^(32 + s) <= 2^31 / 2^(32 + s) = 1 / 2^(s + 1) <= 1 / d, so the floor is exact.  A power of two
// d = 2^(s + 1) has mul = 2^31; d = 1 passes n through (shift < 0).
struct FastDiv {
    uint32_t mul;
    int32_t shift;
    FastDiv() : mul(0), shift(-1) {}
    explicit FastDiv(uint32_t d) : mul(0), shift(-1)
    {
        if (d <= 1) return;
        int s = 0;
        while ((1ull << (s + 1)) < d) ++s;  // 2^s < d <= 2^(s + 1)
        shift = s;
        mul = (uint32_t)(((1ull << (32 + s)) + d - 1) / d);
    }
};

__host__ __device__ inline uint32_t fast_div(uint32_t n, FastDiv d)
{
    return d.shift < 0 ? n : (uint32_t)(((uint64_t)n * d.mul) >> 32 >> d.shift);
}

struct NormParams {
    const void *x, *residual, *gate, *weight;
    void *out, *residual_out;
    float *scales;
    float eps, weight_offset, inv_width;
    long long rows;
    int width;
    int quant;        // GDN_QUANT_*
    bool weight_f32;
    bool two_stages;  // of a row in shared memory (set by the launcher)
};
cudaError_t launch_rms_norm(const NormParams &p, int act_dtype, cudaStream_t st);

struct RopeParams {
    const void *q, *k, *v;
    const int32_t *positions, *slots;
    const float *inv_freq;
    void *q_out, *k_out, *k_cache, *v_cache;
    float mscale;
    long long T, cache_rows;
    int Hq, Hkv, D, n;  // n = rotary / 2 angles
    int split;          // warps that share a token (set by the launcher)
};
cudaError_t launch_rope(const RopeParams &p, int act_dtype, bool interleaved, cudaStream_t st);

constexpr int kAttnUnit = 64, kAttnSms = 148, kAttnMaxCluster = 8;
constexpr int kAttnCtasPerSm = 2;
constexpr int kDirectCtasPerSm(int D) { return D == 256 ? 1 : 2; }
constexpr int kAttnMaxCtas = kAttnSms * kAttnCtasPerSm;
// The paged attention's grid, by the sizes and the longest sequence that the caller expects; any is right for any
// lengths.  direct: CTAs of the cluster that takes a pair of a sequence and a head group, or 0; then ctas fill
// the GPU once (fewer where there is one for each kAttnUnit keys) and share all pairs evenly.
struct AttnPlan {
    int ctas, direct;
};
AttnPlan attn_plan(int B, int Hq, int Hkv, int D, long long max_len);

// The list that the pairs of a sequence and a head group are cut by: one place for each kAttnUnit keys of a pair,
// behind attn_lead places that stand for what a pair costs beside its keys (its queries, the first page's latency,
// its output), so that a CTA of many short pairs gets no more work than one of a long pair.  Measured with 2, 3 and
// 4 leading places at D = 64: 64 sequences of 8 heads of up to 2000 keys 34.0, 31.9, 32.1 us.
__host__ __device__ constexpr int attn_lead(int D) { return D == 64 ? 3 : D == 128 ? 2 : 1; }
// a length outside the table's capacity stands for the whole sequence being refused
__host__ __device__ inline bool attn_refused(int n, long long capacity) { return n < 0 || n > capacity; }
__host__ __device__ inline int attn_places(int D, int n, long long capacity)
{
    return attn_lead(D) + (attn_refused(n, capacity) ? 0 : (n + kAttnUnit - 1) / kAttnUnit);
}
// the keys of places [u0, u0 + take) of a pair of n keys
struct KeyRange {
    int k0, k1;
};
__host__ __device__ inline KeyRange attn_keys(int D, int u0, int take, int n)
{
    const int a = u0 - attn_lead(D), b = a + take;
    const int k1 = b > 0 ? b * kAttnUnit : 0;
    return KeyRange{a > 0 ? a * kAttnUnit : 0, k1 < n ? k1 : n};
}
// Part i of n equal ones of the list begins at i total / n, rounded down; place u lies in the last part that begins
// at or before it.  64-bit divisions take a microsecond of a CTA's start between them; lists of up to 2^22 places
// do without.
__host__ __device__ inline long long attn_part_begin(long long total, int i, int n)
{
    return total < (1 << 22) ? (long long)((uint32_t)total * (uint32_t)i / (uint32_t)n) : total * i / n;
}
__host__ __device__ inline int attn_part_of(long long total, long long u, int n)
{
    return total < (1 << 22) ? (int)((((uint32_t)u + 1) * (uint32_t)n - 1) / (uint32_t)total)
                             : (int)(((u + 1) * n - 1) / total);
}
// the keys that CTA `rank` of a cluster takes of n
__host__ __device__ inline KeyRange attn_cluster_keys(int rank, int cluster, int n)
{
    const int each = (n / cluster + 16) & ~15;  // above n / cluster
    const long long k0 = (long long)rank * each;
    return KeyRange{(int)(k0 < n ? k0 : n), (int)(k0 + each < n ? k0 + each : n)};
}
// cache row of key j of a sequence whose pages `table` lists; -1 on a page outside the cache's P
__host__ __device__ inline int attn_cache_row(const int32_t *table, int j, FastDiv by_page, int page_size, int P)
{
    const int nth = (int)fast_div((uint32_t)j, by_page), page = table[nth];
    return (uint32_t)page < (uint32_t)P ? page * page_size + (j - nth * page_size) : -1;
}

struct AttnParams {
    const void *q, *k, *v;
    const int32_t *table, *lens;
    void *out;
    float *lse;
    int4 *begun;      // [ctas]: sequence, first query head, query heads and pieces of the pair that a CTA began and
                      // did not finish (pieces 0: none)
    float2 *part_ml;  // [ctas][2][16]: a piece's maximum (unscaled) and sum of exponentials
    float *part;      // [ctas][2][16][D]: its unnormalised sum
    float scale_log2;
    int B, Hq, Hkv, group, row_tiles, P, page_size, max_pages, ctas, direct;
    long long capacity;  // page_size * max_pages
    FastDiv by_page;
};
cudaError_t launch_paged_attn(const AttnParams &p, int D, bool f16, cudaStream_t st);

}  // namespace gdn
