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

struct NormParams {
    const void *x, *residual, *gate, *weight;
    void *out, *residual_out;
    float *scales;
    float eps, weight_offset, inv_width;
    long long rows;
    int width;
    int quant;        // GDN_QUANT_*
    bool weight_f32;
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
constexpr int kAttnCtasPerSm(int D) { return D == 64 ? 3 : 2; }
constexpr int kDirectCtasPerSm(int D) { return D == 64 ? 3 : D == 128 ? 2 : 1; }
constexpr int kAttnMaxCtas = kAttnSms * 3;
// The paged attention's grid, by the sizes and the longest sequence that the caller expects; any is right for any
// lengths.  direct: CTAs of the cluster that takes a pair of a sequence and a head group, or 0; then ctas fill
// the GPU once (fewer where there is one for each kAttnUnit keys) and share all pairs evenly.
struct AttnPlan {
    int ctas, direct;
};
AttnPlan attn_plan(int B, int Hq, int Hkv, int D, long long max_len);

struct AttnParams {
    const void *q, *k, *v;
    const int32_t *table, *lens;
    void *out;
    float *lse;
    int4 *begun;      // [ctas]: sequence, first query head, query heads and pieces of the pair that a CTA began and
                      // did not finish (pieces 0: none)
    float2 *part_ml;  // [ctas][2][16]: a piece's maximum (base 2) and sum of exponentials
    float *part;      // [ctas][2][16][D]: its unnormalised sum
    float scale_log2;
    int B, Hq, Hkv, group, row_tiles, P, page_size, max_pages, ctas, direct;
    FastDiv by_page;
};
cudaError_t launch_paged_attn(const AttnParams &p, int D, bool f16, cudaStream_t st);

}  // namespace gdn
