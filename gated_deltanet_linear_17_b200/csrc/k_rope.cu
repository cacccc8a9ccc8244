// Rotary positions of the queries and keys, and the write of the new keys and values into a paged
// cache (gdn_rope_fwd):
//
//   (a, b) -> mscale (a cos th - b sin th, b cos th + a sin th),  th = position * inv_freq[i]
//
// for the columns (i, n + i) of the first 2 n of a head, or (2 i, 2 i + 1) when interleaved.  Three
// multiplications an element against 4 bytes moved: HBM bounds it.  One launch does q, k, v and both
// cache writes, so every row is read once and written once, and the angles of a token are computed
// once for all its heads (into shared memory, then read by every row of the CTA's tokens).
//
// The angle.  position * inv_freq has up to 55 significant bits; fp32 would leave an error of
// position * 2^-24 radians.  It is formed in fp64 and reduced by k 2 pi with 2 pi in two parts, so the
// reduced angle is good to about 1e-15 * k before its rounding to fp32.
//
// Work is cut into units of 8 columns (16 when the unit is a pair of 8-column runs, as in the half
// layout): a thread reads its whole unit before it writes it, so q_out may be q.
#include "gdn_layers.h"
#include "layers.cuh"

namespace gdn {

namespace {

constexpr int kRopeThreads = 256;

// sin and cos of position * f, f fp32
__device__ __forceinline__ float2 turn(int position, float f, float mscale)
{
    constexpr double kTwoPiHi = 6.283185307179586, kTwoPiLo = 2.4492935982947064e-16, kInv = 0.15915494309189535;
    const double x = (double)position * (double)f;
    const double k = rint(x * kInv);
    const double r = fma(-k, kTwoPiLo, fma(-k, kTwoPiHi, x));
    float s, c;
    sincosf((float)r, &s, &c);
    return make_float2(c * mscale, s * mscale);
}

template <class A>
__device__ __forceinline__ void turn8(float (&a)[8], float (&b)[8], const float2 *cs)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float c = cs[j].x, s = cs[j].y, x = a[j], y = b[j];
        a[j] = x * c - y * s;
        b[j] = y * c + x * s;
    }
}

// one unit of a turned head (row: its D elements): u counts the head's units
template <class A, bool INTERLEAVED>
__device__ __forceinline__ void turn_unit(const typename A::raw *src, typename A::raw *dst, typename A::raw *dst2,
                                          int u, int n, int D, const float2 *cs)
{
    using raw = typename A::raw;
    if (INTERLEAVED) {
        const int c = 8 * u;
        Raw8<A> r;
        r.load(src + c);
        if (c < 2 * n) {
            float x[8];
            r.up(x);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (c / 2 + j >= n) break;
                const float2 t = cs[c / 2 + j];
                const float a = x[2 * j], b = x[2 * j + 1];
                x[2 * j] = a * t.x - b * t.y;
                x[2 * j + 1] = b * t.x + a * t.y;
            }
            r.down(x);
        }
        if (dst) r.store(dst + c);
        if (dst2) r.store(dst2 + c);
        return;
    }
    const int pairs = (n + 7) >> 3;
    if (u < pairs) {
        const int i = 8 * u;
        if ((n & 7) == 0) {
            Raw8<A> ra, rb;
            ra.load(src + i);
            rb.load(src + n + i);
            float a[8], b[8];
            ra.up(a);
            rb.up(b);
            turn8<A>(a, b, cs + i);
            ra.down(a);
            rb.down(b);
            if (dst) ra.store(dst + i), rb.store(dst + n + i);
            if (dst2) ra.store(dst2 + i), rb.store(dst2 + n + i);
        } else {
            const int m = min(8, n - i);
            for (int j = 0; j < m; ++j) {
                const float a = A::up(src[i + j]), b = A::up(src[n + i + j]);
                const float2 t = cs[i + j];
                const raw x = A::down(a * t.x - b * t.y), y = A::down(b * t.x + a * t.y);
                if (dst) dst[i + j] = x, dst[n + i + j] = y;
                if (dst2) dst2[i + j] = x, dst2[n + i + j] = y;
            }
        }
        return;
    }
    // the columns that pass unchanged, from 2 n on: 8-column runs of the head, the first perhaps partial
    const int c0 = max(2 * n, 8 * ((2 * n >> 3) + u - pairs)), c1 = 8 * ((2 * n >> 3) + u - pairs + 1);
    if (c1 - c0 == 8) {
        Raw8<A> r;
        r.load(src + c0);
        if (dst && dst != src) r.store(dst + c0);
        if (dst2) r.store(dst2 + c0);
    } else {
        for (int c = c0; c < c1; ++c) {
            const raw x = src[c];
            if (dst) dst[c] = x;
            if (dst2) dst2[c] = x;
        }
    }
}

template <class A, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p)
{
    using raw = typename A::raw;
    extern __shared__ float2 cs[];  // [tokens_per_cta][n]
    const long long t0 = (long long)blockIdx.x * p.tokens_per_cta;
    const int tokens = (int)min((long long)p.tokens_per_cta, p.T - t0);
    for (int i = threadIdx.x; i < tokens * p.n; i += kRopeThreads) {
        const int t = i / p.n;
        cs[i] = turn(p.positions[t0 + t], p.inv_freq[i - t * p.n], p.mscale);
    }
    __syncthreads();
    const int total = tokens * p.token_units;
    const int q_units = p.Hq * p.head_units, k_units = p.Hkv * p.head_units;
    for (int i = threadIdx.x; i < total; i += kRopeThreads) {
        const int tt = (int)fast_div(i, p.by_token);
        int r = i - tt * p.token_units;
        const long long t = t0 + tt;
        const float2 *angles = cs + tt * p.n;
        if (r < q_units) {
            const int h = (int)fast_div(r, p.by_head);
            const long long at = (t * p.Hq + h) * p.D;
            turn_unit<A, INTERLEAVED>(static_cast<const raw *>(p.q) + at, static_cast<raw *>(p.q_out) + at, nullptr,
                                      r - h * p.head_units, p.n, p.D, angles);
            continue;
        }
        r -= q_units;
        long long slot = -1;
        if (p.slots) {
            slot = p.slots[t];
            if (slot >= p.cache_rows) slot = -1;
        }
        if (r < k_units) {
            const int h = (int)fast_div(r, p.by_head);
            const long long at = (t * p.Hkv + h) * p.D;
            raw *out = p.k_out ? static_cast<raw *>(p.k_out) + at : nullptr;
            raw *row = slot >= 0 ? static_cast<raw *>(p.k_cache) + (slot * p.Hkv + h) * p.D : nullptr;
            if (out || row)
                turn_unit<A, INTERLEAVED>(static_cast<const raw *>(p.k) + at, out, row, r - h * p.head_units, p.n,
                                          p.D, angles);
            continue;
        }
        r -= k_units;
        if (slot < 0) continue;
        Raw8<A> x;
        x.load(static_cast<const raw *>(p.v) + t * p.Hkv * p.D + 8 * r);
        x.store(static_cast<raw *>(p.v_cache) + slot * p.Hkv * p.D + 8 * r);
    }
}

template <class A>
cudaError_t launch_type(const RopeParams &p, bool interleaved, cudaStream_t st)
{
    const unsigned grid = (unsigned)((p.T + p.tokens_per_cta - 1) / p.tokens_per_cta);
    const size_t smem = sizeof(float2) * p.tokens_per_cta * p.n;
    if (interleaved) rope_kernel<A, true><<<grid, kRopeThreads, smem, st>>>(p);
    else rope_kernel<A, false><<<grid, kRopeThreads, smem, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeParams &in, int act_dtype, bool interleaved, cudaStream_t st)
{
    RopeParams p = in;
    p.head_units = interleaved ? p.D / 8 : (p.n + 7) / 8 + p.D / 8 - (2 * p.n >> 3);
    const int copied = p.k_cache ? p.Hkv * p.D / 8 : 0;
    p.token_units = (p.Hq + p.Hkv) * p.head_units + copied;
    // about four units a thread; the angles of a CTA's tokens stay within 16 KB of shared memory
    long long tokens = 4 * kRopeThreads / p.token_units;
    const long long most = p.n ? 16384 / (8 * p.n) : tokens;
    tokens = tokens < 1 ? 1 : tokens > most ? most : tokens;
    p.tokens_per_cta = (int)(tokens > p.T ? p.T : tokens);
    p.by_token = FastDiv(p.token_units);
    p.by_head = FastDiv(p.head_units);
    switch (act_dtype) {
    case GDN_DTYPE_BF16: return launch_type<Bf16>(p, interleaved, st);
    case GDN_DTYPE_FP16: return launch_type<F16>(p, interleaved, st);
    default: return launch_type<F32>(p, interleaved, st);
    }
}

}  // namespace gdn
