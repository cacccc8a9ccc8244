// Rotary positions of the queries and keys, and the write of the new keys and values into a paged
// cache (gdn_rope_fwd):
//
//   (a, b) -> mscale (a cos th - b sin th, b cos th + a sin th),  th = position * inv_freq[i]
//
// for the columns (i, n + i) of the first 2 n of a head, or (2 i, 2 i + 1) when interleaved.  Three
// multiplications an element against 4 bytes moved: HBM bounds it.  One launch does q, k, v and both
// cache writes, so every row is read once and written once, and the angles of a token are computed
// once for all its heads.
//
// The angle.  position * inv_freq has up to 55 significant bits; fp32 would leave an error of
// position * 2^-24 radians.  It is formed in fp64 and reduced by k 2 pi with 2 pi in two parts, so the
// reduced angle is good to about 1e-15 * k.  For 16-bit activations it is rounded to fp32 (2^-23 at most), and the fast
// sine and cosine are then within 2^-21 of the exact ones, below a sixteenth of fp16's rounding of a turned element.  fp32
// activations would lose three bits by that: theirs are good to 2^-24 (turn_fp32; 32768 tokens of 16 + 2 heads of 256 202 us
// as with the fast ones, 100000 tokens of 1 + 1 heads of 64, which share no angles, 35 against 31; with sincos in fp64 42).
//
// Layout.  A lane holds 8 neighbouring columns, a row (one head of q, k or v) lies in D / 8 lanes of one
// warp, and a lane keeps its columns for all rows of its token: its cosines and signed sines, eight of each,
// stay in registers, y_j = x_j c_j + partner_j s_j.  The partner of a column lies in the same lane
// (interleaved), in the lane n / 8 away (shuffles), or, when n is no multiple of 8, across two lanes (read
// again, from L1).  A warp takes as many tokens as it has room for rows, and reads up to four heads ahead of its
// work on them; where there are few tokens, several warps share their heads.
//
// Measured (bf16, 32768 tokens of 16 + 2 heads of 256 with the cache's write): 106 us, 6.3 TB/s, 98 % of the copy
// rate; with the factors read from shared memory for every head 198 us.  4099 tokens of 32 + 8 heads of 128, pairs,
// fp16: 15.2 us, 5.5 TB/s, of it 2.5 the kernel's start and end.  64 tokens: 2.8 us.
#include <algorithm>

#include "gdn_layers.h"
#include "layers.cuh"

namespace gdn {

namespace {

// 4 warps: with 8 a CTA 2 to 3 % slower at 4000 tokens and more, at the start and end of the grid
constexpr int kRopeThreads = 128, kRopeWarps = kRopeThreads / 32, kAhead = 4;
enum Layout { kPairs, kHalves, kHalvesUnaligned };

// mscale times the cosine and sine of position * f
__device__ __forceinline__ float2 turn(int position, float f, float mscale)
{
    constexpr double kTwoPiHi = 6.283185307179586, kTwoPiLo = 2.4492935982947064e-16, kInv = 0.15915494309189535;
    const double x = (double)position * (double)f;
    const double k = rint(x * kInv);
    const float r = (float)fma(-k, kTwoPiLo, fma(-k, kTwoPiHi, x));
    return make_float2(__cosf(r) * mscale, __sinf(r) * mscale);
}

// The same to fp32's rounding.  The angle is reduced to |r| <= pi/4 by k quarters of a turn; with r = hi + lo in fp32 and
// z = hi^2, the Taylor series sin r = hi + lo cos r + hi z (-1/3! + z/5! - ..), cos r = 1 - z/2 - hi lo + z^2 (1/4! - ..)
// end at hi^9 and hi^10 (the next terms are below 2e-9), and what 1 - z/2 and z lose to their rounding is added again.
__device__ __forceinline__ float2 turn_fp32(int position, float f, float mscale)
{
    constexpr double kQuarterHi = 1.5707963267948966, kQuarterLo = 6.123233995736766e-17, kInv = 0.6366197723675814;
    constexpr double kWhole = 6755399441055744.0;  // 1.5 * 2^52: a sum with it is rounded to whole numbers
    const double x = (double)position * (double)f, t = fma(x, kInv, kWhole), k = t - kWhole;
    const int quarter = __double2loint(t);
    const double r = fma(-k, kQuarterLo, fma(-k, kQuarterHi, x));
    const float hi = (float)r, lo = (float)(r - (double)hi), z = hi * hi, z_lo = fmaf(hi, hi, -z);
    float c = fmaf(z, -1.f / 3628800.f, 1.f / 40320.f);
    c = fmaf(c, z, -1.f / 720.f);
    c = fmaf(c, z, 1.f / 24.f);
    const float half = 0.5f * z, near = 1.f - half;
    c = near + (((1.f - near) - half) + fmaf(z * z, c, fmaf(-hi, lo, -0.5f * z_lo)));
    float s = fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
    s = fmaf(s, z, 1.f / 120.f);
    s = fmaf(s, z, -1.f / 6.f);
    s = hi + fmaf(hi * z, s, lo * c);
    const float cq = quarter & 1 ? s : c, sq = quarter & 1 ? c : s;
    return make_float2((quarter + 1 & 2 ? -cq : cq) * mscale, (quarter & 2 ? -sq : sq) * mscale);
}

// CTAs an SM that the registers are cut for: six where next to nothing is spilled for it
constexpr int rope_ctas(int size, Layout layout, int dim) { return size == 4 || layout == kHalvesUnaligned || dim == 0 ? 4 : 6; }

// DIM: the head dimension, or 0 for any other than those built
template <class A, Layout LAYOUT, int DIM>
__global__ void __launch_bounds__(kRopeThreads, rope_ctas(sizeof(typename A::raw), LAYOUT, DIM))
    rope_kernel(const RopeParams p)
{
    using raw = typename A::raw;
    extern __shared__ __align__(16) float2 angles[];  // [tokens of the CTA][n, rounded up to an even number]
    begin_early();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int D = DIM ? DIM : p.D, n = p.n, pitch = (n + 1) & ~1;
    const int lanes = D / 8, per = 32 / lanes;  // lanes a row, tokens a warp
    const int sub = lane / lanes, c = 8 * (lane - sub * lanes);
    const int split = p.split, tokens = kRopeWarps / split * per;  // warps that share their tokens' heads, tokens a CTA
    const long long t0 = (long long)blockIdx.x * tokens;
    const int mine = warp / split * per + sub, first_row = warp % split, step = split;  // token of the CTA; its heads
    const long long t = t0 + mine;
    const bool live = sub < per && t < p.T;
    const int at0 = first_row * D + c, jump = step * D;

    const raw *q = static_cast<const raw *>(p.q) + t * p.Hq * D + at0;
    Raw8<A> ahead[kAhead];
    auto read = [&](const raw *src, int i0, int rows) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (live && first_row + (i0 + i) * step < rows) ahead[i].load(src + (i0 + i) * jump);
    };
    read(q, 0, p.Hq);
    long long slot = -1;
    if (p.slots && live) {
        slot = p.slots[t];
        if (slot >= p.cache_rows) slot = -1;
    }

    const int here = (int)min((long long)tokens, p.T - t0) * n;
    for (int i = threadIdx.x; i < here; i += kRopeThreads) {
        const int tt = i / n, j = i - tt * n;
        const int position = p.positions[t0 + tt];
        const float f = p.inv_freq[j];
        angles[tt * pitch + j] = sizeof(raw) == 4 ? turn_fp32(position, f, p.mscale) : turn(position, f, p.mscale);
    }
    __syncthreads();

    // this lane's factors; `kept`: its columns that pass unchanged, a bit each
    float2 cs[4], sn[4];
    uint32_t kept = 0;
    const bool turns = c < 2 * n;
    if (turns && live) {
        const float2 *a = angles + mine * pitch;
        if (LAYOUT == kHalves) {
            const float4 *f = reinterpret_cast<const float4 *>(a + (c < n ? c : c - n));
            const float2 sign = c < n ? make_float2(-1.f, -1.f) : make_float2(1.f, 1.f);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 v = f[j];
                cs[j] = make_float2(v.x, v.z);
                sn[j] = fmul2(make_float2(v.y, v.w), sign);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int cc = c + j;
                float2 f = make_float2(1.f, 0.f);
                if (cc >= 2 * n) kept |= 1u << j;
                else if (LAYOUT == kPairs) f = a[cc / 2];
                else f = a[cc < n ? cc : cc - n];
                const bool minus = LAYOUT == kPairs ? !(j & 1) : cc < n;
                (j & 1 ? cs[j / 2].y : cs[j / 2].x) = f.x;
                (j & 1 ? sn[j / 2].y : sn[j / 2].x) = minus ? -f.y : f.y;
            }
        }
    }
    const int reach = n / 8, from = !turns ? lane : c < n ? lane + reach : lane - reach;  // kHalves: the partner's lane

    // one row that lies at src, from its 8 columns x here
    auto turned = [&](Raw8<A> &x, const raw *src) {
        Raw8<A> other;
        if (LAYOUT == kHalves) other = x.shuffled(from);
        if (live && turns) {
            float2 own[4], with[4];
            x.up2(own);
            if (LAYOUT == kPairs) {
#pragma unroll
                for (int j = 0; j < 4; ++j) with[j] = make_float2(own[j].y, own[j].x);
            } else if (LAYOUT == kHalves) {
                other.up2(with);
            } else {
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = c + j < 2 * n ? A::up(src[c + j < n ? j + n : j - n]) : 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) with[j] = make_float2(f[2 * j], f[2 * j + 1]);
            }
            float2 z[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                z[j] = ffma2(with[j], sn[j], fmul2(own[j], cs[j]));
                if (LAYOUT != kHalves) {
                    if (kept >> (2 * j) & 1) z[j].x = own[j].x;
                    if (kept >> (2 * j + 1) & 1) z[j].y = own[j].y;
                }
            }
            x.down2(z);
        }
        if (LAYOUT == kHalvesUnaligned) __syncwarp();  // q_out may be q: the partners are read before the writes
    };
    // the rows of one kind: `ahead` holds the first kAhead of them
    auto rows_of = [&](const raw *src, raw *out, raw *cached, int rows, bool turn) {
        for (int i0 = 0; first_row + i0 * step < rows; i0 += kAhead) {
            Raw8<A> x[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) x[i] = ahead[i];
            if (first_row + (i0 + kAhead) * step < rows) read(src, i0 + kAhead, rows);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (first_row + (i0 + i) * step >= rows) break;  // the whole warp is done
                if (turn) turned(x[i], src + (i0 + i) * jump);
                if (live && out) x[i].store(out + (i0 + i) * jump);
                if (live && cached) x[i].store(cached + (i0 + i) * jump);
            }
        }
    };
    rows_of(q, static_cast<raw *>(p.q_out) + t * p.Hq * D + at0, nullptr, p.Hq, true);
    const long long kv = t * p.Hkv * D + at0, row = slot * p.Hkv * D + at0;
    raw *k_out = p.k_out ? static_cast<raw *>(p.k_out) + kv : nullptr;
    raw *k_row = slot >= 0 ? static_cast<raw *>(p.k_cache) + row : nullptr;
    read(static_cast<const raw *>(p.k) + kv, 0, p.Hkv);
    rows_of(static_cast<const raw *>(p.k) + kv, k_out, k_row, p.Hkv, true);
    if (slot >= 0) {
        read(static_cast<const raw *>(p.v) + kv, 0, p.Hkv);
        rows_of(static_cast<const raw *>(p.v) + kv, nullptr, static_cast<raw *>(p.v_cache) + row, p.Hkv, false);
    }
}

template <class A, Layout LAYOUT>
cudaError_t launch_dim(const RopeParams &p, cudaStream_t st)
{
    const int tokens = kRopeWarps / p.split * (32 / (p.D / 8));
    const unsigned grid = (unsigned)((p.T + tokens - 1) / tokens);
    const size_t smem = sizeof(float2) * tokens * ((p.n + 1) & ~1);
    switch (p.D) {
    case 64: return launch_early(rope_kernel<A, LAYOUT, 64>, grid, kRopeThreads, smem, st, p);
    case 80: return launch_early(rope_kernel<A, LAYOUT, 80>, grid, kRopeThreads, smem, st, p);
    case 96: return launch_early(rope_kernel<A, LAYOUT, 96>, grid, kRopeThreads, smem, st, p);
    case 128: return launch_early(rope_kernel<A, LAYOUT, 128>, grid, kRopeThreads, smem, st, p);
    case 192: return launch_early(rope_kernel<A, LAYOUT, 192>, grid, kRopeThreads, smem, st, p);
    case 256: return launch_early(rope_kernel<A, LAYOUT, 256>, grid, kRopeThreads, smem, st, p);
    default: return launch_early(rope_kernel<A, LAYOUT, 0>, grid, kRopeThreads, smem, st, p);
    }
}

template <class A>
cudaError_t launch_type(const RopeParams &p, bool interleaved, cudaStream_t st)
{
    if (interleaved) return launch_dim<A, kPairs>(p, st);
    return p.n % 8 == 0 ? launch_dim<A, kHalves>(p, st) : launch_dim<A, kHalvesUnaligned>(p, st);
}

}  // namespace

cudaError_t launch_rope(const RopeParams &in, int act_dtype, bool interleaved, cudaStream_t st)
{
    RopeParams p = in;
    // split the heads over warps as long as all CTAs find room at once (148 SMs of six): a second turn of CTAs costs more
    // than idle warps (2000 tokens of 16 + 2 heads of 256: 7.2 us with 2000 warps, 8.8 with 4000, 10.6 with 8000; 4099 of
    // 32 + 8 of 128, fp16: 15.2 us with 2050, 16.7 with 4100)
    const int heads = std::max(p.Hq, p.Hkv), per = 32 / (p.D / 8);
    p.split = 1;
    while (p.split < kRopeWarps && p.split < heads && (p.T + per - 1) / per * p.split * 2 <= 148 * 6 * kRopeWarps) p.split *= 2;
    switch (act_dtype) {
    case GDN_DTYPE_BF16: return launch_type<Bf16>(p, interleaved, st);
    case GDN_DTYPE_FP16: return launch_type<F16>(p, interleaved, st);
    default: return launch_type<F32>(p, interleaved, st);
    }
}

}  // namespace gdn
