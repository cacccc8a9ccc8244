// Root-mean-square norm of rows, with the residual's addition, the SiLU gate of a delta-rule
// layer's output and an 8-bit output with scales (gdn_rms_norm):
//
//   z = x + residual,  y = z rstd (w + w0) [gate / (1 + e^-gate)],  rstd = 1 / sqrt(mean(z^2) + eps)
//
// About 10 flops an element, so HBM bounds it as long as the instructions an element takes stay few:
// a B200 SM moves an element of a bf16 row in some 30 instruction slots.  So every matrix is read and
// written once, a row stays in registers (z, fp32) between its sum of squares and its output, a thread
// holds 32 columns of it (what a row costs beside its elements, the reductions and the addresses, is
// shared by them; with 16 the norm of a 16384 x 4096 prefill took 94 us at 36 instructions an element),
// and the arithmetic is packed in pairs.  L threads share a row: 4 to 32 lanes of a warp (up to 1024
// columns: the sums are a few shuffles) or a CTA of up to 1024.
//
// A row's units are the 16-byte blocks of memory that it touches, so a thread's accesses are aligned
// whatever the width is.  kFull: width = a thread's columns times L.  kAligned: any whole number of blocks.
// kShifted: a row begins ph elements into a block, so column c lies at place c + ph, and the elements of the
// first and last block that belong to the neighbouring rows are masked.  (All matrices have the same width
// and aligned bases, so one ph serves all; an 8-bit row's blocks are half as long and aligned too.)  A group
// of 128 columns then begins inside a unit: that unit's lane keeps two maxima, and a row's scales come from
// shared memory.
//
// Measured: 16384 x 4096 bf16 with a residual and row scales 76 us, 6.1 TB/s, 95 % of the copy rate; 1048576 heads
// of 128 with a gate and 8 bits 110 us, 6.1 TB/s; 4099 x 1537 fp32 with residual and gate (kShifted) 27 us, 4.6 TB/s;
// 8 x 2048 2.5 us.
#include <algorithm>
#include <type_traits>

#include "gdn_layers.h"
#include "layers.cuh"

namespace gdn {

namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126: keeps 1 / scale finite for an all-zero row
constexpr float kLog2e = 1.44269504f;
constexpr int kNormSms = 148, kNormSmem = 227 * 1024;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// max |y| / 448, at least kMinScale, and 1 / scale: a multiplication or an approximate reciprocal and one step of Newton, so
// that each is rounded about once.  (Infinity has no such step.)  Then y (1 / scale) is within 2^-23 of y / scale; the
// division itself, two operations an element, moved 2 % fewer bytes at rounding borders and took 2 to 4 % longer.
__device__ __forceinline__ float scale_of_max(float m)
{
    const float c = 1.f / kE4m3Max, q = m * c, e = fmaf(-q, kE4m3Max, m);
    return absmax_nan(kMinScale, m < INFINITY ? fmaf(e, c, q) : q);
}
__device__ __forceinline__ float inverse(float scale)
{
    const float r = rcp(scale), e = fmaf(-scale, r, 1.f);
    return scale < INFINITY ? fmaf(r, e, r) : r;
}
// g / (1 + e^-g); e^-g = infinity gives -0, as the formula does
__device__ __forceinline__ float2 silu(float2 g)
{
    const float2 t = fmul2(g, make_float2(-kLog2e, -kLog2e));
    const float2 d = fadd2(make_float2(ex2(t.x), ex2(t.y)), make_float2(1.f, 1.f));
    return fmul2(g, make_float2(rcp(d.x), rcp(d.y)));
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float x)
{
#pragma unroll
    for (int o = LANES >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
template <int LANES>
__device__ __forceinline__ float lanes_max(float x)
{
#pragma unroll
    for (int o = LANES >> 1; o > 0; o >>= 1) x = absmax_nan(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

enum Kind { kFull, kAligned, kShifted };

// 16 bytes of the activations' type as N fp32 in pairs, and back
template <class A>
struct Unit {
    using raw = typename A::raw;
    static constexpr int N = 16 / (int)sizeof(raw);
    static __device__ __forceinline__ void up(const uint4 &w, float2 (&x)[N / 2])
    {
        if constexpr (N == 8) {
            x[0] = A::up2(w.x), x[1] = A::up2(w.y), x[2] = A::up2(w.z), x[3] = A::up2(w.w);
        } else {
            x[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
            x[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
        }
    }
    static __device__ __forceinline__ uint4 down(const float2 (&x)[N / 2])
    {
        if constexpr (N == 8)
            return make_uint4(A::down2(x[0].x, x[0].y), A::down2(x[1].x, x[1].y), A::down2(x[2].x, x[2].y),
                              A::down2(x[3].x, x[3].y));
        else
            return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x),
                              __float_as_uint(x[1].y));
    }
    static __device__ __forceinline__ void store8(uint8_t *p, const float2 (&x)[N / 2])
    {
        const uint32_t lo = pack_e4m3(x[0].x, x[0].y, x[1].x, x[1].y);
        if constexpr (N == 8)
            *reinterpret_cast<uint2 *>(p) = make_uint2(lo, pack_e4m3(x[2].x, x[2].y, x[3].x, x[3].y));
        else
            *reinterpret_cast<uint32_t *>(p) = lo;
    }
};

__device__ __forceinline__ float weight_at(const NormParams &p, int c, bool f16)
{
    if (p.weight_f32) return static_cast<const float *>(p.weight)[c];
    const uint16_t w = static_cast<const uint16_t *>(p.weight)[c];
    return f16 ? F16::up(w) : Bf16::up(w);
}

constexpr int kNarrowBlock = 128;  // threads of a CTA whose warps hold whole rows
__host__ __device__ constexpr int norm_block(int L) { return L <= 32 ? kNarrowBlock : L; }
// CTAs an SM that the registers leave room for
__host__ __device__ constexpr int norm_ctas(int L) { return L <= 384 ? 768 / norm_block(L) : 1024 / L; }
// Rows come through shared memory: cp.async brings a group's next row while it works on this one.  A thread
// fetches what it will use itself, so no barrier orders it, and one stage will do: the next row's x and residual
// are asked for as soon as this one's sum is in registers, its gate after this one's use.  A second stage, with the next
// row on its way before this one is waited for, is taken where it costs no CTA its room and a row is more than a warp's
// (16384 x 4096 bf16 with a residual and row scales 76 us, 86 with one stage; with a gate too, where it costs two CTAs of
// six, 105 against 94; heads of 128 with a gate 68.5 against 62); rows that begin inside a block have too many
// instructions to gain by it (fp16, 1537 columns with a residual: 146 against 129).  fp32 rows beyond 16384 columns,
// too wide for three of them to lie there, go straight to registers.
template <class A>
__host__ __device__ constexpr bool norm_ring(int L, int PER) { return L * PER * (int)sizeof(typename A::raw) <= 65536; }
__host__ __device__ constexpr bool norm_two_stages(Kind kind, int L) { return kind != kShifted && L > 32; }
// Where warps hold whole rows, and in kShifted, the weights lie in shared memory in fp32, offset added; else they come
// from L1 in 16-byte blocks.  In order, or in kShifted in lines along which a unit's neighbours lie beside it, with zeros
// outside the row.  L <= 32: 2 N - 1 lines, line r holds at i the weight N i + r - (N - 1); a unit i of a row that begins
// ph elements into a block reads lines N - 1 - ph to 2 N - 2 - ph at i, all at one distance.  L > 32, for half the
// room: N lines, line r holds the weight N i + r at i + 1; a unit's element j lies in line (j - ph) mod N, at i + 1, or
// at i where j < ph.  (With a weight at a time from L1: 16384 x 4097 bf16 with a residual 120 us, so 90.)  Up to 10240
// places of 16 bits, 12288 of fp32: beyond, they take a CTA's room (12001 columns bf16 with a residual 98 us against
// 110, but with a gate too 182 against 139).
template <class A>
__host__ __device__ constexpr int norm_line(int L, int PER) { return L * PER / Unit<A>::N + 1; }
__host__ __device__ constexpr bool norm_weights(Kind kind, int L, int PER)
{
    return L <= 32 || (kind == kShifted && L * PER <= (PER == 16 ? 12288 : 10240));
}
template <class A>
__host__ __device__ constexpr int norm_weight_bytes(Kind kind, int L, int PER)
{
    return !norm_weights(kind, L, PER) ? 0
           : kind != kShifted          ? L * PER * 4
                                       : ((L <= 32 ? 2 * Unit<A>::N - 1 : Unit<A>::N) * norm_line<A>(L, PER) * 4 + 15) / 16 * 16;
}
__host__ __device__ constexpr int pow2(int n) { return n <= 1 ? 1 : 2 * pow2((n + 1) / 2); }

// A group of L threads of PER columns each strides over the rows.
template <class A, Kind KIND, int L, int PER>
__global__ void __launch_bounds__(norm_block(L), norm_ctas(L)) rms_norm_kernel(const NormParams p)
{
    using U = Unit<A>;
    using raw = typename A::raw;
    constexpr bool kRing = norm_ring<A>(L, PER), kShared = norm_weights(KIND, L, PER), kShift = KIND == kShifted;
    constexpr bool kF16 = std::is_same<A, F16>::value;
    constexpr int N = U::N, H = N / 2, NV = PER / N;
    constexpr int W = L < 32 ? L : 32, kWarps = pow2(L / 32);  // warps, rounded up for the shuffles
    constexpr int kBlock = norm_block(L), kRows = L <= 32 ? kBlock / L : 1, kStep = L * N;
    constexpr int kGroupLanes = 128 / N;  // lanes that hold a group of 128 columns
    __shared__ float red[2][32];
    // kShifted, a row's groups: maxima of the elements behind the phase of their first unit, and of those before it
    // (which belong to the group before)
    constexpr int kGroups = L * PER / 128 + 1;
    __shared__ float group_max[kShift ? kRows : 1][kShift ? kGroups : 1], group_lead[kShift ? kRows : 1][kShift ? kGroups : 1];
    extern __shared__ __align__(16) uint8_t smem[];
    begin_early();
    const int t = L <= 32 ? (int)threadIdx.x % L : (int)threadIdx.x;
    const int width = KIND == kFull ? PER * L : p.width, quant = p.quant;
    const int v0 = t * N;  // place of this thread's first element, phase added
    const int first = (int)(L <= 32 ? blockIdx.x * kRows + threadIdx.x / L : blockIdx.x);
    const int stride = (int)gridDim.x * kRows, rows = (int)p.rows;
    const int mine_row = L <= 32 ? (int)threadIdx.x / L : 0, groups = (width + GDN_QUANT_GROUP - 1) / GDN_QUANT_GROUP;
    const bool residual = p.residual != nullptr, gated = p.gate != nullptr;
    const raw *x = static_cast<const raw *>(p.x), *res = static_cast<const raw *>(p.residual),
              *gate = static_cast<const raw *>(p.gate);
    const long long end = p.rows * width;
    // elements of the row's first block before the row
    auto phase = [&](int row) { return kShift ? (int)((long long)row * width) & (N - 1) : 0; };

    float *weights = reinterpret_cast<float *>(smem);
    uint8_t *ring = smem + norm_weight_bytes<A>(KIND, L, PER);
    constexpr int kLine = norm_line<A>(L, PER);
    // this thread's 16 bytes of (matrix, unit); matrices in the order x, residual, gate
    constexpr int kPlane = kBlock * 16, kMatrix = NV * kPlane;
    const int gate_at = residual ? 2 * kMatrix : kMatrix;
    const bool two = norm_two_stages(KIND, L) && p.two_stages;
    const int stage_bytes = two ? kMatrix * (1 + residual + gated) : 0;
    const uint8_t *mine = ring + threadIdx.x * 16;
    const uint32_t mine_addr = smem_addr(mine);
    // elements of the matrix from the row's first on (a block of its last rows may end behind them), as an int
    auto rest_of = [&](int row) { return (int)min(end - (long long)row * width, 1LL << 20); };
    // a row's x and residual, or its gate, to a stage
    auto fetch = [&](int stage, int row, bool sum, bool gates) {
        if (row < rows) {
            const uint32_t to = mine_addr + stage * stage_bytes;
            const int c0 = v0 - phase(row), rest = kShift ? rest_of(row) : 0;
            const long long at = (long long)row * width + c0;
            const raw *fx = x + at, *fr = res + at, *fg = gate + at;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = c0 + k * kStep;
                if (KIND != kFull && c >= width) continue;
                const int bytes = !kShift ? 16 : min(16, (rest - c) * (int)sizeof(raw));
                if (sum) cp_async16_part(to + k * kPlane, fx + k * kStep, bytes);
                if (sum && residual) cp_async16_part(to + kMatrix + k * kPlane, fr + k * kStep, bytes);
                if (gates && gated) cp_async16_part(to + gate_at + k * kPlane, fg + k * kStep, bytes);
            }
        }
    };
    // Units from here on: m points at the unit's first element, c is its column, `in` whether the whole unit lies
    // in the row.
    auto load = [&](const raw *m, int c, int rest) {  // without a ring
        if (!kShift || c + N <= rest) return *reinterpret_cast<const uint4 *>(m);
        uint32_t w[4] = {};
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (c + j < rest) {
                if constexpr (sizeof(raw) == 2) w[j / 2] |= (uint32_t)m[j] << 16 * (j & 1);
                else w[j] = __float_as_uint(m[j]);
            }
        return make_uint4(w[0], w[1], w[2], w[3]);
    };
    auto mask = [&](int c, bool in, float2 (&v)[H]) {  // clears what is not in the row
        if constexpr (kShift) {
            if (in) return;
#pragma unroll
            for (int j = 0; j < N; ++j)
                if ((unsigned)(c + j) >= (unsigned)width) (j & 1 ? v[j / 2].y : v[j / 2].x) = 0.f;
        }
    };
    auto store = [&](raw *m, int c, bool in, const float2 (&v)[H]) {
        if (!kShift || in) {
            *reinterpret_cast<uint4 *>(m) = U::down(v);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if ((unsigned)(c + j) < (unsigned)width) m[j] = A::down(j & 1 ? v[j / 2].y : v[j / 2].x);
        }
    };
    auto store8 = [&](uint8_t *m, int c, bool in, const float2 (&v)[H]) {
        if (!kShift || in) {
            U::store8(m, v);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if ((unsigned)(c + j) < (unsigned)width) m[j] = to_e4m3(j & 1 ? v[j / 2].y : v[j / 2].x);
        }
    };
    int lines[kShared && kShift && L > 32 ? N : 1];  // places of the weights of this row's first unit here
    auto weigh = [&](int k, int c, bool in, float2 (&w)[H]) {  // the weights of unit k
        if constexpr (kShared && !kShift) {
#pragma unroll
            for (int i = 0; i < N / 4; ++i) {
                const float4 v = reinterpret_cast<const float4 *>(weights + c)[i];
                w[2 * i] = make_float2(v.x, v.y);
                w[2 * i + 1] = make_float2(v.z, v.w);
            }
            return;
        } else if constexpr (kShared) {
#pragma unroll
            for (int j = 0; j < N; ++j) (j & 1 ? w[j / 2].y : w[j / 2].x) = weights[L <= 32 ? lines[0] + j * kLine + k * L : lines[j] + k * L];
            return;
        }
        if (!kShift || in) {
            if (p.weight_f32) {
                const float *m = static_cast<const float *>(p.weight) + c;
                if (!kShift || (c & 3) == 0) {
#pragma unroll
                    for (int i = 0; i < N / 4; ++i) {
                        const float4 v = reinterpret_cast<const float4 *>(m)[i];
                        w[2 * i] = make_float2(v.x, v.y);
                        w[2 * i + 1] = make_float2(v.z, v.w);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < H; ++j) w[j] = make_float2(m[2 * j], m[2 * j + 1]);
                }
            } else if (!kShift || (c & (N - 1)) == 0) {
                U::up(*reinterpret_cast<const uint4 *>(static_cast<const raw *>(p.weight) + c), w);
            } else {
                const raw *m = static_cast<const raw *>(p.weight) + c;
#pragma unroll
                for (int j = 0; j < H; ++j) w[j] = make_float2(A::up(m[2 * j]), A::up(m[2 * j + 1]));
            }
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float f = (unsigned)(c + j) < (unsigned)width ? weight_at(p, c + j, kF16) : 0.f;
                (j & 1 ? w[j / 2].y : w[j / 2].x) = f;
            }
        }
#pragma unroll
        for (int j = 0; j < H; ++j) w[j] = fadd2(w[j], make_float2(p.weight_offset, p.weight_offset));
    };

    // turns of the loop: the same for all threads of a warp; a group without a row left does the last turn on
    // nothing and writes nothing
    const int warp_first = first - (L < 32 ? ((int)threadIdx.x & 31) / L : 0);
    const int turns = warp_first >= rows ? 0 : (rows - 1 - warp_first) / stride + 1;
    if (kRing) fetch(0, first, true, true);
    if (kShared) {
        if (!kShift) {
            for (int c = threadIdx.x; c < width; c += kBlock) weights[c] = weight_at(p, c, kF16) + p.weight_offset;
        } else {
            for (int i = threadIdx.x; L <= 32 && i < (2 * N - 1) * kLine; i += kBlock) {
                const int line = i / kLine, c = (i - line * kLine) * N + line - (N - 1);
                weights[i] = c >= 0 && c < width ? weight_at(p, c, kF16) + p.weight_offset : 0.f;
            }
            if (L > 32 && threadIdx.x < N) weights[threadIdx.x * kLine] = 0.f;
            for (int c = threadIdx.x; L > 32 && c < L * PER; c += kBlock)
                weights[c % N * kLine + c / N + 1] = c < width ? weight_at(p, c, kF16) + p.weight_offset : 0.f;
        }
    }
    if (kShift) {
        for (int i = threadIdx.x; i < kRows * kGroups; i += kBlock) group_max[0][i] = group_lead[0][i] = 0.f;
    }
    if (kShared || L > 32) {
        if (threadIdx.x < 64) red[threadIdx.x / 32][threadIdx.x % 32] = 0.f;  // for warps that there are not
        __syncthreads();
    }
    for (int turn = 0; turn < turns; ++turn) {
        const int row = first + turn * stride;
        const bool live = row < rows;
        const int ph = phase(row), c0 = v0 - ph, rest = kShift ? rest_of(row) : 0;
        const long long at = (long long)row * width + c0;
        const raw *rx = x + at, *rr = res + at, *rg = gate + at;
        const int next = row < rows - stride ? row + stride : rows;
        const uint8_t *held = mine + (turn & 1) * stage_bytes;
        if (kRing) {
            cp_async_commit();
            if (two) {
                fetch((turn + 1) & 1, next, true, true);
                cp_async_commit();
                cp_async_wait<1>();
            } else {
                cp_async_wait<0>();
            }
        }
        auto has = [&](int k) {
            return live && (KIND == kFull || c0 + k * kStep < width);
        };
        auto inside = [&](int c) { return !kShift || (c >= 0 && c + N <= width); };
        float2 z[NV][H], sum2 = make_float2(0.f, 0.f);
        constexpr int kBatch = kRing ? 1 : NV / 2;  // units in flight at a time where there is no ring
#pragma unroll
        for (int k0 = 0; k0 < NV; k0 += kBatch) {
            uint4 xw[kBatch], rw[kBatch];
            if (!kRing) {
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int k = k0 + i, c = c0 + k * kStep;
                    if (!has(k)) continue;
                    xw[i] = load(rx + k * kStep, c, rest);
                    if (residual) rw[i] = load(rr + k * kStep, c, rest);
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int k = k0 + i, c = c0 + k * kStep;
                if (!has(k)) continue;
                const bool in = inside(c);
                if (kRing) xw[i] = *reinterpret_cast<const uint4 *>(held + k * kPlane);
                U::up(xw[i], z[k]);
                if (residual) {
                    float2 r[H];
                    if (kRing) rw[i] = *reinterpret_cast<const uint4 *>(held + kMatrix + k * kPlane);
                    U::up(rw[i], r);
#pragma unroll
                    for (int j = 0; j < H; ++j) z[k][j] = fadd2(z[k][j], r[j]);
                    store(static_cast<raw *>(p.residual_out) + at + k * kStep, c, in, z[k]);
                }
                mask(c, in, z[k]);
#pragma unroll
                for (int j = 0; j < H; ++j) sum2 = ffma2(z[k][j], z[k][j], sum2);
            }
        }
        if (kRing && !two) fetch(0, next, true, false);
        float sum = lanes_sum<W>(sum2.x + sum2.y);
        if (L > 32) {
            if ((t & 31) == 0) red[0][t >> 5] = sum;
            __syncthreads();
            sum = lanes_sum<kWarps>(red[0][t & (kWarps - 1)]);
        }
        const float rstd = rsqrtf(fmaf(sum, p.inv_width, p.eps));

        if constexpr (kShared && kShift) {
#pragma unroll
            for (int j = 0; j < (L <= 32 ? 1 : N); ++j)
                lines[j] = L <= 32 ? (N - 1 - ph) * kLine + t : ((j - ph) & (N - 1)) * kLine + t + (j >= ph);
        }
        const bool leads = (t & (kGroupLanes - 1)) == 0;  // whether this thread's units begin groups
        float most = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (KIND != kFull && k * kStep - (kShift ? N - 1 : 0) >= width) break;  // no thread has such a unit
            const int c = c0 + k * kStep;
            const bool in = inside(c);
            float m = 0.f, lead = 0.f;
            if (has(k)) {
                float2 w[H];
                weigh(k, c, in, w);
#pragma unroll
                for (int j = 0; j < H; ++j) z[k][j] = fmul2(fmul2(z[k][j], make_float2(rstd, rstd)), w[j]);
                if (gated) {
                    float2 g[H];
                    U::up(kRing ? *reinterpret_cast<const uint4 *>(held + gate_at + k * kPlane) : load(rg + k * kStep, c, rest), g);
                    mask(c, in, g);
#pragma unroll
                    for (int j = 0; j < H; ++j) z[k][j] = fmul2(z[k][j], silu(g[j]));
                }
                if (quant == GDN_QUANT_NONE) store(static_cast<raw *>(p.out) + at + k * kStep, c, in, z[k]);
                else if (kShift && quant == GDN_QUANT_BLOCK) {
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const float f = j & 1 ? z[k][j / 2].y : z[k][j / 2].x;
                        if (leads && j < ph) lead = absmax_nan(lead, f);
                        else m = absmax_nan(m, f);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < H; ++j) m = absmax_nan(absmax_nan(m, z[k][j].x), z[k][j].y);
                }
            }
            if (quant == GDN_QUANT_BLOCK) {
                m = lanes_max<kGroupLanes < W ? kGroupLanes : W>(m);
                if (kShift) {
                    if (leads) group_max[mine_row][(t + k * L) / kGroupLanes] = m, group_lead[mine_row][(t + k * L) / kGroupLanes] = lead;
                } else {
                    const float scale = scale_of_max(m), inv = inverse(scale);
                    if (has(k)) {
#pragma unroll
                        for (int j = 0; j < H; ++j) z[k][j] = fmul2(z[k][j], make_float2(inv, inv));
                        store8(static_cast<uint8_t *>(p.out) + at + k * kStep, c, in, z[k]);
                        if (leads) p.scales[(long long)row * groups + c / GDN_QUANT_GROUP] = scale;
                    }
                }
            }
            most = absmax_nan(absmax_nan(most, m), lead);
        }
        if (kRing && gated && !two) fetch(0, next, false, true);
        if (kShift && quant == GDN_QUANT_BLOCK) {
            if (L > 32) __syncthreads();
            else __syncwarp();
            // (two scales a unit, so without scale_of_max's second step: 16384 x 1537 fp32 with a gate 86 us, 89 with it)
            auto scale_of = [&](int g) {
                return absmax_nan(kMinScale, absmax_nan(group_max[mine_row][g], group_lead[mine_row][g + 1]) * (1.f / kE4m3Max));
            };
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (!has(k)) continue;
                const int c = c0 + k * kStep, g = (t + k * L) / kGroupLanes;
                // (the phase may leave the row's last unit nothing behind it)
                const float scale = g < groups ? scale_of(g) : kMinScale, inv = __fdividef(1.f, scale);
                if (leads && g < groups) p.scales[(long long)row * groups + g] = scale;
                const float before = leads && ph > 0 && g > 0 ? __fdividef(1.f, scale_of(g - 1)) : inv;
#pragma unroll
                for (int j = 0; j < N; ++j) (j & 1 ? z[k][j / 2].y : z[k][j / 2].x) *= leads && j < ph ? before : inv;
                store8(static_cast<uint8_t *>(p.out) + at + k * kStep, c, inside(c), z[k]);
            }
            if (L <= 32) __syncwarp();  // (L > 32: the barrier below) before the next row's maxima
        }
        if (quant == GDN_QUANT_ROW) {
            most = lanes_max<W>(most);
            if (L > 32) {
                if ((t & 31) == 0) red[1][t >> 5] = most;
                __syncthreads();
                most = lanes_max<kWarps>(red[1][t & (kWarps - 1)]);
            }
            const float scale = scale_of_max(most), inv = inverse(scale);
            if (live && t == 0) p.scales[row] = scale;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (!has(k)) continue;
#pragma unroll
                for (int j = 0; j < H; ++j) z[k][j] = fmul2(z[k][j], make_float2(inv, inv));
                const int c = c0 + k * kStep;
                store8(static_cast<uint8_t *>(p.out) + at + k * kStep, c, inside(c), z[k]);
            }
        } else if (L > 32) {
            __syncthreads();  // red[0] is read before the next row writes it
        }
    }
}

// The dynamic shared memory of a launch that reads this many matrices, and whether it holds two stages of a row.
struct NormSmem {
    int bytes;
    bool two_stages;
};
constexpr int norm_beside(Kind kind, int L, int PER)  // the static part, and the driver's KB
{
    return 1280 + (kind == kShifted ? norm_block(L) * PER / 16 : 0);
}
template <class A>
constexpr NormSmem norm_smem(Kind kind, int L, int PER, int matrices)
{
    const int stage = norm_ring<A>(L, PER) ? norm_block(L) * PER * (int)sizeof(typename A::raw) * matrices : 0;
    const int one = norm_weight_bytes<A>(kind, L, PER) + stage;
    const bool two = norm_two_stages(kind, L) && kNormSmem / (one + stage + norm_beside(kind, L, PER)) >= norm_ctas(L);
    return NormSmem{two ? one + stage : one, two};
}
template <class A>
constexpr int norm_smem_most(Kind kind, int L, int PER)  // of all launches of an instance
{
    int most = 0;
    for (int matrices = 1; matrices <= 3; ++matrices)
        if (norm_smem<A>(kind, L, PER, matrices).bytes > most) most = norm_smem<A>(kind, L, PER, matrices).bytes;
    return most;
}

template <class A, Kind KIND, int L, int PER>
cudaError_t launch_kernel(const NormParams &p, cudaStream_t st)
{
    NormParams q = p;
    const auto kern = rms_norm_kernel<A, KIND, L, PER>;
    constexpr int block = norm_block(L), rows = L <= 32 ? block / L : 1, beside = norm_beside(KIND, L, PER);
    const NormSmem smem = norm_smem<A>(KIND, L, PER, 1 + (p.residual != nullptr) + (p.gate != nullptr));
    q.two_stages = smem.two_stages;
    // The limit belongs to the kernel, not to the launch, and host threads share it: every call sets it to the same value,
    // so that none takes from another between its setting and its launch.
    constexpr int most = norm_smem_most<A>(KIND, L, PER);
    static_assert(most + beside <= kNormSmem, "a row's matrices fit into an SM");
    if (most > 47 * 1024) {  // 48 KB with the static part
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return e;
    }
    const int per_sm = std::max(1, std::min(norm_ctas(L), kNormSmem / (smem.bytes + beside)));
    const long long want = (p.rows + rows - 1) / rows;
    return launch_early(kern, (unsigned)std::min<long long>(want, (long long)kNormSms * per_sm), block, smem.bytes, st, q);
}

// The threads of a row: the fewest of those built that hold `places` places, at least `least`.  A thread holds 32
// columns of a 16-bit type; 16 of fp32, whose elements have twice the time and take twice the room (1537 columns
// with residual and gate: 39 us with 32, 8 warps an SM), until a CTA has no more threads.
template <class A, Kind KIND, int L, int... MORE>
cudaError_t launch_lanes(const NormParams &p, int places, int least, cudaStream_t st)
{
    constexpr int PER = sizeof(typename A::raw) == 4 ? 16 : 32;
    if constexpr (sizeof...(MORE) > 0) {
        if (L < least || L * PER < places) return launch_lanes<A, KIND, MORE...>(p, places, least, st);
    } else if constexpr (PER == 16) {
        if (L * PER < places) return launch_kernel<A, KIND, L, 32>(p, st);
    }
    return launch_kernel<A, KIND, L, PER>(p, st);
}

template <class A>
cudaError_t launch_type(NormParams p, cudaStream_t st)
{
    constexpr int N = Unit<A>::N, PER = sizeof(typename A::raw) == 4 ? 16 : 32;
    const int width = p.width;
    if (p.quant == GDN_QUANT_BLOCK && width <= GDN_QUANT_GROUP) p.quant = GDN_QUANT_ROW;  // one group a row
    const int least = p.quant == GDN_QUANT_BLOCK ? 128 / N : 0;  // lanes that hold a group
    if (width % N == 0) {
        int lanes = std::max(4, least);
        while (lanes < 1024 && lanes * PER < width) lanes *= 2;
        return lanes * PER == width || 1024 * 32 == width
                   ? launch_lanes<A, kFull, 4, 8, 16, 32, 64, 128, 256, 512, 1024>(p, width, least, st)
                   : launch_lanes<A, kAligned, 4, 8, 16, 32, 64, 96, 128, 160, 192, 256, 320, 384, 448, 512, 640, 768, 1024>(p, width, least, st);
    }
    // a row that begins inside a block takes up to a unit more
    return launch_lanes<A, kShifted, 4, 8, 16, 32, 64, 96, 128, 160, 192, 256, 320, 384, 512, 768, 1024>(p, width + N - 1, least, st);
}

}  // namespace

cudaError_t launch_rms_norm(const NormParams &p, int act_dtype, cudaStream_t st)
{
    switch (act_dtype) {
    case GDN_DTYPE_BF16: return launch_type<Bf16>(p, st);
    case GDN_DTYPE_FP16: return launch_type<F16>(p, st);
    default: return launch_type<F32>(p, st);
    }
}

}  // namespace gdn
