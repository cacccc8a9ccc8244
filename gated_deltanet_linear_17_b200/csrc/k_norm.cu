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
// whatever the width is: in a row that begins p elements into a block, column c lies at place c + p, and
// the elements of the first and last block that belong to the neighbouring rows are masked.  (All
// matrices have the same width and aligned bases, so one p serves all; 8-bit rows begin at a multiple of
// half a block minus p, and their stores are aligned too.)  kFull: width = 32 L, no masks.  Groups of
// 128 columns in rows that are not whole blocks fall across the blocks; such rows (kElements) take element
// accesses: a warp holds the groups, lane l the columns l, l + 32, l + 64, l + 96 of each.
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

enum Kind { kFull, kBlocks, kElements };

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
__host__ __device__ constexpr int norm_ctas(int L) { return (L <= 256 ? 768 : 1024) / norm_block(L); }
// Rows up to 8192 columns come through two stages in shared memory: cp.async brings a group's next row while it
// works on this one.  A thread fetches what it will use itself, so no barrier orders the stages.  Wider rows go
// straight to registers.
__host__ __device__ constexpr bool norm_ring(Kind kind, int L) { return kind != kElements && L <= 256; }
// Where warps hold whole rows, the weights lie in shared memory in fp32, offset added, one float of padding behind
// every N: the lanes of a warp then read N columns apart from different banks.
__host__ __device__ constexpr bool norm_weights(Kind kind, int L) { return kind != kElements && L <= 32; }
template <int N>
__host__ __device__ constexpr int padded(int c) { return c + c / N; }

// A group of L threads strides over the rows; each of them holds 32 columns.
template <class A, Kind KIND, int L>
__global__ void __launch_bounds__(norm_block(L), norm_ctas(L)) rms_norm_kernel(const NormParams p)
{
    using U = Unit<A>;
    using raw = typename A::raw;
    constexpr bool kEl = KIND == kElements, kRing = norm_ring(KIND, L), kShared = norm_weights(KIND, L);
    constexpr bool kF16 = std::is_same<A, F16>::value;
    constexpr int N = kEl ? 4 : U::N, H = N / 2, NV = 32 / N, W = L < 32 ? L : 32, kWarps = L / 32;
    constexpr int kBlock = norm_block(L), kRows = L <= 32 ? kBlock / L : 1, kStep = L * N;
    constexpr int kGroupLanes = kEl ? 32 : 128 / N;  // lanes that hold a group of 128 columns
    __shared__ float red[2][32];
    extern __shared__ __align__(16) uint8_t smem[];
    const int t = L <= 32 ? (int)threadIdx.x % L : (int)threadIdx.x;
    const int width = KIND == kFull ? 32 * L : p.width, quant = p.quant;
    const int v0 = kEl ? (t >> 5) * 128 + (t & 31) : t * N;  // place of this thread's first element, phase added
    const int first = (int)(L <= 32 ? blockIdx.x * kRows + threadIdx.x / L : blockIdx.x);
    const int stride = (int)gridDim.x * kRows, rows = (int)p.rows;
    const bool residual = p.residual != nullptr, gated = p.gate != nullptr;
    const raw *x = static_cast<const raw *>(p.x), *res = static_cast<const raw *>(p.residual),
              *gate = static_cast<const raw *>(p.gate);
    const long long end = p.rows * width;
    // elements of the row's first block before the row
    auto phase = [&](int row) { return KIND == kBlocks ? (int)((long long)row * width) & (N - 1) : 0; };

    float *weights = reinterpret_cast<float *>(smem);
    uint8_t *ring = smem + (kShared ? (padded<U::N>(32 * L) * 4 + 15) / 16 * 16 : 0);
    // this thread's 16 bytes of (stage, matrix, unit); matrices in the order x, residual, gate
    constexpr int kPlane = kBlock * 16, kMatrix = NV * kPlane;
    const int gate_at = residual ? 2 * kMatrix : kMatrix, stage_bytes = kMatrix * (1 + residual + gated);
    uint8_t *mine = ring + threadIdx.x * 16;
    const uint32_t mine_addr = smem_addr(mine);
    auto fetch = [&](int stage, int row) {
        if (row < rows) {
            const int ph = phase(row);
            const long long at = (long long)row * width - ph + v0;
            const uint32_t dst = mine_addr + stage * stage_bytes;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int v = v0 + k * kStep;
                if (KIND != kFull && v - ph >= width) continue;
                const long long e = at + k * kStep;
                // the last block of the matrix may be a part of one
                const int bytes = KIND == kFull ? 16 : (int)min(16LL, (end - e) * (long long)sizeof(raw));
                cp_async16_part(dst + k * kPlane, x + e, bytes);
                if (residual) cp_async16_part(dst + kMatrix + k * kPlane, res + e, bytes);
                if (gated) cp_async16_part(dst + gate_at + k * kPlane, gate + e, bytes);
            }
        }
        cp_async_commit();
    };
    // without a ring: the unit at element e (column c of its row) from memory
    auto load = [&](const raw *m, long long e, int c) {
        if constexpr (kEl) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[j] = 0;
                if (c + 32 * j < width) {
                    if constexpr (sizeof(raw) == 2) w[j] = __float_as_uint(A::up(m[e + 32 * j]));
                    else w[j] = __float_as_uint(m[e + 32 * j]);
                }
            }
            return make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            if (KIND == kFull || e + N <= end) return *reinterpret_cast<const uint4 *>(m + e);
            uint4 w = make_uint4(0, 0, 0, 0);
            for (int j = 0; e + j < end; ++j) reinterpret_cast<raw *>(&w)[j] = m[e + j];
            return w;
        }
    };
    auto up = [&](const uint4 &w, float2 (&v)[H]) {
        if constexpr (kEl) {
            v[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
            v[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
        } else {
            U::up(w, v);
        }
    };
    // clears what is not in the row; c: column of the unit's first element
    auto mask = [&](int c, float2 (&v)[H]) {
        if (KIND != kBlocks || (c >= 0 && c + N <= width)) return;
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (c + j < 0 || c + j >= width) (j & 1 ? v[j / 2].y : v[j / 2].x) = 0.f;
    };
    // e: the unit's first element in the matrix
    auto store = [&](raw *m, long long e, int c, const float2 (&v)[H]) {
        if constexpr (kEl) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + 32 * j < width) m[e + 32 * j] = A::down(j & 1 ? v[j / 2].y : v[j / 2].x);
        } else if (KIND == kFull || (c >= 0 && c + N <= width)) {
            *reinterpret_cast<uint4 *>(m + e) = U::down(v);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (c + j >= 0 && c + j < width) m[e + j] = A::down(j & 1 ? v[j / 2].y : v[j / 2].x);
        }
    };
    auto store8 = [&](long long e, int c, const float2 (&v)[H]) {
        uint8_t *m = static_cast<uint8_t *>(p.out) + e;
        if constexpr (kEl) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + 32 * j < width) m[32 * j] = to_e4m3(j & 1 ? v[j / 2].y : v[j / 2].x);
        } else if (KIND == kFull || (c >= 0 && c + N <= width)) {
            U::store8(m, v);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (c + j >= 0 && c + j < width) m[j] = to_e4m3(j & 1 ? v[j / 2].y : v[j / 2].x);
        }
    };
    auto weigh = [&](int c, float2 (&w)[H]) {
        if constexpr (kShared) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                // the columns of one unit lie in one run of N (kFull), or in two
                const float f = KIND == kFull || (c + j >= 0 && c + j < width) ? weights[padded<N>(c + j)] : 0.f;
                (j & 1 ? w[j / 2].y : w[j / 2].x) = f;
            }
        } else {
            if (!kEl && !p.weight_f32 && (KIND == kFull || (!(c & (N - 1)) && c + N <= width))) {
                up(*reinterpret_cast<const uint4 *>(static_cast<const raw *>(p.weight) + c), w);
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int cc = kEl ? c + 32 * j : c + j;
                    float f;
                    if constexpr (sizeof(raw) == 2) f = cc >= 0 && cc < width ? weight_at(p, cc, kF16) : 0.f;
                    else f = cc >= 0 && cc < width ? static_cast<const float *>(p.weight)[cc] : 0.f;
                    (j & 1 ? w[j / 2].y : w[j / 2].x) = f;
                }
            }
#pragma unroll
            for (int j = 0; j < H; ++j) w[j] = fadd2(w[j], make_float2(p.weight_offset, p.weight_offset));
        }
    };

    // turns of the loop: the same for all threads of a warp; a group without a row left does the last turn on
    // nothing and writes nothing
    const int warp_first = first - (L < 32 ? ((int)threadIdx.x & 31) / L : 0);
    const int turns = warp_first >= rows ? 0 : (rows - 1 - warp_first) / stride + 1;
    if (kRing) fetch(0, first);
    if (kShared) {
        for (int c = threadIdx.x; c < width; c += kBlock) weights[padded<N>(c)] = weight_at(p, c, kF16) + p.weight_offset;
        __syncthreads();
    }
    for (int turn = 0; turn < turns; ++turn) {
        const int row = first + turn * stride;
        const bool live = row < rows;
        const int ph = phase(row);
        const long long at = (long long)row * width - ph + v0;
        const uint8_t *held = mine + (turn & 1) * stage_bytes;
        if (kRing) {
            fetch((turn + 1) & 1, row < rows - stride ? row + stride : rows);
            cp_async_wait<1>();
        }
        auto has = [&](int k) {
            if (KIND == kFull) return live;
            return live && (kEl ? v0 - (t & 31) + k * kStep < width : v0 + k * kStep - ph < width);
        };
        float2 z[NV][H], sum2 = make_float2(0.f, 0.f);
        constexpr int kBatch = kRing ? 1 : NV / 2;  // units in flight at a time where there is no ring
#pragma unroll
        for (int k0 = 0; k0 < NV; k0 += kBatch) {
            uint4 xw[kBatch], rw[kBatch];
            if (!kRing) {
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int k = k0 + i, c = v0 + k * kStep - ph;
                    if (!has(k)) continue;
                    xw[i] = load(x, at + k * kStep, c);
                    if (residual) rw[i] = load(res, at + k * kStep, c);
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int k = k0 + i, c = v0 + k * kStep - ph;
                if (!has(k)) continue;
                if (kRing) xw[i] = *reinterpret_cast<const uint4 *>(held + k * kPlane);
                up(xw[i], z[k]);
                if (residual) {
                    float2 r[H];
                    if (kRing) rw[i] = *reinterpret_cast<const uint4 *>(held + kMatrix + k * kPlane);
                    up(rw[i], r);
#pragma unroll
                    for (int j = 0; j < H; ++j) z[k][j] = fadd2(z[k][j], r[j]);
                    store(static_cast<raw *>(p.residual_out), at + k * kStep, c, z[k]);
                }
                mask(c, z[k]);
#pragma unroll
                for (int j = 0; j < H; ++j) sum2 = ffma2(z[k][j], z[k][j], sum2);
            }
        }
        float sum = lanes_sum<W>(sum2.x + sum2.y);
        if (L > 32) {
            if ((t & 31) == 0) red[0][t >> 5] = sum;
            __syncthreads();
            sum = lanes_sum<kWarps>(red[0][t & (kWarps - 1)]);
        }
        const float rstd = rsqrtf(fmaf(sum, p.inv_width, p.eps));

        float most = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = v0 + k * kStep - ph;
            const long long e = at + k * kStep;
            float m = 0.f;
            if (has(k)) {
                float2 w[H];
                weigh(c, w);
#pragma unroll
                for (int j = 0; j < H; ++j) z[k][j] = fmul2(fmul2(z[k][j], make_float2(rstd, rstd)), w[j]);
                if (gated) {
                    float2 g[H];
                    up(kRing ? *reinterpret_cast<const uint4 *>(held + gate_at + k * kPlane) : load(gate, e, c), g);
                    mask(c, g);
#pragma unroll
                    for (int j = 0; j < H; ++j) z[k][j] = fmul2(z[k][j], silu(g[j]));
                }
                if (quant == GDN_QUANT_NONE) store(static_cast<raw *>(p.out), e, c, z[k]);
                else {
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        // past the row's end a NaN of rstd must not reach a group's maximum
                        if (kEl && c + 32 * j >= width) continue;
                        m = absmax_nan(m, j & 1 ? z[k][j / 2].y : z[k][j / 2].x);
                    }
                }
            }
            if (quant == GDN_QUANT_BLOCK) {
                m = lanes_max<kGroupLanes < W ? kGroupLanes : W>(m);
                const float scale = absmax_nan(kMinScale, m * (1.f / kE4m3Max)), inv = __fdividef(1.f, scale);
                if (has(k)) {
#pragma unroll
                    for (int j = 0; j < H; ++j) z[k][j] = fmul2(z[k][j], make_float2(inv, inv));
                    store8(e, c, z[k]);
                    if ((t & (kGroupLanes - 1)) == 0)
                        p.scales[(long long)row * ((width + GDN_QUANT_GROUP - 1) / GDN_QUANT_GROUP) +
                                 c / GDN_QUANT_GROUP] = scale;
                }
            }
            most = absmax_nan(most, m);
        }
        if (quant == GDN_QUANT_ROW) {
            most = lanes_max<W>(most);
            if (L > 32) {
                if ((t & 31) == 0) red[1][t >> 5] = most;
                __syncthreads();
                most = lanes_max<kWarps>(red[1][t & (kWarps - 1)]);
            }
            const float scale = absmax_nan(kMinScale, most * (1.f / kE4m3Max)), inv = __fdividef(1.f, scale);
            if (live && t == 0) p.scales[row] = scale;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (!has(k)) continue;
#pragma unroll
                for (int j = 0; j < H; ++j) z[k][j] = fmul2(z[k][j], make_float2(inv, inv));
                store8(at + k * kStep, v0 + k * kStep - ph, z[k]);
            }
        } else if (L > 32) {
            __syncthreads();  // red[0] is read before the next row writes it
        }
    }
}

template <class A, Kind KIND, int L>
cudaError_t launch_kernel(const NormParams &p, cudaStream_t st)
{
    const auto kern = rms_norm_kernel<A, KIND, L>;
    constexpr int block = norm_block(L), rows = L <= 32 ? block / L : 1;
    const int matrices = 1 + (p.residual != nullptr) + (p.gate != nullptr);
    size_t smem = norm_ring(KIND, L) ? (size_t)2 * block * 32 * sizeof(typename A::raw) * matrices : 0;
    if (norm_weights(KIND, L)) smem += (padded<Unit<A>::N>(32 * L) * 4 + 15) / 16 * 16;
    if (smem > 47 * 1024) {  // 48 KB with the static part
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    const int per_sm = std::max(1, std::min(norm_ctas(L), (int)(kNormSmem / (smem + 1280))));
    const long long want = (p.rows + rows - 1) / rows;
    kern<<<(unsigned)std::min<long long>(want, (long long)kNormSms * per_sm), block, smem, st>>>(p);
    return cudaGetLastError();
}

// The threads of a row: as few as hold `places` places, 32 each, and at least `least`.
template <class A, Kind KIND>
cudaError_t launch_lanes(const NormParams &p, int places, int least, cudaStream_t st)
{
    const int lanes = std::max(least, (places + 31) / 32);
    if (KIND != kElements) {
        if (lanes <= 4) return launch_kernel<A, KIND == kElements ? kFull : KIND, 4>(p, st);
        if (lanes <= 8) return launch_kernel<A, KIND == kElements ? kFull : KIND, 8>(p, st);
        if (lanes <= 16) return launch_kernel<A, KIND == kElements ? kFull : KIND, 16>(p, st);
        if (lanes > 32 && lanes <= 64) return launch_kernel<A, KIND == kElements ? kFull : KIND, 64>(p, st);
        if (lanes > 128 && lanes <= 256) return launch_kernel<A, KIND == kElements ? kFull : KIND, 256>(p, st);
    }
    if (lanes <= 32) return launch_kernel<A, KIND, 32>(p, st);
    if (lanes <= 128) return launch_kernel<A, KIND, 128>(p, st);
    if (lanes <= 512) return launch_kernel<A, KIND, 512>(p, st);
    return launch_kernel<A, KIND, 1024>(p, st);
}

template <class A>
cudaError_t launch_type(NormParams p, cudaStream_t st)
{
    constexpr int N = Unit<A>::N;
    const int width = p.width;
    if (p.quant == GDN_QUANT_BLOCK && width <= GDN_QUANT_GROUP) p.quant = GDN_QUANT_ROW;  // one group a row
    const int least = p.quant == GDN_QUANT_BLOCK ? 128 / N : 0;  // lanes that hold a group
    if (width % N == 0) {
        const bool full = width >= 128 && width <= 32768 && (width & (width - 1)) == 0 && width / 32 >= least;
        return full ? launch_lanes<A, kFull>(p, width, least, st) : launch_lanes<A, kBlocks>(p, width, least, st);
    }
    if (p.quant == GDN_QUANT_BLOCK) return launch_lanes<A, kElements>(p, width, 0, st);
    // a row that begins inside a block may take a unit more; the widest do not find room for it
    if (width + N - 1 > GDN_NORM_MAX_WIDTH) return launch_lanes<A, kElements>(p, width, 0, st);
    return launch_lanes<A, kBlocks>(p, width + N - 1, 0, st);
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
