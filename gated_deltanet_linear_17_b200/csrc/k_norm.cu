// Root-mean-square norm of rows, with the residual's addition, the SiLU gate of a delta-rule
// layer's output and an 8-bit output with scales (gdn_rms_norm):
//
//   z = x + residual,  y = z rstd (w + w0) [gate / (1 + e^-gate)],  rstd = 1 / sqrt(mean(z^2) + eps)
//
// About 10 flops an element, so HBM bounds it: every matrix is read once and written once.  A row
// stays in registers between its sum of squares and its output (z in fp32, the gate as it lies in
// memory), held by a group of lanes of one warp (rows up to 1024 columns: the row's sum is a few
// shuffles, no barrier) or by a CTA (up to 32768).
//
// Two layouts.  Rows whose width is a multiple of 8 take 8 neighbouring columns a lane (16-byte
// accesses of a 16-bit type); 16 neighbouring lanes then hold one group of 128 columns, and a
// group's maximum is four shuffles.  Any other width (rows that start at any element) takes
// element accesses: a warp holds groups of 128 columns, lane l the columns l, l + 32, l + 64, l + 96.
#include "gdn_layers.h"
#include "layers.cuh"

namespace gdn {

namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126: keeps 1 / scale finite for an all-zero row

__device__ __forceinline__ float silu(float g) { return __fdividef(g, 1.f + __expf(-g)); }

template <int N>
__device__ __forceinline__ float group_sum(float x)
{
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ float lanes_sum(float x, int lanes)
{
    for (int o = lanes >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ float lanes_max(float x, int lanes)
{
    for (int o = lanes >> 1; o > 0; o >>= 1) x = absmax_nan(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

// One lane's part of a row: NV units of 8 neighbouring columns (VECT) or of 4 columns 32 apart.
template <class A, bool VECT>
struct Unit;
template <class A>
struct Unit<A, true> {
    static constexpr int N = 8;
    using raw = typename A::raw;
    Raw8<A> r;
    static __device__ __forceinline__ int column(int k, int lane, int lanes) { return (lane + k * lanes) * 8; }
    __device__ __forceinline__ void load(const raw *row, int c, int) { r.load(row + c); }
    __device__ __forceinline__ void up(float (&x)[8]) const { r.up(x); }
    static __device__ __forceinline__ void store(raw *row, int c, int, const float (&x)[8])
    {
        Raw8<A> o;
        o.down(x);
        o.store(row + c);
    }
    static __device__ __forceinline__ void store8(uint8_t *row, int c, int, const float (&x)[8])
    {
        *reinterpret_cast<uint2 *>(row + c) =
            make_uint2(pack_e4m3(x[0], x[1], x[2], x[3]), pack_e4m3(x[4], x[5], x[6], x[7]));
    }
    static __device__ __forceinline__ bool has(int c, int, int width) { return c < width; }
    static constexpr int kGroupLanes = 16;  // lanes that hold one group of 128 columns
};
template <class A>
struct Unit<A, false> {
    static constexpr int N = 4;
    using raw = typename A::raw;
    raw r[4];
    static __device__ __forceinline__ int column(int k, int lane, int lanes)
    {
        return ((lane >> 5) + k * (lanes >> 5)) * 128 + (lane & 31);
    }
    __device__ __forceinline__ void load(const raw *row, int c, int width)
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = c + 32 * j < width ? row[c + 32 * j] : raw(0);
    }
    __device__ __forceinline__ void up(float (&x)[4]) const
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = A::up(r[j]);
    }
    static __device__ __forceinline__ void store(raw *row, int c, int width, const float (&x)[4])
    {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c + 32 * j < width) row[c + 32 * j] = A::down(x[j]);
    }
    static __device__ __forceinline__ void store8(uint8_t *row, int c, int width, const float (&x)[4])
    {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c + 32 * j < width) row[c + 32 * j] = to_e4m3(x[j]);
    }
    static __device__ __forceinline__ bool has(int c, int lane, int width) { return c - (lane & 31) < width; }
    static constexpr int kGroupLanes = 32;
};

// lanes: threads that share a row; a group of one warp's lanes (CTA = false; a power of two, 32 when
// !VECT) or the whole CTA (CTA = true).
template <class A, bool VECT, int NV, bool CTA, int QUANT>
__global__ void __launch_bounds__(CTA ? 512 : 256) rms_norm_kernel(const NormParams p, int lanes_log2)
{
    using U = Unit<A, VECT>;
    using raw = typename A::raw;
    constexpr int N = U::N;
    __shared__ float red[2][16];
    const int lanes = CTA ? (int)blockDim.x : 1 << lanes_log2;
    const int lane = CTA ? (int)threadIdx.x : (int)threadIdx.x & (lanes - 1);
    const int width = p.width;
    long long row = CTA ? blockIdx.x : (long long)blockIdx.x * (256 >> lanes_log2) + (threadIdx.x >> lanes_log2);
    const bool live = row < p.rows;
    if (!live) row = p.rows - 1;  // the lanes of a missing row follow the last one and write nothing
    const long long at = row * width;
    const raw *x = static_cast<const raw *>(p.x) + at;
    const raw *gate = p.gate ? static_cast<const raw *>(p.gate) + at : nullptr;

    float z[NV][N], sum = 0.f;
    U gr[NV];
    {
        U xr[NV], rr[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = U::column(k, lane, lanes);
            if (!U::has(c, lane, width)) continue;
            xr[k].load(x, c, width);
            if (p.residual) rr[k].load(static_cast<const raw *>(p.residual) + at, c, width);
            if (gate && NV <= 4) gr[k].load(gate, c, width);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = U::column(k, lane, lanes);
            if (!U::has(c, lane, width)) continue;
            xr[k].up(z[k]);
            if (p.residual) {
                float r[N];
                rr[k].up(r);
#pragma unroll
                for (int j = 0; j < N; ++j) z[k][j] += r[j];
                if (live) U::store(static_cast<raw *>(p.residual_out) + at, c, width, z[k]);
            }
#pragma unroll
            for (int j = 0; j < N; ++j) sum = fmaf(z[k][j], z[k][j], sum);
        }
    }
    sum = lanes_sum(sum, CTA ? 32 : lanes);
    if (CTA) {
        if ((threadIdx.x & 31) == 0) red[0][threadIdx.x >> 5] = sum;
        __syncthreads();
        sum = 0.f;
        for (int i = 0; i < lanes >> 5; ++i) sum += red[0][i];
    }
    const float rstd = 1.f / sqrtf(fmaf(sum, p.inv_width, p.eps));

    float most = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = U::column(k, lane, lanes);
        const bool has = U::has(c, lane, width);
        float m = 0.f;
        if (has) {
            float w[N], g[N];
            if (p.weight_f32) {
                Unit<F32, VECT> u;
                u.load(static_cast<const float *>(p.weight), c, width);
                u.up(w);
            } else {
                U u;
                u.load(static_cast<const raw *>(p.weight), c, width);
                u.up(w);
            }
            if (gate) {
                if (NV > 4) gr[k].load(gate, c, width);
                gr[k].up(g);
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                z[k][j] = z[k][j] * rstd * (w[j] + p.weight_offset);
                if (gate) z[k][j] *= silu(g[j]);
                // past the row's end (element accesses) a NaN of rstd or the gate must not reach the maximum
                if (VECT || c + 32 * j < width) m = absmax_nan(m, z[k][j]);
            }
            if (QUANT == GDN_QUANT_NONE && live) U::store(static_cast<raw *>(p.out) + at, c, width, z[k]);
        }
        if (QUANT == GDN_QUANT_BLOCK) {
            m = lanes_max(m, U::kGroupLanes);
            const float scale = absmax_nan(kMinScale, m * (1.f / kE4m3Max)), inv = 1.f / scale;
            if (has && live) {
#pragma unroll
                for (int j = 0; j < N; ++j) z[k][j] *= inv;
                U::store8(static_cast<uint8_t *>(p.out) + at, c, width, z[k]);
                if ((lane & (U::kGroupLanes - 1)) == 0)
                    p.scales[row * ((width + GDN_QUANT_GROUP - 1) / GDN_QUANT_GROUP) + c / GDN_QUANT_GROUP] = scale;
            }
        }
        most = absmax_nan(most, m);
    }
    if (QUANT == GDN_QUANT_ROW) {
        most = lanes_max(most, CTA ? 32 : lanes);
        if (CTA) {
            if ((threadIdx.x & 31) == 0) red[1][threadIdx.x >> 5] = most;
            __syncthreads();
            most = 0.f;
            for (int i = 0; i < lanes >> 5; ++i) most = absmax_nan(most, red[1][i]);
        }
        const float scale = absmax_nan(kMinScale, most * (1.f / kE4m3Max)), inv = 1.f / scale;
        if (live) {
            if (lane == 0) p.scales[row] = scale;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = U::column(k, lane, lanes);
                if (!U::has(c, lane, width)) continue;
#pragma unroll
                for (int j = 0; j < N; ++j) z[k][j] *= inv;
                U::store8(static_cast<uint8_t *>(p.out) + at, c, width, z[k]);
            }
        }
    }
}

template <class A, bool VECT, int NV, bool CTA>
cudaError_t launch_quant(const NormParams &p, int quant, int lanes, cudaStream_t st)
{
    int log2 = 0;
    while ((1 << log2) < lanes) ++log2;
    const unsigned grid = (unsigned)(CTA ? p.rows : (p.rows + (256 >> log2) - 1) / (256 >> log2));
    const unsigned block = CTA ? lanes : 256;
    switch (quant) {
    case GDN_QUANT_NONE: rms_norm_kernel<A, VECT, NV, CTA, GDN_QUANT_NONE><<<grid, block, 0, st>>>(p, log2); break;
    case GDN_QUANT_ROW: rms_norm_kernel<A, VECT, NV, CTA, GDN_QUANT_ROW><<<grid, block, 0, st>>>(p, log2); break;
    default: rms_norm_kernel<A, VECT, NV, CTA, GDN_QUANT_BLOCK><<<grid, block, 0, st>>>(p, log2); break;
    }
    return cudaGetLastError();
}

int ceil_div(int a, int b) { return (a + b - 1) / b; }
int round32(int a) { return ceil_div(a, 32) * 32; }

// The number of lanes and of units a lane holds, by the row's width.
template <class A>
cudaError_t launch_type(const NormParams &p, int quant, cudaStream_t st)
{
    if (p.width % 8 == 0) {
        const int units = p.width / 8;
        if (units <= 32) return launch_quant<A, true, 1, false>(p, quant, units <= 16 ? 16 : 32, st);
        if (units <= 128) return launch_quant<A, true, 4, false>(p, quant, 32, st);
        if (units <= 1024) return launch_quant<A, true, 2, true>(p, quant, round32(ceil_div(units, 2)), st);
        return launch_quant<A, true, 8, true>(p, quant, round32(ceil_div(units, 8)), st);
    }
    const int groups = ceil_div(p.width, 128);
    if (groups <= 4) return launch_quant<A, false, 4, false>(p, quant, 32, st);
    if (groups <= 64) return launch_quant<A, false, 4, true>(p, quant, 32 * ceil_div(groups, 4), st);
    return launch_quant<A, false, 16, true>(p, quant, 32 * ceil_div(groups, 16), st);
}

}  // namespace

cudaError_t launch_rms_norm(const NormParams &p, int act_dtype, int quant, cudaStream_t st)
{
    switch (act_dtype) {
    case GDN_DTYPE_BF16: return launch_type<Bf16>(p, quant, st);
    case GDN_DTYPE_FP16: return launch_type<F16>(p, quant, st);
    default: return launch_type<F32>(p, quant, st);
    }
}

}  // namespace gdn
