// Device helpers shared by the kernels of gdn_layers.h: 8-element accesses of the three
// activation types, and launches that overlap.
#pragma once

#include "common.cuh"
#include "layers.h"

namespace gdn {

// ---------------------------------------------------------------- launches that overlap their predecessor's end
// Every kernel of gdn_layers.h is launched with launch_early: its launch is prepared while the kernel before it in
// the stream ends, and begin_early waits, before the first access to memory, until that one is complete and its
// writes visible.  No kernel lets its successor's CTAs in before its own have left the SMs
// (griddepcontrol.launch_dependents), but for the paged attention its join: a grid cut to fill the GPU once finds
// no room for its last CTAs where a few that still run have broken up an SM's shared memory, and they start only
// when others end (37 ragged sequences 55 -> 80 us).
__device__ __forceinline__ void begin_early() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <class K, class P>
cudaError_t launch_early(K kernel, unsigned grid, unsigned block, size_t smem, cudaStream_t st, const P &p,
                         unsigned cluster = 1)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// ---------------------------------------------------------------- 8 elements at a time
// (16 bytes of a 16-bit type, 32 of fp32; the address is 16-byte aligned)
struct Bf16 {
    using raw = uint16_t;
    static __device__ __forceinline__ float up(uint16_t x) { return bf2f(x); }
    static __device__ __forceinline__ uint16_t down(float x) { return f2bf(x); }
    static __device__ __forceinline__ float2 up2(uint32_t w) { return unpack2<false>(w); }
    static __device__ __forceinline__ uint32_t down2(float a, float b) { return pack_bf2(a, b); }
};
struct F16 {
    using raw = uint16_t;
    static __device__ __forceinline__ float up(uint16_t x) { return __half2float(__ushort_as_half(x)); }
    static __device__ __forceinline__ uint16_t down(float x) { return __half_as_ushort(__float2half_rn(x)); }
    static __device__ __forceinline__ float2 up2(uint32_t w) { return unpack_h2(w); }
    static __device__ __forceinline__ uint32_t down2(float a, float b) { return pack_h2(a, b); }
};
struct F32 {
    using raw = float;
    static __device__ __forceinline__ float up(float x) { return x; }
    static __device__ __forceinline__ float down(float x) { return x; }
};

// the 8 elements as they lie in memory
template <class A>
struct Raw8 {
    uint4 w;
    __device__ __forceinline__ void load(const typename A::raw *p) { w = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void store(typename A::raw *p) const { *reinterpret_cast<uint4 *>(p) = w; }
    // the 8 elements that lane `from` holds
    __device__ __forceinline__ Raw8 shuffled(int from) const
    {
        Raw8 r;
        r.w.x = __shfl_sync(0xffffffffu, w.x, from);
        r.w.y = __shfl_sync(0xffffffffu, w.y, from);
        r.w.z = __shfl_sync(0xffffffffu, w.z, from);
        r.w.w = __shfl_sync(0xffffffffu, w.w, from);
        return r;
    }
    __device__ __forceinline__ void up2(float2 (&x)[4]) const
    {
        x[0] = A::up2(w.x), x[1] = A::up2(w.y), x[2] = A::up2(w.z), x[3] = A::up2(w.w);
    }
    __device__ __forceinline__ void down2(const float2 (&x)[4])
    {
        w = make_uint4(A::down2(x[0].x, x[0].y), A::down2(x[1].x, x[1].y), A::down2(x[2].x, x[2].y),
                       A::down2(x[3].x, x[3].y));
    }
};
template <>
struct Raw8<F32> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void store(float *p) const
    {
        reinterpret_cast<float4 *>(p)[0] = a;
        reinterpret_cast<float4 *>(p)[1] = b;
    }
    __device__ __forceinline__ Raw8 shuffled(int from) const
    {
        Raw8 r;
        r.a.x = __shfl_sync(0xffffffffu, a.x, from), r.a.y = __shfl_sync(0xffffffffu, a.y, from);
        r.a.z = __shfl_sync(0xffffffffu, a.z, from), r.a.w = __shfl_sync(0xffffffffu, a.w, from);
        r.b.x = __shfl_sync(0xffffffffu, b.x, from), r.b.y = __shfl_sync(0xffffffffu, b.y, from);
        r.b.z = __shfl_sync(0xffffffffu, b.z, from), r.b.w = __shfl_sync(0xffffffffu, b.w, from);
        return r;
    }
    __device__ __forceinline__ void up2(float2 (&x)[4]) const
    {
        x[0] = make_float2(a.x, a.y), x[1] = make_float2(a.z, a.w);
        x[2] = make_float2(b.x, b.y), x[3] = make_float2(b.z, b.w);
    }
    __device__ __forceinline__ void down2(const float2 (&x)[4])
    {
        a = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
        b = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
    }
};

// four floats -> four e4m3 bytes (nearest, halves to even, beyond 448 to 448, NaN kept), lowest byte first
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d)
{
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)hi << 16 | lo;
}
__device__ __forceinline__ uint8_t to_e4m3(float a) { return (uint8_t)(pack_e4m3(a, 0.f, 0.f, 0.f) & 0xff); }

}  // namespace gdn
