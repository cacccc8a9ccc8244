// Attention of one new token of each sequence over a paged key/value cache (gdn_paged_attn_fwd):
//
//   s_j = scale q . k_j,  out = sum_j e^{s_j} v_j / sum_j e^{s_j},  lse = log sum_j e^{s_j}
//
// Every key and value is read from HBM once for each 16 of the G = Hq / Hkv query heads of its head (once up to G = 16,
// twice from 17 on): up to 16 flops a byte of a 16-bit cache, so the cache's bytes bound it, and the matrix
// products only have to keep up: mma.sync, which takes its operands from any shared-memory tile and leaves
// the softmax its scores in registers; one octet of query rows costs a sixth of the SM's time.
//
// The split.  The work is one list of units of 64 keys, ordered by sequence, then by key/value head
// (and group of 16 query heads), then along the keys.  The grid fills the GPU once and CTA i of C takes
// the i-th of C equal parts of the list, whatever the lengths are: a long sequence is cut over many
// CTAs, short ones share one.  Every CTA finds its part by a scan over the lengths, so nothing about them
// has to be known on the host.  A part covers the end of one (sequence, head) pair, whole pairs, and
// the beginning of another.  Whole pairs are written out; an incomplete one leaves its unnormalised sum,
// maximum and sum of exponentials in one of the CTA's two places in the workspace, and a second kernel
// joins a pair's pieces in their order, so the result does not depend on the order in which CTAs run.
//
// Short sequences (attn_plan) do without the list, the workspace and the second kernel: each pair is one
// cluster's, its keys cut over the cluster's CTAs, which join their results through distributed shared
// memory.
//
// Inside a CTA the warps take tiles of 16 or 32 keys in turn.  A warp is on its own until the end of the
// piece: its own ring of tiles in shared memory, filled by cp.async a few tiles ahead, its own running
// maximum, sum and output accumulators (fp32, in registers), no CTA barrier.  At the end of a piece the
// warps' results are joined through shared memory, while the next piece's tiles are on their way.
//
// Roundings.  Scores, exponentials, sums and outputs are fp32.  An exponential's argument is a score's distance from the
// maximum, times scale log2 e: the maximum's own is exactly 0 however large the scores are.  (A fused score * scale - ref
// is off by up to |ref| 2^-24 there, which leaves the range of an exponent from |ref| of 2^31 on.)  The
// probabilities enter their product with V as a pair of 16-bit numbers, p = hi + lo: one rounded number would put an error
// as large as the output's own rounding into it, and the second product costs nothing beside the memory traffic.  In bf16
// the pair holds 16 bits or more of p, whatever its size.  fp16 ends at 2^-24, so there every weight is 2^15 p (kRaise; up
// to 32768), and the pair is good to 22 bits or 2^-25, which is 2^-40 of the largest weight: 16 bits of a key that lies 16.6
// nats below the largest score, 11 bits at 20.  The sum of exponentials takes them unrounded, so lse is good to fp32.  The
// tensor core cuts off what an addition to its accumulator drops
// (up to 2^-23 of the accumulator, always towards zero), so no more than 512 additions (256 tiles of 16 keys) go to one: a
// piece of the list ends after kMostKeys keys, and the CTA adds its pieces of a pair up in fp32, rounded; a cluster's CTA that
// gets more keys than its hint said sums a tile's products on their own and adds them so.  (300 rows over 131072 keys of
// positive values, D = 256: on average 8e-5 too small, without that 3.2e-4; over 10^6 keys, D = 128, 4e-5 against 1.5e-3.)
//
// Measured (bf16): 256 sequences of 1024 to 16384 keys, 16 / 2 heads of 256: 698 us, 6.75 TB/s (a read-only stream
// passes the copy rate); 64 of 1 to 8192 keys, 32 / 8 heads of 128: 172 us, 6.4 TB/s; one of 131072 keys, 16 / 2
// heads of 256: 52 us, 5.2 TB/s, 8 us of them the start, the CTAs' uneven end and the join; one of 700 keys: 7.5 us.
#include <algorithm>

#include "gdn_layers.h"
#include "layers.cuh"

namespace gdn {

namespace {

constexpr float kLn2 = 0.693147181f;

// NT: octets of query rows (1 or 2).  A warp's ring of 256-column tiles takes 48 KB: two CTAs of two warps an SM
// where the CTAs fill the GPU, one of four where short sequences leave room (DIRECT).
template <int D, int NT, bool DIRECT>
struct Shape {
    static constexpr int kWarps = D == 256 && !DIRECT ? 2 : 4, kThreads = 32 * kWarps;
    static constexpr int kTile = D == 64 ? 32 : 16;  // keys a warp takes at a time: 16 narrow ones are too little work
    static constexpr int kSteps = kTile / 16;        // for what a tile costs beside them (16 sequences of 8 heads, up
                                                     // to 8000 keys: 39 us with 16, 36 us with 32)
    static constexpr int kCtas = DIRECT ? kDirectCtasPerSm(D) : kAttnCtasPerSm;
    static constexpr int kChain = 256 / kSteps;      // tiles whose products go to one accumulator
    static constexpr int kStages = 3;
    static constexpr int kHalf = kTile * D * 2;      // bytes of a tile's keys (or values)
    static constexpr int kStage = 2 * kHalf;
    static constexpr int kRing = kStages * kStage;   // per warp
    static constexpr int kRows = 8 * NT;
    static constexpr int kQ = kRows * D * 2;         // query rows, behind the rings
    static constexpr int kSmem = kWarps * kRing + kQ;
    static constexpr bool kQInRegs = D * NT < 512;   // query fragments stay in registers
    static_assert(kStage >= kRows * D * 4, "a warp's sums fit into a stage");
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

__device__ __forceinline__ void ldsm_x2(uint32_t addr, uint32_t &r0, uint32_t &r1)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];\n" : "=r"(r0), "=r"(r1) : "r"(addr));
}

// 2^x to 2^-22, relative; below 2^-126 zero
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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

// where a CTA's part of the list begins, and the list's length
struct Part {
    long long first, last, total;  // the part's first place, and the one behind it
    int ctas;        // CTAs that have a part: the grid, or fewer where there are fewer places (so that no part in
                     // between is empty and a pair's pieces lie in neighbouring CTAs)
    int b, n;        // sequence of the first place, and its length
    int pair, u0;    // head group of the first place, and its number there
};

// All threads call it.  Thread t sums the places of its run of sequences; a scan over the threads finds the
// run that holds the CTA's first place, and the run's thread the sequence.
template <int D, int kThreads>
__device__ __forceinline__ void find_part(const AttnParams &p, Part &found)  // (in shared memory)
{
    constexpr int kWarps = kThreads / 32;
    __shared__ long long warp_total[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int run = (p.B + kThreads - 1) / kThreads, b0 = min(tid * run, p.B), b1 = min(b0 + run, p.B);
    const int heads = p.Hkv * p.row_tiles;
    long long mine = 0;
    int n = 0;
    for (int b = b1 - 1; b >= b0; --b) {
        n = p.lens[b];
        mine += attn_places(D, n, p.capacity);
    }
    long long upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += y;
    }
    if (lane == 31) warp_total[warp] = upto;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) upto += warp_total[w];
        total += warp_total[w];
    }
    total *= heads;
    const int ctas = (int)min(total, (long long)gridDim.x), i = blockIdx.x;
    const long long first = attn_part_begin(total, i, ctas);  // past the list for a CTA without a part
    const long long begin = (upto - mine) * heads;
    if (first >= begin && first < upto * heads) {
        long long rest = first - begin;  // places before the first in the run, then in its sequence
        int b = b0, each;
        for (;; n = p.lens[++b]) {  // n: the length of sequence b
            each = attn_places(D, n, p.capacity);
            if (rest < (long long)each * heads) break;
            rest -= (long long)each * heads;
        }
        const int pair = rest < (1LL << 31) ? (int)((uint32_t)rest / (uint32_t)each) : (int)(rest / each);
        found = Part{first, attn_part_begin(total, i + 1, ctas), total, ctas, b, n, pair, (int)(rest - (long long)pair * each)};
    }
    if (tid == 0 && i >= ctas) found.ctas = ctas;
    __syncthreads();
}

__device__ __forceinline__ void cluster_arrive_wait()
{
    asm volatile("barrier.cluster.arrive;\nbarrier.cluster.wait;" ::: "memory");
}
// the address of shared-memory address a in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t in_cta(uint32_t a, int rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t a)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ float2 cluster_load2(uint32_t a)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
    return v;
}

// the power of two that weights (and with them sums of weights and of values) are raised by
template <bool F16>
constexpr float kRaise = F16 ? 15.f : 0.f;

// 4 columns from 4 c on of one query head's output, x unnormalised, and its lse; top: the maximum, unscaled
template <int D, bool F16>
__device__ __forceinline__ void write_out(const AttnParams &p, long long head, int c, float4 x, float top, float sum)
{
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + head * D + 4 * c) =
        make_uint2(pack2<F16>(x.x * inv, x.y * inv), pack2<F16>(x.z * inv, x.w * inv));
    if (p.lse && c == 0) p.lse[head] = sum == 0.f ? -INFINITY : kLn2 * fmaf(top, p.scale_log2, log2f(sum) - kRaise<F16>);
}

// One piece of a CTA's work: keys [k0, k1) of head group `pair` of sequence b (of the list, `take` places from u0
// on), and how many places of the CTA's part lie behind it.  `from`: the place at which the CTA began the pair, before u0
// where the pair's keys are more than one piece here.
template <int D>
constexpr int kMostKeys = D == 256 ? 8192 : 16384;  // 512 additions to an accumulator in 2 (4) warps
struct Piece {
    int b, pair, n, n_next;  // n: the sequence's length as given, n_next: of the sequence behind it
    int u0, take, k0, k1, from;
    long long left;
};
template <int D>
__device__ __forceinline__ void cut(Piece &c, const AttnParams &p)  // the piece that begins at u0
{
    c.take = (int)min(c.left, (long long)min(kMostKeys<D> / kAttnUnit, attn_places(D, c.n, p.capacity) - c.u0));
    c.left -= c.take;
    const KeyRange k = attn_keys(D, c.u0, c.take, attn_refused(c.n, p.capacity) ? 0 : c.n);
    c.k0 = k.k0;
    c.k1 = k.k1;
}
template <int D>
__device__ __forceinline__ void next_piece(Piece &c, const AttnParams &p, int heads)
{
    c.u0 += c.take;
    if (c.u0 < attn_places(D, c.n, p.capacity)) {
        cut<D>(c, p);
        return;
    }
    c.u0 = c.from = 0;
    if (++c.pair == heads) {
        c.pair = 0;
        ++c.b;
        c.n = c.n_next;
        c.n_next = c.b + 1 < p.B ? p.lens[c.b + 1] : 0;
    }
    cut<D>(c, p);
}

// DIRECT: a cluster of p.direct CTAs a pair, one piece a CTA.  Otherwise the pieces of the CTA's part of the list, one
// behind the other: a warp's ring runs on over their borders (it fetches the next piece's tiles while it works on
// this one's), and only the join of the warps at a piece's end stops the CTA.
template <int D, int NT, bool F16, bool DIRECT>
__global__ void __launch_bounds__(Shape<D, NT, DIRECT>::kThreads, Shape<D, NT, DIRECT>::kCtas)
    paged_attn_kernel(const AttnParams p)
{
    using S = Shape<D, NT, DIRECT>;
    constexpr int kWarps = S::kWarps, kThreads = S::kThreads, kRows = S::kRows, kStages = S::kStages, kTile = S::kTile, kSteps = S::kSteps;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float wm[kWarps][kRows], wl[kWarps][kRows];
    __shared__ int wslot[kWarps];     // the stage that holds a warp's sums while the warps are joined
    __shared__ float2 joined[kRows];  // DIRECT: maximum and sum of this CTA's part of the keys
    __shared__ float2 carried[2][kRows];  // of the pair's pieces so far, to one half and from the other in turn
    begin_early();
    if (!DIRECT) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join's small CTAs
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t ring = smem_addr(smem) + warp * S::kRing;
    const uint32_t qs = smem_addr(smem) + kWarps * S::kRing;
    const uint16_t *kc = static_cast<const uint16_t *>(p.k), *vc = static_cast<const uint16_t *>(p.v);
    const int heads = p.Hkv * p.row_tiles;

    Piece now;
    __shared__ Part part;
    const int rank = DIRECT ? (int)blockIdx.x % p.direct : 0;
    if (DIRECT) {
        const int at = (int)blockIdx.x / p.direct;
        now.b = at / heads;
        now.pair = at - now.b * heads;
        now.n = p.lens[now.b];
        const KeyRange k = attn_cluster_keys(rank, p.direct, attn_refused(now.n, p.capacity) ? 0 : now.n);
        now.k0 = k.k0;
        now.k1 = k.k1;
        now.left = now.n_next = now.u0 = now.take = now.from = 0;
    } else {
        find_part<D, kThreads>(p, part);
        if ((int)blockIdx.x >= part.ctas) {
            if (tid == 0) p.begun[blockIdx.x] = make_int4(0, 0, 0, 0);
            return;
        }
        now.b = part.b;
        now.pair = part.pair;
        now.n = part.n;
        now.n_next = now.b + 1 < p.B ? p.lens[now.b + 1] : 0;
        now.u0 = now.from = part.u0;
        now.left = part.last - part.first;
        cut<D>(now, p);
    }

    // this warp's tiles of a piece: those at k0 + kTile (warp + kWarps i)
    auto tiles_of = [&](const Piece &c) {
        const int tiles = (c.k1 - c.k0 + kTile - 1) / kTile;
        return tiles > warp ? (tiles - warp + kWarps - 1) / kWarps : 0;
    };
    // The next tile to be looked up: the i-th of piece `ahead`, of which this warp has `count`.
    Piece ahead = now;
    int i_ahead = 0, count = tiles_of(ahead), hkv_ahead = ahead.pair / p.row_tiles;
    const int32_t *table = p.table + (long long)ahead.b * p.max_pages;
    // A tile to be fetched: the cache row of its key (lane % kTile), -1 behind the piece's last key, -2 on a page outside
    // the cache; and its head, or -1 when there is none left.  It is looked up a tile ahead of its use.
    struct Tile {
        int row, hkv;
    };
    auto look_up = [&]() {
        while (i_ahead >= count && ahead.left > 0) {
            next_piece<D>(ahead, p, heads);
            i_ahead = 0;
            count = tiles_of(ahead);
            hkv_ahead = ahead.pair / p.row_tiles;
            table = p.table + (long long)ahead.b * p.max_pages;
        }
        Tile t = {-1, -1};
        if (i_ahead >= count) return t;
        t.hkv = hkv_ahead;
        const int j = ahead.k0 + kTile * (warp + kWarps * i_ahead) + (lane & (kTile - 1));
        if (j < ahead.k1) {
            t.row = attn_cache_row(table, j, p.by_page, p.page_size, p.P);
            if (t.row < 0) t.row = -2;
        }
        ++i_ahead;
        return t;
    };
    // Lane l copies 16-byte chunk l % kChunks of rows l / kChunks + i kLaneRows.  The row's low bits that the lane
    // sets and those that i sets are apart, so the chunk's place (sw) is an exclusive or with a constant.
    constexpr int kChunks = D / 8, kLaneRows = 32 / kChunks;
    const uint32_t lane_row = lane / kChunks, lane_at = lane_row * (D * 2), lane_x = ((lane % kChunks) ^ lane_row) << 4;
    const uint32_t row_bytes = p.Hkv * D * 2;
    const char *lane_k = reinterpret_cast<const char *>(kc) + (lane % kChunks) * 16;
    const char *lane_v = reinterpret_cast<const char *>(vc) + (lane % kChunks) * 16;
    uint32_t bad_pages = 0;  // a bit for each stage whose tile has one
    auto fetch = [&](int stage, const Tile &t) {
        if (t.hkv >= 0) {
            const uint32_t dst = ring + stage * S::kStage + lane_at, head = (uint32_t)t.hkv * (D * 2);
            const char *k = lane_k + head, *v = lane_v + head;
#pragma unroll
            for (int i = 0; i < kTile / kLaneRows; ++i) {
                const int rr = __shfl_sync(0xffffffffu, t.row, lane_row + i * kLaneRows);
                const uint64_t at = (uint64_t)(uint32_t)max(rr, 0) * row_bytes;
                const uint32_t to = dst + i * 512 + (lane_x ^ (((i * kLaneRows) & 7) << 4));
                cp_async16(to, k + at, rr >= 0);
                cp_async16(to + S::kHalf, v + at, rr >= 0);
            }
            const uint32_t bad = __any_sync(0xffffffffu, t.row == -2);
            bad_pages = (bad_pages & ~(1u << stage)) | bad << stage;
        }
        cp_async_commit();
    };
    // A thread's 16-byte parts of a piece's query rows (rows past the group's zero)
    constexpr int kParts = (kRows * (D / 8) + kThreads - 1) / kThreads;
    auto read_queries = [&](uint4 (&x)[kParts], const Piece &c) {
        const int hkv = c.pair / p.row_tiles, row0 = (c.pair - hkv * p.row_tiles) * kRows;
        const uint16_t *q = static_cast<const uint16_t *>(p.q) + ((long long)c.b * p.Hq + hkv * p.group + row0) * D;
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            const int id = tid + i * kThreads, r = id / (D / 8), ch = id % (D / 8);
            x[i] = make_uint4(0, 0, 0, 0);
            if (r < min(kRows, p.group - row0)) x[i] = reinterpret_cast<const uint4 *>(q + (long long)r * D)[ch];
        }
    };
    auto keep_queries = [&](const uint4 (&x)[kParts]) {
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            const int id = tid + i * kThreads, r = id / (D / 8), ch = id % (D / 8);
            if (r < kRows) *reinterpret_cast<uint4 *>(smem + kWarps * S::kRing + sw<D>(r, ch)) = x[i];
        }
    };

    // the first tiles are on their way before the queries are waited for
    Tile tile;
    {
        Tile t[kStages - 1];
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) t[i] = look_up();
        tile = look_up();
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) fetch(i, t[i]);
    }
    {
        uint4 x[kParts];
        read_queries(x, now);
        keep_queries(x);
    }
    __syncthreads();

    auto query = [&](int k, uint32_t (&a)[4]) {  // 16 columns of the query rows (rows 8 .. 15 zero when NT is 1)
        if (NT == 2) ldsm_x4(qs + sw<D>(lane & 15, 2 * k + (lane >> 4)), a[0], a[1], a[2], a[3]);
        else {
            ldsm_x2(qs + sw<D>(lane & 7, 2 * k + ((lane >> 3) & 1)), a[0], a[2]);
            a[1] = a[3] = 0;
        }
    };

    int stage = 0;  // of this warp's next tile; the one before it is free
    int turn = 0;   // of the halves of `carried`
    for (;;) {
        const int hkv = now.pair / p.row_tiles, row0 = (now.pair - hkv * p.row_tiles) * kRows;
        const int rows = min(kRows, p.group - row0), head0 = hkv * p.group + row0;

        // o: the output transposed, o[t][r][e] at column 16 t + lane / 4 (+ 8 for e >= 2) of query row
        // 8 r + 2 (lane % 4) (+ 1 for odd e); m, l: of query row 8 r + lane / 4 (l this lane's part of the sum)
        float o[D / 16][NT][4], m[NT], l[NT];
#pragma unroll
        for (int r = 0; r < NT; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int t = 0; t < D / 16; ++t) o[t][r][0] = o[t][r][1] = o[t][r][2] = o[t][r][3] = 0.f;
        }
        uint32_t qf[S::kQInRegs ? D / 16 : 1][4];
        if (S::kQInRegs) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) query(k, qf[k]);
        }
        bool bad = attn_refused(now.n, p.capacity);

        const int mine = tiles_of(now);
        for (int i = 0; i < mine; ++i) {
            cp_async_wait<kStages - 2>();
            __syncwarp();
            fetch(stage == 0 ? kStages - 1 : stage - 1, tile);
            tile = look_up();
            const uint32_t ks = ring + stage * S::kStage, vs = ks + S::kHalf;
            bad |= bad_pages >> stage & 1;
            stage = stage + 1 == kStages ? 0 : stage + 1;

            // scores of the query rows against the tile's keys; with 16 of them even and odd steps apart, to halve the
            // chain of additions
            float s[2 * kSteps][4] = {}, s1[2][4] = {};
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                if (!S::kQInRegs) query(k, qf[0]);
                const uint32_t *a = qf[S::kQInRegs ? k : 0];
#pragma unroll
                for (int h = 0; h < kSteps; ++h) {
                    uint32_t b0, b1, b2, b3;
                    ldsm_x4(ks + sw<D>(16 * h + (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)), b0, b1,
                            b2, b3);
                    mma<F16>(kSteps == 1 && k & 1 ? s1[0] : s[2 * h], a, b0, b1);
                    mma<F16>(kSteps == 1 && k & 1 ? s1[1] : s[2 * h + 1], a, b2, b3);
                }
            }
            if (kSteps == 1) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 2 * NT; ++e) s[t][e] += s1[t][e];
            }
            const int left = now.k1 - (now.k0 + kTile * (warp + kWarps * i));  // keys of this tile (1 .. kTile, or more)
            if (left < kTile) {
#pragma unroll
                for (int t = 0; t < 2 * kSteps; ++t)
#pragma unroll
                    for (int e = 0; e < 2 * NT; ++e)
                        if (8 * t + 2 * (lane & 3) + (e & 1) >= left) s[t][e] = -INFINITY;
            }
            float alpha[NT], ref[NT];  // maxima are of the scores as they are (the scale is positive)
            bool moved = false;
#pragma unroll
            for (int r = 0; r < NT; ++r) {
                float top = -INFINITY;
#pragma unroll
                for (int t = 0; t < 2 * kSteps; ++t) top = fmaxf(top, fmaxf(s[t][2 * r], s[t][2 * r + 1]));
                const float most = fmaxf(m[r], quad_max(top));
                ref[r] = most == -INFINITY ? 0.f : most;  // every score -infinity so far: the exponentials are 0
                alpha[r] = ex2((m[r] - ref[r]) * p.scale_log2);
                moved |= alpha[r] != 1.f;
                m[r] = most;
                l[r] *= alpha[r];
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int r = 0; r < NT; ++r) {
                    const float a0 = __shfl_sync(0xffffffffu, alpha[r], 8 * (lane & 3));
                    const float a1 = __shfl_sync(0xffffffffu, alpha[r], 8 * (lane & 3) + 4);
#pragma unroll
                    for (int t = 0; t < D / 16; ++t) {
                        o[t][r][0] *= a0;
                        o[t][r][1] *= a1;
                        o[t][r][2] *= a0;
                        o[t][r][3] *= a1;
                    }
                }
            }
            // The scores' fragment (query row lane / 4, keys 2 (lane % 4) + ..) is, packed, the second operand of
            // V^T P^T (its column lane / 4, its rows 2 (lane % 4) + ..): no exchange between lanes.
            uint32_t hi[NT][2 * kSteps], lo[NT][2 * kSteps];
#pragma unroll
            for (int r = 0; r < NT; ++r)
#pragma unroll
                for (int t = 0; t < 2 * kSteps; ++t) {
                    const float2 below = fadd2(make_float2(s[t][2 * r], s[t][2 * r + 1]), make_float2(-ref[r], -ref[r]));
                    const float2 scale = make_float2(p.scale_log2, p.scale_log2);
                    const float2 x = F16 ? ffma2(below, scale, make_float2(kRaise<F16>, kRaise<F16>)) : fmul2(below, scale);
                    const float p0 = ex2(x.x), p1 = ex2(x.y);
                    l[r] += p0 + p1;
                    split2<F16>(p0, p1, hi[r][t], lo[r][t]);
                }
            // 16 columns of the output
            auto add_products = [&](int t, float (&x)[NT][4]) {
#pragma unroll
                for (int h = 0; h < kSteps; ++h) {
                    uint32_t a[4];
                    ldsm_x4_t(vs + sw<D>(16 * h + (lane & 7) + ((lane >> 4) << 3), 2 * t + ((lane >> 3) & 1)), a[0],
                              a[1], a[2], a[3]);
#pragma unroll
                    for (int r = 0; r < NT; ++r) mma<F16>(x[r], a, hi[r][2 * h], hi[r][2 * h + 1]);
#pragma unroll
                    for (int r = 0; r < NT; ++r) mma<F16>(x[r], a, lo[r][2 * h], lo[r][2 * h + 1]);
                }
            };
            if (!DIRECT || __builtin_expect(mine <= S::kChain, 1)) {
#pragma unroll
                for (int t = 0; t < D / 16; ++t) add_products(t, o[t]);
            } else {
#pragma unroll
                for (int t = 0; t < D / 16; ++t) {
                    float x[NT][4] = {};
                    add_products(t, x);
#pragma unroll
                    for (int r = 0; r < NT; ++r)
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            const float2 sum = fadd2(make_float2(o[t][r][e], o[t][r][e + 1]), make_float2(x[r][e], x[r][e + 1]));
                            o[t][r][e] = sum.x;
                            o[t][r][e + 1] = sum.y;
                        }
                }
            }
        }

        const int all = DIRECT ? 0 : attn_places(D, now.n, p.capacity);
        // the CTA's last piece of the pair; all of the pair in this CTA; pieces of the pair before this one
        const bool done = DIRECT || now.left == 0 || now.u0 + now.take == all;
        const bool whole = DIRECT ? p.direct == 1 : now.from == 0 && now.u0 + now.take == all;
        const bool carries = !DIRECT && now.u0 != now.from;

        // The end of the piece: join the warps.  A warp's sums go to its free stage; the next piece's queries are on
        // their way meanwhile.
        const bool last = DIRECT || now.left == 0;
        Piece next = now;
        uint4 x_next[kParts];
        if (!last) {
            next_piece<D>(next, p, heads);
            read_queries(x_next, next);
        }
        if (bad) {
#pragma unroll
            for (int r = 0; r < NT; ++r) l[r] = NAN;
        }
#pragma unroll
        for (int r = 0; r < NT; ++r) {
            l[r] = quad_sum(l[r]);
            if ((lane & 3) == 0) {
                wm[warp][lane / 4 + 8 * r] = m[r];
                wl[warp][lane / 4 + 8 * r] = l[r];
            }
        }
        // DIRECT: no copy is on its way any more, and the CTAs of a cluster have to agree on the stage
        const int slot = DIRECT || stage == 0 ? kStages - 1 : stage - 1;
        if (lane == 0) wslot[warp] = slot;
        if (DIRECT) cp_async_wait<0>();
        __syncthreads();
        // row `row`, column d of a warp's sums lies at row D + (d ^ 8 (row / 2 % 4)): the four rows that a quad writes
        // fall into different banks
        auto sums = [&](int w) { return reinterpret_cast<float *>(smem + w * S::kRing + wslot[w] * S::kStage); };
        auto swizzled = [](int row, int d) { return row * D + (d ^ (((row >> 1) & 3) << 3)); };
        auto top_of = [&](int row) {
            float top = wm[0][row];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) top = fmaxf(top, wm[w][row]);
            return top == -INFINITY ? 0.f : top;
        };
        float *os = sums(warp);
#pragma unroll
        for (int r = 0; r < NT; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = 8 * r + 2 * (lane & 3) + e;
                if (row >= rows) continue;
                const float f = ex2((wm[warp][row] - top_of(row)) * p.scale_log2);
#pragma unroll
                for (int t = 0; t < D / 16; ++t) {
                    os[swizzled(row, 16 * t + lane / 4)] = o[t][r][e] * f;
                    os[swizzled(row, 16 * t + lane / 4 + 8)] = o[t][r][2 + e] * f;
                }
            }
        if (!last) keep_queries(x_next);  // every warp is done with this piece's
        __syncthreads();
        for (int i = tid; i < rows * (D / 4); i += kThreads) {
            const int row = i / (D / 4), c = i % (D / 4), at = swizzled(row, 4 * c);
            float top = top_of(row);
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float4 y = *reinterpret_cast<const float4 *>(sums(w) + at);
                x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
                sum += wl[w][row] * ex2((wm[w][row] - top) * p.scale_log2);
            }
            // place 1: the pair begins here; place 0: it began in an earlier CTA.  (Place 1 is free while whole pairs carry
            // their sums there: the piece that it is for is the part's last.)
            const long long to = (2LL * blockIdx.x + (now.from == 0)) * 16 + row;
            float4 *const sum_at = reinterpret_cast<float4 *>(p.part + to * D) + c;  // (DIRECT: not used)
            if (carries) {
                const float2 ml = carried[turn][row];
                const float4 y = *sum_at;
                const float both = fmaxf(ml.x, sum == 0.f ? -INFINITY : top), ref = both == -INFINITY ? 0.f : both;
                const float f = sum == 0.f ? 0.f : ex2((top - ref) * p.scale_log2), g = ex2((ml.x - ref) * p.scale_log2);
                x.x = fmaf(y.x, g, x.x * f), x.y = fmaf(y.y, g, x.y * f);
                x.z = fmaf(y.z, g, x.z * f), x.w = fmaf(y.w, g, x.w * f);
                sum = fmaf(ml.y, g, sum * f);
                top = ref;
            }
            if (!done) {
                *sum_at = x;
                if (c == 0) carried[turn ^ 1][row] = make_float2(sum == 0.f ? -INFINITY : top, sum);
            } else if (whole) {
                write_out<D, F16>(p, (long long)now.b * p.Hq + head0 + row, c, x, top, sum);
            } else if (DIRECT) {
                *reinterpret_cast<float4 *>(sums(0) + at) = x;  // where this thread read the first warp's part
                if (c == 0) joined[row] = make_float2(sum == 0.f ? -INFINITY : top, sum);
            } else {
                // a piece without a weight has no maximum either: its stand-in 0 would drown scores far below it
                *sum_at = x;
                if (c == 0) p.part_ml[to] = make_float2(sum == 0.f ? -INFINITY : top, sum);
            }
        }
        if (DIRECT) {
            if (whole) return;
            cluster_arrive_wait();
            for (int i = rank * kThreads + tid; i < rows * (D / 4); i += p.direct * kThreads) {
                const int row = i / (D / 4), c = i % (D / 4);
                const uint32_t ml = smem_addr(joined + row), xs = smem_addr(sums(0) + swizzled(row, 4 * c));
                float2 part_ml[kAttnMaxCluster];
                float4 part_x[kAttnMaxCluster];
                float top = -INFINITY, sum = 0.f;
#pragma unroll
                for (int r = 0; r < kAttnMaxCluster; ++r) {
                    if (r >= p.direct) break;
                    part_ml[r] = cluster_load2(in_cta(ml, r));
                    part_x[r] = cluster_load4(in_cta(xs, r));
                }
#pragma unroll
                for (int r = 0; r < kAttnMaxCluster; ++r)
                    if (r < p.direct) top = fmaxf(top, part_ml[r].x);
                top = top == -INFINITY ? 0.f : top;
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int r = 0; r < kAttnMaxCluster; ++r) {
                    if (r >= p.direct) break;
                    const float w = ex2((part_ml[r].x - top) * p.scale_log2);
                    sum = fmaf(w, part_ml[r].y, sum);
                    x.x = fmaf(w, part_x[r].x, x.x), x.y = fmaf(w, part_x[r].y, x.y);
                    x.z = fmaf(w, part_x[r].z, x.z), x.w = fmaf(w, part_x[r].w, x.w);
                }
                write_out<D, F16>(p, (long long)now.b * p.Hq + head0 + row, c, x, top, sum);
            }
            cluster_arrive_wait();  // no CTA leaves while another reads its shared memory
            return;
        }
        if (last) {
            // a pair that begins here and goes on in other CTAs is the part's last; the CTA that holds its last place
            int4 begun = make_int4(0, 0, 0, 0);
            if (!whole && now.from == 0) {
                const int until = attn_part_of(part.total, part.last - (now.u0 + now.take) + all - 1, part.ctas);
                begun = make_int4(now.b, head0, rows, until - (int)blockIdx.x + 1);
            }
            if (tid == 0) p.begun[blockIdx.x] = begun;
            break;
        }
        turn ^= 1;
        now = next;
        __syncthreads();  // the free stages, wm, wl and wslot are free again
    }
    cp_async_wait<0>();
}

// Joins the pieces of every pair that a CTA of the first kernel began and did not finish: piece 0 lies in
// that CTA's place 1, piece j in place 0 of the j-th CTA after it.  Every CTA reads the list of such pairs;
// a query head of a pair of few pieces is one warp's work, of many pieces (a long sequence cut over the whole
// GPU) one CTA's for each 32 columns, its threads spread over the pieces.  Where a CTA (8K registers, 8 KB) finds room
// beside the first kernel's two on an SM, it lies there before that ends, and what is left behind its end is two
// loads, one waiting for the other: at D = 256, and at D = 64 with up to 8 query heads.  The others' registers (D = 128:
// 59K of 64K and more) let it in as their CTAs leave.
constexpr int kJoinThreads = 128, kJoinWarps = kJoinThreads / 32, kJoinCtas = 4 * kAttnSms, kFewPieces = 4;

template <int D, bool F16>
__global__ void __launch_bounds__(kJoinThreads, 8) paged_attn_join_kernel(const AttnParams p)
{
    constexpr int kBlock = 32, kBlocks = D / kBlock;                  // columns of a CTA's item, items of a row
    constexpr int kCols = kBlock / 4, kGroups = kJoinThreads / kCols;  // threads along the columns, along the pieces
    constexpr int kPer = (kAttnMaxCtas + kJoinThreads - 1) / kJoinThreads;  // records a thread takes
    __shared__ int4 list[kAttnMaxCtas];
    __shared__ uint32_t upto[kAttnMaxCtas], warp_total[kJoinWarps];  // many << 16 | few: items up to and with this one
    __shared__ float4 part[kGroups][kCols];
    __shared__ float2 part_ml[kGroups];
    // pieces that a thread reads at a time (131072 keys cut by 296 CTAs, 3, 5 and 8 at a time: one head of 256, 18.5 pieces a
    // thread, 35.9, 34.2, 35.2 us; two, 9.25, 53.1, 52.0, 53.0; four of 128, 4.6, 50.8, 50.5, 51.4; eight, 2.3, 88.7, 88.8, 89.8)
    constexpr int kInFlight = 5;
    begin_early();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t items[kPer], mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int at = tid * kPer + i;
        items[i] = 0;
        if (at < p.ctas) {
            const int4 r = p.begun[at];
            list[at] = r;
            if (r.w > 0) items[i] = r.w > kFewPieces ? (uint32_t)(r.z * kBlocks) << 16 : (uint32_t)r.z;
        }
        mine += items[i];
    }
    uint32_t run = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, run, d);
        if (lane >= d) run += y;
    }
    if (lane == 31) warp_total[warp] = run;
    __syncthreads();
    uint32_t total = 0;
    run -= mine;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        if (w < warp) run += warp_total[w];
        total += warp_total[w];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        run += items[i];
        if (tid * kPer + i < p.ctas) upto[tid * kPer + i] = run;
    }
    __syncthreads();
    const int many = total >> 16, few = total & 0xffff;
    // record that holds item `item` of a kind, and the item's number in it
    auto find = [&](int item, int shift, int *inner) {
        int lo = 0, hi = p.ctas - 1;  // smallest record whose running count exceeds the item
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if ((int)(upto[mid] >> shift & 0xffff) > item) hi = mid;
            else lo = mid + 1;
        }
        *inner = item - (lo ? (int)(upto[lo - 1] >> shift & 0xffff) : 0);
        return lo;
    };
    auto write = [&](const int4 &rec, int row, int c, float4 x, float top, float sum) {
        write_out<D, F16>(p, (long long)rec.x * p.Hq + rec.y + row, c, x, top, sum);
    };
    auto place = [&](int first, int j, int row) { return (2LL * (first + j) + (j == 0)) * 16 + row; };

    for (int item = warp * gridDim.x + blockIdx.x; item < few; item += gridDim.x * kJoinWarps) {
        int row;
        const int first = find(item, 0, &row);
        const int4 rec = list[first];
        float2 ml = make_float2(-INFINITY, 0.f);
        if (lane < rec.w) ml = p.part_ml[place(first, lane, row)];
        constexpr int kPerLane = (D / 4 + 31) / 32;  // columns (by fours) lane, lane + 32
        float4 y[kPerLane][kFewPieces];
#pragma unroll
        for (int i = 0; i < kPerLane; ++i)
#pragma unroll
            for (int j = 0; j < kFewPieces; ++j) {
                y[i][j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (j < rec.w && lane + 32 * i < D / 4)
                    y[i][j] = reinterpret_cast<const float4 *>(p.part + place(first, j, row) * D)[lane + 32 * i];
            }
        float top = ml.x;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        top = top == -INFINITY ? 0.f : top;
        const float w = ex2((ml.x - top) * p.scale_log2), sum = warp_sum(w * ml.y);
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int j = 0; j < kFewPieces; ++j) {
                const float wj = __shfl_sync(0xffffffffu, w, j);
                x.x = fmaf(wj, y[i][j].x, x.x), x.y = fmaf(wj, y[i][j].y, x.y);
                x.z = fmaf(wj, y[i][j].z, x.z), x.w = fmaf(wj, y[i][j].w, x.w);
            }
            if (lane + 32 * i < D / 4) write(rec, row, lane + 32 * i, x, top, sum);
        }
    }

    for (int item = blockIdx.x; item < many; item += gridDim.x) {
        int inner;
        const int first = find(item, 16, &inner), row = inner / kBlocks, block = inner % kBlocks;
        const int4 rec = list[first];
        const int count = rec.w;
        const int c = block * kCols + tid % kCols, g = tid / kCols;
        // this thread's pieces g, g + kGroups, ..: maxima, sums and columns in one go, joined as they come
        float top = -INFINITY, sum = 0.f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j0 = g; j0 < count; j0 += kGroups * kInFlight) {
            float2 ml[kInFlight];
            float4 y[kInFlight];
            float now = top;
#pragma unroll
            for (int i = 0; i < kInFlight; ++i) {
                const int j = j0 + i * kGroups;
                ml[i] = make_float2(-INFINITY, 0.f);
                y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (j < count) {
                    ml[i] = p.part_ml[place(first, j, row)];
                    y[i] = reinterpret_cast<const float4 *>(p.part + place(first, j, row) * D)[c];
                }
            }
#pragma unroll
            for (int i = 0; i < kInFlight; ++i) now = fmaxf(now, ml[i].x);
            const float ref = now == -INFINITY ? 0.f : now, keep = ex2((top - ref) * p.scale_log2);
            x.x *= keep, x.y *= keep, x.z *= keep, x.w *= keep, sum *= keep;
#pragma unroll
            for (int i = 0; i < kInFlight; ++i) {
                const float w = ex2((ml[i].x - ref) * p.scale_log2);
                sum = fmaf(w, ml[i].y, sum);
                x.x = fmaf(w, y[i].x, x.x), x.y = fmaf(w, y[i].y, x.y);
                x.z = fmaf(w, y[i].z, x.z), x.w = fmaf(w, y[i].w, x.w);
            }
            top = now;
        }
        part[g][tid % kCols] = x;
        if (tid % kCols == 0) part_ml[g] = make_float2(top, sum);
        __syncthreads();
        if (g == 0) {
            top = -INFINITY;
#pragma unroll
            for (int i = 0; i < kGroups; ++i) top = fmaxf(top, part_ml[i].x);
            top = top == -INFINITY ? 0.f : top;
            x = make_float4(0.f, 0.f, 0.f, 0.f), sum = 0.f;
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                const float4 y = part[i][tid];
                const float w = ex2((part_ml[i].x - top) * p.scale_log2);
                sum = fmaf(w, part_ml[i].y, sum);
                x.x = fmaf(w, y.x, x.x), x.y = fmaf(w, y.y, x.y), x.z = fmaf(w, y.z, x.z), x.w = fmaf(w, y.w, x.w);
            }
            write(rec, row, c, x, top, sum);
        }
        __syncthreads();
    }
}

template <int D, int NT, bool F16>
cudaError_t launch(const AttnParams &p, cudaStream_t st)
{
    if (p.direct) {
        using S = Shape<D, NT, true>;
        const auto kern = paged_attn_kernel<D, NT, F16, true>;
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        if (e != cudaSuccess) return e;
        return launch_early(kern, (unsigned)(p.B * p.Hkv * p.row_tiles * p.direct), S::kThreads, S::kSmem, st, p,
                            (unsigned)p.direct);
    }
    using S = Shape<D, NT, false>;
    const auto kern = paged_attn_kernel<D, NT, F16, false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_early(kern, (unsigned)p.ctas, S::kThreads, S::kSmem, st, p);
    if (e != cudaSuccess) return e;
    return launch_early(paged_attn_join_kernel<D, F16>, kJoinCtas, kJoinThreads, 0, st, p);
}

}  // namespace

// A cluster a pair where that leaves a CTA few keys; measured (us on the device, clusters against the list; a
// second figure: lengths from an eighth to the whole):
//   1 sequence of 2 heads, clusters of 8: D = 128, 1024 keys 6.7 / 8.5, 2048 keys (256 a CTA) 8.5 / 8.4, 4096 keys
//   11.9 / 9.0; D = 256, 1024 keys 10.0 / 12.8, 2048 keys 12.7 / 13.1, 4096 keys 17.8 / 13.8
//   4 sequences of 8 heads: D = 128, clusters of 8, 4096 keys (512 a CTA) 14.3, 13.1 / 18.1, 16.2; D = 256, clusters
//   of 4, 2048 keys (512) 18.0, 16.7 / 22.8, 19.7
//   64 sequences of 8 heads, more pairs than CTAs fit at once: D = 128, 512 keys 29, 20 / 33, 22, 1024 keys 49, 38 /
//   54, 35; D = 256, one CTA an SM, 64 keys 15 / 19, 256 keys 42, 30 / 36, 27
constexpr int kDirectKeys = 256, kDirectKeysMany = 512, kManyPairs = 16, kDirectKeysQueued = 64;
static_assert(kDirectKeysQueued >= kAttnUnit, "a list has two units or more");

AttnPlan attn_plan(int B, int Hq, int Hkv, int D, long long max_len)
{
    const long long pairs = (long long)B * Hkv * ((Hq / Hkv + 15) / 16), slots = kAttnSms * kDirectCtasPerSm(D);
    int cluster = 1;
    while (cluster < kAttnMaxCluster && pairs * cluster * 2 <= slots) cluster *= 2;
    const int keys = D == 256 && pairs > slots ? kDirectKeysQueued : pairs < kManyPairs ? kDirectKeys : kDirectKeysMany;
    if (max_len <= (long long)keys * cluster && pairs < (1 << 24)) return AttnPlan{0, cluster};
    const long long most = pairs * std::max(1LL, (max_len + kAttnUnit - 1) / kAttnUnit);  // (a table may have no columns)
    return AttnPlan{(int)std::min(most, (long long)kAttnSms * kAttnCtasPerSm), 0};
}

template <int D, bool F16>
cudaError_t launch_rows(const AttnParams &p, cudaStream_t st)
{
    return p.group <= 8 ? launch<D, 1, F16>(p, st) : launch<D, 2, F16>(p, st);
}

cudaError_t launch_paged_attn(const AttnParams &p, int D, bool f16, cudaStream_t st)
{
    switch (D) {
    case 64: return f16 ? launch_rows<64, true>(p, st) : launch_rows<64, false>(p, st);
    case 128: return f16 ? launch_rows<128, true>(p, st) : launch_rows<128, false>(p, st);
    default: return f16 ? launch_rows<256, true>(p, st) : launch_rows<256, false>(p, st);
    }
}

}  // namespace gdn
