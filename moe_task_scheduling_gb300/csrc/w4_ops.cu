// w4_ops.cu -- products with 4-bit weights for a few rows (decoding), the
// routed SwiGLU experts over such weights, and the weights' own conversion.
//
//   w[n, k] = scale[k / group, n] * (q[n, k] - 8),  q in 0..15
//
// q is row-major, two inputs a byte (the even one in the low half); scale is
// bf16 with the group first, so that a tile of rows reads consecutive scales.
#include <cmath>
#include <type_traits>

#include "../../include/etmoe.h"
#include "et_api.h"
#include "ops_device.cuh"

namespace et {
namespace {

constexpr int kW4Rows = 64;        // weight rows of a warp (gate/up: 32 of each)
constexpr int kW4Blk = 128;        // inputs of a stage: 64 bytes of a row
constexpr int kW4Warps = 4;        // of a CTA; the down kernel takes twice as many where that evens its spread
constexpr int kW4WarpsMax = 8;
constexpr int kW4Stages = 2;       // k-blocks of a ring, one computed and one copied: three or four gained nothing (the
                                   // unpacking, not the memory, sets the pace) and took room from other CTAs
constexpr int kW4RowsMax = 64;     // most rows of x (tokens)
constexpr int kW4KMax = 8;         // experts of a token
constexpr int kW4EMax = 256;
constexpr int kW4ClusterMax = 8;
constexpr int kSmemSm = 228 * 1024;  // shared memory of an SM; each CTA takes 1 KB beside its own
constexpr int kW4Pad = kW4Rows + 8;  // row length of a warp's fp32 tile, padded against bank conflicts
constexpr int kW4RoutedMax = kW4RowsMax * kW4KMax;

enum W4Mode { kW4Gemv = 0, kW4GateUp = 1, kW4Down = 2, kW4GateUpAlone = 3, kW4DownAlone = 4 };
__host__ __device__ constexpr bool w4_is_alone(int mode) { return mode == kW4GateUpAlone || mode == kW4DownAlone; }

struct W4Args {
    const bf16* x;            // [rows, K]
    const uint8_t *q0, *q1;   // [E][N, K/2]; q1: the up projection
    const bf16 *s0, *s1;      // [E][K/group, N]
    bf16* out;                // [rows, N]
    float* y;                 // [T k, N]: a row's own output (kW4DownAlone)
    const int32_t* idx;       // [T, k]
    const float* w;           // [T, k]
    const int32_t* d_T;
    int T_host, T_max, N, K, E, k;
    EtHeader* hdr;
    int x_rows;               // rows of x a stage holds = most rows of a pass or segment
    int sum_rows;             // rows of a warp's fp32 tile: x_rows, or (down) the tokens
    uint32_t magic;           // 0x43004300 (see unpack8)
};

// Eight 4-bit values -> four packed pairs of q - 8 in bf16, pairs (0,4) (1,5)
// (2,6) (3,7).  0x4300 is 128.0 with a unit of 1 in its last place, so or-ing a
// nibble in gives 128 + q exactly, and taking 136 off is exact too: what is
// multiplied is the weight itself, so a large x whose weight is 0 adds nothing.
// (Summing (128 + q) x and taking 136 sum(x) off saved 4 % of the time -- T = 4,
// Mixtral-shaped, 111 us in place of 116 -- and left the rounding of 136 |x| in the
// sum.  A packed subtraction in place of the fma: 117.)  `magic` (0x43004300) comes
// from a kernel parameter, because a second constant known to the compiler makes
// and-or two operations instead of one.
__device__ __forceinline__ void unpack8(uint32_t v, uint32_t magic, uint32_t (&o)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t b;
        asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(b) : "r"(v >> (4 * i)), "r"(magic));
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(o[i]) : "r"(b), "r"(0x3f803f80u), "r"(0xc308c308u));  // b * 1 - 136
    }
}

// d = a b + c
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1, const float (&c)[4]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// A warp's part of a stage in shared memory: 64 rows of 64 bytes of weights,
// 128 / group rows of 64 scales; and the x rows (256 bytes each) that the RW
// warps of a k-split share.
struct W4Stage {
    uint8_t *w, *s, *x;
};

// The order of the inputs inside a group's products is free as long as weights
// and x agree.  Lane (r = lane / 4, t = lane % 4) takes G / 32 consecutive 32-bit
// words of a group of a row, one 4-, 8- or 16-byte read; the 16-byte pieces of
// weights (4 a row) and x (16 a row) are swizzled so that the lanes of each
// phase of these reads, and of the x reads, touch different banks.
template <int G>
__device__ __forceinline__ int swz_w(int piece, int row) {
    return G == 32 ? piece ^ ((row >> 1) & 3) : G == 64 ? piece ^ (row & 2) : piece;
}
template <int G>
__device__ __forceinline__ int swz_x(int piece, int row) {
    return G == 32 ? piece ^ ((row & 1) << 2) : G == 64 ? piece ^ (row & 1)
                                              : piece ^ ((piece >> 3) & 1) ^ ((row & 1) << 1);
}

template <int W>
__device__ __forceinline__ void ld_words(const uint8_t* a, uint32_t (&v)[W]) {
    if (W == 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(a);
        v[0] = u.x; v[1 % W] = u.y; v[2 % W] = u.z; v[3 % W] = u.w;
    } else if (W == 2) {
        const uint2 u = *reinterpret_cast<const uint2*>(a);
        v[0] = u.x; v[1 % W] = u.y;
    } else {
        v[0] = *reinterpret_cast<const uint32_t*>(a);
    }
}

// One k-block: acc += scale * sum((q - 8) x) over each group, the products exact,
// summed in fp32 by the tensor core, the scale applied in fp32 after it.
template <int NT, int G>
__device__ __forceinline__ void compute_stage(const W4Stage& st, int nc, uint32_t magic,
                                              float (&acc)[4][NT][4]) {
    constexpr int W = G / 32;  // words of a lane and row in a group
    const int lane = threadIdx.x & 31;
    const int r = lane >> 2, t = lane & 3;
    float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int g = 0; g < kW4Blk / G; ++g) {
        uint32_t b[W][NT][4];
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (j * 8 + r < nc) v = *reinterpret_cast<const uint4*>(st.x + (j * 8 + r) * 256 + (swz_x<G>(g * (G / 8) + t * W + i, r) << 4));
                b[i][j][0] = __byte_perm(v.x, v.z, 0x5410);
                b[i][j][1] = __byte_perm(v.x, v.z, 0x7632);
                b[i][j][2] = __byte_perm(v.y, v.w, 0x5410);
                b[i][j][3] = __byte_perm(v.y, v.w, 0x7632);
            }
        const __nv_bfloat16* sa = reinterpret_cast<const __nv_bfloat16*>(st.s + g * 128) + r;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            uint32_t lo[W], hi[W];
            float part[NT][4];
            const uint8_t* a = st.w + (m * 16 + r) * 64 + (swz_w<G>(g * (G / 32) + (t * W >> 2), r) << 4) + ((t * W & 3) << 2);
            ld_words<W>(a, lo);
            ld_words<W>(a + 512, hi);
            const float s0 = __bfloat162float(sa[m * 16]), s1 = __bfloat162float(sa[m * 16 + 8]);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                uint32_t u[4], v[4];
                unpack8(lo[i], magic, u);
                unpack8(hi[i], magic, v);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    mma16816(part[j], u[0], v[0], u[1], v[1], b[i][j][0], b[i][j][1], i == 0 ? zero : part[j]);
                    mma16816(part[j], u[2], v[2], u[3], v[3], b[i][j][2], b[i][j][3], part[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                acc[m][j][0] += s0 * part[j][0];
                acc[m][j][1] += s0 * part[j][1];
                acc[m][j][2] += s1 * part[j][2];
                acc[m][j][3] += s1 * part[j][3];
            }
        }
    }
}

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t v;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(v));
    return v;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t v;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(v));
    return v;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A float of the same shared address in CTA `rank` of the cluster.
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr, uint32_t rank) {
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// The routed rows of a call, grouped by expert, in shared memory.  Rows r = t k + j
// whose index is -1 are left out; an index outside [-1, E) is recorded and left out.
struct W4Routing {
    float* wt;          // [R] gate weight of an entry of `order`
    int16_t* order;     // [R] rows by expert, ascending within one
    int16_t* tok;       // [R] their tokens
    int16_t* seg_e;     // [R] segments: up to `width` rows of one expert: the expert,
    int16_t* seg_r;     // [R] its first entry in `order`,
    int16_t* seg_n;     // [R] its rows
    int16_t* e;         // [R] row -> expert (-1: none)
    int16_t* cnt;       // [W][E'] rows of an expert in a warp's share, then their first entry
    int* shared;        // [W + 2]: scan totals, n_seg, whether a token names an expert twice
    int Ep;             // E rounded up to even
    int n_seg, twice;

    __host__ __device__ static int bytes(int R, int E, int W) {
        return (R * 16 + W * ((E + 1) & ~1) * 2 + (W + 2) * 4 + 127) / 128 * 128;
    }
    template <int W>
    __device__ __forceinline__ void place(uint8_t* at, int R, int E) {
        wt = reinterpret_cast<float*>(at);
        shared = reinterpret_cast<int*>(wt + R);
        cnt = reinterpret_cast<int16_t*>(shared + W + 2);
        Ep = (E + 1) & ~1;
        order = cnt + W * Ep;
        tok = order + R;
        seg_e = tok + R;
        seg_r = seg_e + R;
        seg_n = seg_r + R;
        e = seg_n + R;
    }
};
static_assert(kW4Warps * 32 * 2 >= kW4EMax, "two experts a thread");
static_assert(kW4RoutedMax <= kW4Warps * 128, "four rows a thread");

// Up to 32 rows (decoding): one warp, experts in the order of their first row,
// one barrier.  More: all warps, experts ascending.
template <int W>
__device__ __forceinline__ void build_routing(const W4Args& p, W4Routing& rt, int T, int width) {
    const int R = T * p.k, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (R <= 32) {
        if (warp == 0) {
            int e = lane < R ? p.idx[lane] : -1;
            const float wt = lane < R ? p.w[lane] : 0.0f;
            if (e < -1 || e >= p.E) {
                record_status(p.hdr, ET_ERR_BOUNDS, kWhereExpertIndex);
                e = -1;
            }
            __syncwarp();
            const uint32_t same = __match_any_sync(0xffffffffu, e);
            const int before = __popc(same & ((1u << lane) - 1u)), c = __popc(same);
            const bool lead = e >= 0 && before == 0;
            const int v = lead ? c | ((c + width - 1) / width << 16) : 0;  // rows, segments
            int inc = v;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, inc, off);
                if (lane >= off) inc += up;
            }
            const int base = inc - v;
            const int r0 = __shfl_sync(0xffffffffu, base & 0xffff, __ffs(same) - 1);
            bool again = false;  // an earlier row of this token with this expert
            for (int o = 1; o < p.k; ++o) {
                const int other = __shfl_up_sync(0xffffffffu, e, o);
                again |= lane % p.k >= o && e >= 0 && other == e;
            }
            if (e >= 0) {
                rt.order[r0 + before] = static_cast<int16_t>(lane);
                rt.tok[r0 + before] = static_cast<int16_t>(lane / p.k);
                rt.wt[r0 + before] = wt;
            }
            if (lead) {
                int s0 = base >> 16;
                for (int o = 0; o < c; o += width, ++s0) {
                    rt.seg_e[s0] = static_cast<int16_t>(e);
                    rt.seg_r[s0] = static_cast<int16_t>(r0 + o);
                    rt.seg_n[s0] = static_cast<int16_t>(min(width, c - o));
                }
            }
            again = __any_sync(0xffffffffu, again);
            if (lane == 31) {
                rt.shared[W] = inc >> 16;
                rt.shared[W + 1] = again;
            }
        }
        __syncthreads();
        rt.n_seg = rt.shared[W];
        rt.twice = rt.shared[W + 1];
        return;
    }
    const int span = (R + W * 32 - 1) / (W * 32) * 32;  // consecutive rows of a warp
    int e[4], at[4];
    float wt[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = warp * span + i * 32 + lane;
        const bool in = i * 32 < span && r < R;
        e[i] = in ? p.idx[r] : -1;
        wt[i] = in ? p.w[r] : 0.0f;
    }
    for (int i = tid; i < W * rt.Ep / 2; i += blockDim.x) reinterpret_cast<int*>(rt.cnt)[i] = 0;
    if (tid == 0) rt.shared[W + 1] = 0;
    __syncthreads();
    // a row's place among its warp's rows of that expert
    int16_t* mine = rt.cnt + warp * rt.Ep;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i * 32 >= span) break;
        const int r = warp * span + i * 32 + lane;
        if (e[i] < -1 || e[i] >= p.E) {
            record_status(p.hdr, ET_ERR_BOUNDS, kWhereExpertIndex);
            e[i] = -1;
        }
        __syncwarp();
        const uint32_t same = __match_any_sync(0xffffffffu, e[i]);
        const int before = __popc(same & ((1u << lane) - 1u));
        int have = 0;
        if (e[i] >= 0) have = mine[e[i]];
        __syncwarp();
        if (e[i] >= 0 && before == 0) mine[e[i]] = static_cast<int16_t>(have + __popc(same));
        __syncwarp();
        at[i] = have + before;
        if (r < R) rt.e[r] = static_cast<int16_t>(e[i]);
    }
    __syncthreads();
    // exclusive sums over the experts, of rows (low half) and segments (high half)
    int c[2], v[2], sum = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int x = 2 * tid + h;
        c[h] = 0;
        if (x < p.E)
#pragma unroll
            for (int w = 0; w < W; ++w) c[h] += rt.cnt[w * rt.Ep + x];
        v[h] = c[h] | ((c[h] + width - 1) / width << 16);
        sum += v[h];
    }
    int inc = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += up;
    }
    if (lane == 31) rt.shared[warp] = inc;
    // a token's rows against its earlier ones
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = warp * span + i * 32 + lane;
        if (i * 32 < span && r < R && e[i] >= 0)
            for (int o = r - r % p.k; o < r; ++o)
                if (rt.e[o] == e[i]) rt.shared[W + 1] = 1;
    }
    __syncthreads();
    int base = inc - sum;
    for (int w = 0; w < warp; ++w) base += rt.shared[w];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int x = 2 * tid + h;
        if (c[h] > 0) {
            const int r0 = base & 0xffff;
            int s0 = base >> 16, a = r0;
            for (int o = 0; o < c[h]; o += width, ++s0) {
                rt.seg_e[s0] = static_cast<int16_t>(x);
                rt.seg_r[s0] = static_cast<int16_t>(r0 + o);
                rt.seg_n[s0] = static_cast<int16_t>(min(width, c[h] - o));
            }
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const int n = rt.cnt[w * rt.Ep + x];
                rt.cnt[w * rt.Ep + x] = static_cast<int16_t>(a);
                a += n;
            }
        }
        base += v[h];
    }
    if (tid == static_cast<int>(blockDim.x) - 1) rt.shared[W] = base >> 16;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = warp * span + i * 32 + lane;
        if (i * 32 < span && r < R && e[i] >= 0) {
            const int o = mine[e[i]] + at[i];
            rt.order[o] = static_cast<int16_t>(r);
            rt.tok[o] = static_cast<int16_t>(r / p.k);
            rt.wt[o] = wt[i];
        }
    }
    rt.n_seg = rt.shared[W];
    rt.twice = rt.shared[W + 1];
    __syncthreads();
}

// One CTA of W = 4 warps (or 8): RW row groups x KW = W / RW splits of the inputs.  The
// RW warps of a split share its x rows and meet at a named barrier once a
// k-block; splits run on their own, each through its own ring, and the copies
// run ahead across the units of a CTA.
//   kW4Gemv    a unit is a tile of weight rows and up to x_rows <= 8 NT rows of x.
//   kW4GateUp  a unit is a tile (half gate, half up) and a segment: up to x_rows
//              rows of one expert.
//     Both: with as many units as CTAs that fit, or more, a CTA takes units in
//     turn and splits their inputs over its warps; with fewer, a cluster of CTAs
//     takes one unit and splits its inputs over all their warps.
//   kW4Down    a cluster takes a tile of the output and splits the list of
//              (segment, k-block) over its warps; a warp adds what it has for a
//              segment, times the gate weight, to its own fp32 rows by token, and
//              the sum over splits and CTAs is the layer's output.
//   kW4GateUpAlone, kW4DownAlone
//              a warp takes a unit (a tile and a segment) by itself, with nothing to
//              sum and nobody to meet; down then writes a routed row's share in fp32
//              for w4_combine_kernel.  For calls with units enough (w4_launch_gate_up and
//              w4_launch_down say which).
//
// What bounds it.  An item -- 64 weight rows x 128 inputs, 4.2 KB -- is about 600
// instructions of a warp (352 unpack it, 32 are products, the rest copy, scale and
// address), and a scheduler's share of the measured copy rate brings it in 730 cycles.  The
// products are mma.sync, whose operands are registers: a tcgen05 product takes the
// weights from shared memory or TMEM, where their four bytes for every byte read would
// have to be written first, and its rate is not needed for 8 or 16 columns.  Memory and
// instructions being about even (issue slots busy 55 %, HBM 4.5 TB/s in a long gate/up
// product), what remains is launch, latency, and an uneven number of items an SM.  T = 4,
// Mixtral-shaped: 116 us, 63 % of the copy rate; T = 32, fine-grained: 72 us, 57 %;
// M = 1, 4096 x 14336: 10.7 us, 42 %, of which 3.4 are spent before and after the items.
// Not kept, since they gained nothing: deeper rings, several row tiles interleaved, sums
// pushed to one CTA of a cluster.
template <int MODE, int NT, int G, int W>
struct W4Shape {
    static constexpr int RW = NT;                             // row groups
    static constexpr int KW = W / RW;                         // splits of the inputs
    static constexpr int kTile = RW * kW4Rows;                // weight rows of a CTA
    static constexpr int kOut = MODE == kW4GateUp || MODE == kW4GateUpAlone ? kTile / 2 : kTile;
    static constexpr int kWarpBytes = kW4Rows * 64 + (kW4Blk / G) * 128;
    static_assert(RW == 1 || (RW == 2 && KW == 2), "two named barriers");
    static __host__ __device__ int stage_bytes(int x_rows) { return RW * kWarpBytes + x_rows * 256; }
    static __host__ __device__ int ring_bytes(int x_rows) { return KW * kW4Stages * stage_bytes(x_rows); }
};

// Three CTAs an SM: 168 registers a thread and twelve warps.  With 128 and sixteen, or
// no limit: T = 32, 64 experts of 7168 x 2048 288 us, 296, 293; T = 32, Mixtral-shaped
// 206, 223, 218; M = 16, 28672 x 8192 37.1, 39.4, 36.9; M = 1, 4096 x 14336 10.7, 10.7, 11.2.
template <int MODE, int NT, int G, int W>
__global__ void __launch_bounds__(W * 32, W == kW4Warps ? 3 : 1) w4_kernel(const W4Args p) {
    using S = W4Shape<MODE, NT, G, W>;
    constexpr bool kDown = MODE == kW4Down;
    constexpr bool kGateUp = MODE == kW4GateUp || MODE == kW4GateUpAlone;
    constexpr bool kAlone = w4_is_alone(MODE);
    constexpr bool kAfter = MODE == kW4Down || MODE == kW4DownAlone;  // reads h
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rw = warp % S::RW, kw = warp / S::RW;
    const int csize = static_cast<int>(cluster_size()), crank = static_cast<int>(cluster_rank());
    const int split = kAlone ? 0 : crank * S::KW + kw, splits = kAlone ? 1 : csize * S::KW;
    const int KB = (p.K + kW4Blk - 1) / kW4Blk;
    const int tiles = (p.N + S::kOut - 1) / S::kOut;
    // The down kernel is scheduled while the gate/up kernel of its call drains.  Routing
    // and the first weights come in meanwhile, under a flag that gate/up releases when it
    // has waited for everything before it: who acquires it may read all of that.  Only h
    // is not there yet, and waited for below.  A CTA that finds no flag waits for gate/up
    // itself.  Waiting for gate/up first took T = 1, fine-grained, from 14.7 to 15.4 us,
    // T = 8 from 40.0 to 43.3; reading without the flag, which no rule of the memory model
    // covers, 14.3 and 40.0.
    if (!kAfter) grid_wait();
    if (kGateUp && blockIdx.x == 0 && threadIdx.x == 0)
        asm volatile("st.release.gpu.global.s32 [%0], 1;" ::"l"(&p.hdr->w4_ready) : "memory");
    if (!kGateUp || blockIdx.x > 0 || threadIdx.x == 0) grid_release();  // after the flag
    int seen = 0;
    if (kAfter) {
        if (threadIdx.x == 0) {
            int ready;
            asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(ready) : "l"(&p.hdr->w4_ready) : "memory");
            if (!ready) grid_wait();
        }
        __syncthreads();
        if (threadIdx.x == 0) seen = atomicAdd(&p.hdr->w4_seen, 1);
    }
    // The last CTA to look takes the flag back for the next call.
    auto wait_h = [&]() {
        grid_wait();
        if (threadIdx.x == 0 && seen == static_cast<int>(gridDim.x) - 1) p.hdr->w4_ready = p.hdr->w4_seen = 0;
    };
    bool ok;
    const int T = row_count(p.d_T, p.T_host, p.T_max, p.hdr, &ok);
    if (!ok) {  // the same for every CTA of the cluster
        if (kAfter) wait_h();
        return;
    }

    // shared memory: [rings][fp32 sums: a tile a warp][routing]
    const int sbytes = S::stage_bytes(p.x_rows);
    uint8_t* ring = smem + kw * kW4Stages * sbytes;
    float* sums = reinterpret_cast<float*>(smem + S::ring_bytes(p.x_rows));
    W4Routing rt;
    if (MODE != kW4Gemv) {
        rt.template place<W>(reinterpret_cast<uint8_t*>(sums + (kAlone ? 0 : W * p.sum_rows * kW4Pad)), p.T_max * p.k, p.E);
        build_routing<W>(p, rt, T, p.x_rows);
    }

    // The units of this CTA (or cluster), and the items -- k-blocks -- of one unit
    // that are this split's.  Down: one unit, whose items are (segment, k-block).
    const int passes = MODE == kW4Gemv ? (T + p.x_rows - 1) / p.x_rows : 1;
    const int n_units = kDown ? tiles : tiles * (MODE == kW4Gemv ? passes : rt.n_seg);
    const int u0 = kAlone ? blockIdx.x * W + warp : blockIdx.x / csize, ustep = kAlone ? gridDim.x * W : gridDim.x / csize;
    const int items = kDown ? rt.n_seg * KB : KB;
    const int i0 = static_cast<int>(static_cast<unsigned>(items) * split / splits);
    const int i1 = static_cast<int>(static_cast<unsigned>(items) * (split + 1) / splits);
    if (kDown) {
        for (int i = threadIdx.x; i < W * T * kW4Pad; i += blockDim.x) sums[i] = 0.0f;
        __syncthreads();
    }
    auto tile_of = [&](int u) { return kDown ? u : MODE == kW4Gemv ? u / passes : u % tiles; };
    auto part_of = [&](int u) { return kDown ? 0 : MODE == kW4Gemv ? u % passes : u / tiles; };  // segment or pass
    auto rows_of = [&](int part) {
        return MODE == kW4Gemv ? min(p.x_rows, T - part * p.x_rows) : static_cast<int>(rt.seg_n[part]);
    };

    // A stage of the ring: [RW warps: 64 rows of 64 bytes of weights, 128 / group rows
    // of 64 scales][x rows of 256 bytes].
    auto stage_at = [&](int slot) {
        uint8_t* b = ring + slot * sbytes;
        return W4Stage{b + rw * S::kWarpBytes, b + rw * S::kWarpBytes + kW4Rows * 64, b + S::RW * S::kWarpBytes};
    };
    // Where the copies are: the next item, its ring slot, and what this lane copies --
    // of the weights the row lane / 4 of each 8, piece lane % 4 of its 64 bytes; of
    // the scales 8 rows of one group; of x the rows lane / 16 + 2 rw of each 2 RW,
    // piece lane % 16.  A warp's rows are [nw, nw + 64) of one matrix, or 32 + 32 of two.
    constexpr int kRowsW = kGateUp ? kW4Rows / 2 : kW4Rows;
    constexpr int kXMost = NT * 8 / (2 * S::RW);  // x rows of a lane
    const size_t ld8 = static_cast<size_t>(p.K) * 4;  // bytes of 8 rows
    const int wr = lane >> 2, wc = lane & 3, sg = lane >> 3, sc = lane & 7, xc = lane & 15;
    const int sn8 = kGateUp ? (sc & 3) * 8 : sc * 8;
    const uint32_t ring_u = smem_addr(ring);
    const uint32_t w_to = ring_u + rw * S::kWarpBytes + wr * 64 + (swz_w<G>(wc, wr) << 4);  // row + 8: the same swizzle
    const uint32_t s_to = ring_u + rw * S::kWarpBytes + kW4Rows * 64 + sg * 128 + (sc << 4);
    const uint32_t x_to = ring_u + S::RW * S::kWarpBytes;
    int pu = i0 < i1 ? u0 : n_units, pi = i0, kb = 0, left = 0, nc_p = 0;
    uint32_t slot_off = 0;
    const uint32_t ring_len = kW4Stages * sbytes;
    const uint8_t *qa, *qb;
    const bf16 *sp, *xp[kXMost];
    auto seek = [&]() {  // to item pi of unit pu
        const int part = kDown ? pi / KB : part_of(pu);
        kb = kDown ? pi - part * KB : pi;
        nc_p = rows_of(part);
        const int e = MODE == kW4Gemv ? 0 : rt.seg_e[part];
        const int nw = tile_of(pu) * S::kOut + rw * kRowsW;
        left = p.N - nw;  // rows there are: a multiple of 8
        const size_t at = ((static_cast<size_t>(e) * p.N + nw + wr) * p.K >> 1) + kb * 64 + wc * 16;
        qa = p.q0 + at;
        if (kGateUp) qb = p.q1 + at;
        const bf16* s = (kGateUp && sc >= 4) ? p.s1 : p.s0;
        sp = s + (static_cast<size_t>(e) * (p.K / G) + kb * (kW4Blk / G) + sg) * p.N + nw + sn8;
#pragma unroll
        for (int i = 0; i < kXMost; ++i) {
            const int r = (lane >> 4) + 2 * rw + i * 2 * S::RW;
            int row = 0;
            if (r < nc_p)
                row = MODE == kW4Gemv ? part * p.x_rows + r : kAfter ? rt.order[rt.seg_r[part] + r] : rt.tok[rt.seg_r[part] + r];
            xp[i] = p.x + static_cast<size_t>(row) * p.K + kb * kW4Blk + xc * 8;
        }
    };
    if (pu < n_units) seek();
    // Post the copies of the next item and move on.  Pieces outside the matrices are
    // filled with zeros.
    auto post_w = [&]() {
        const uint32_t dst = w_to + slot_off;
        const int left_k = p.K - kb * kW4Blk;
        if (left_k >= kW4Blk && left >= kRowsW) {
            const uint8_t* q = qa;
#pragma unroll
            for (int g = 0; g < 8; ++g, q += ld8) {
                if (kGateUp && g == 4) q = qb;
                cp_async16(dst + g * 512, q);
            }
            if (sg < kW4Blk / G) cp_async16(s_to + slot_off, sp);
        } else {
            const bool kin = wc * 32 < left_k;
#pragma unroll
            for (int g = 0; g < 8; ++g) {
                const int g8 = kGateUp ? g & 3 : g;
                const bool in = kin && g8 * 8 < left;
                cp_async16(dst + g * 512, in ? (kGateUp && g >= 4 ? qb : qa) + g8 * ld8 : p.q0, in);
            }
            if (sg < kW4Blk / G) {
                const bool in = sg * G < left_k && sn8 < left;
                cp_async16(s_to + slot_off, in ? sp : p.s0, in);
            }
        }
    };
    auto post_x = [&]() {  // shared out among the split's warps
        const bool kin = kb * kW4Blk + xc * 8 < p.K;
#pragma unroll
        for (int i = 0; i < kXMost; ++i) {
            const int r = (lane >> 4) + 2 * rw + i * 2 * S::RW;
            if (r < nc_p) cp_async16(x_to + slot_off + r * 256 + (swz_x<G>(xc, r) << 4), kin ? xp[i] : p.x, kin);
        }
    };
    auto post = [&](bool first) {
        if (pu < n_units) post_w();
        if (kAfter && first) wait_h();  // in every CTA: who waits for this kernel counts on it
        if (pu < n_units) {
            post_x();
            slot_off = slot_off + sbytes == ring_len ? 0 : slot_off + sbytes;
            if (++pi == i1) {
                pi = i0;
                pu = kDown ? n_units : pu + ustep;
                if (pu < n_units) seek();
            } else if (kDown && kb + 1 == KB) {
                seek();
            } else {
                ++kb;
                qa += 64;
                if (kGateUp) qb += 64;
                sp += static_cast<size_t>(kW4Blk / G) * p.N;
#pragma unroll
                for (int i = 0; i < kXMost; ++i) xp[i] += kW4Blk;
            }
        }
        cp_async_commit();
    };
    auto meet = [&]() {
        if (S::RW == 1) __syncwarp();
        else if (kw == 0) asm volatile("bar.sync 1, 64;" ::: "memory");
        else asm volatile("bar.sync 2, 64;" ::: "memory");
    };
    post(true);

    int cslot = 0;
    for (int u = u0; u < n_units; u += ustep) {
        float acc[4][NT][4];
        auto clear = [&]() {
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.0f;
        };
        clear();
        int cpart = kDown && i0 < i1 ? i0 / KB : part_of(u), ckb = i0 - cpart * KB;  // ckb: down only
        int nc = kDown ? (i0 < i1 ? rows_of(cpart) : 0) : rows_of(cpart);
        for (int i = i0; i < i1; ++i) {
            cp_async_wait<0>();  // the item's: the next one's are posted below
            meet();
            post(false);
            compute_stage<NT, G>(stage_at(cslot), nc, p.magic, acc);
            cslot = cslot + 1 == kW4Stages ? 0 : cslot + 1;
            if (kDown && (i + 1 == i1 || ++ckb == KB)) {
                // the segment's rows by token.  If a token holds two rows of one
                // expert, the quarter-warps (two rows each) take turns.
                float* mine = sums + static_cast<size_t>(warp) * T * kW4Pad;
                const int r = lane >> 2, t = lane & 3;
                const bool turns = rt.twice != 0;
                for (int q = 0; q < (turns ? 4 : 1); ++q) {
                    if (!turns || t == q) {
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int col = j * 8 + 2 * t + h;
                                if (col < nc) {
                                    const int o = rt.seg_r[cpart] + col;
                                    const float wt = rt.wt[o];
                                    float* dst = mine + rt.tok[o] * kW4Pad + r;
#pragma unroll
                                    for (int m = 0; m < 4; ++m) {
                                        dst[m * 16] += wt * acc[m][j][h];
                                        dst[m * 16 + 8] += wt * acc[m][j][2 + h];
                                    }
                                }
                            }
                    }
                    __syncwarp();
                }
                clear();
                ckb = 0;
                ++cpart;
                if (i + 1 < i1) nc = rows_of(cpart);
            }
        }

        if (kAlone) {
            const int r = lane >> 2, t = lane & 3, n0 = tile_of(u) * S::kOut + r;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int col = 2 * t + h;
                if (col < nc) {
                    const int o = rt.seg_r[cpart] + col;
                    const size_t row = static_cast<size_t>(rt.order[o]) * p.N;
                    const float wt = kGateUp ? 0.0f : rt.wt[o];
#pragma unroll
                    for (int m = 0; m < (kGateUp ? 2 : 4); ++m)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const int n = n0 + m * 16 + q * 8;
                            const float v = acc[m][0][2 * q + h];
                            if (n >= p.N) continue;
                            if (kGateUp) p.out[row + n] = __float2bfloat16_rn(v / (1.0f + expf(-v)) * acc[(m + 2) & 3][0][2 * q + h]);
                            else p.y[row + n] = wt * v;
                        }
                }
            }
            continue;
        }

        // sums over the splits, in order: a warp's tile is [nc][64], the first RW
        // tiles make the CTA's
        if (kDown) {
            nc = T;
        } else {
            const int r = lane >> 2, t = lane & 3;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int col = j * 8 + 2 * t + h;
                    if (col < nc) {
                        float* dst = sums + (warp * nc + col) * kW4Pad + r;
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            dst[m * 16] = acc[m][j][h];
                            dst[m * 16 + 8] = acc[m][j][2 + h];
                        }
                    }
                }
        }
        __syncthreads();
        if (csize > 1) {
            if (S::KW > 1) {
                for (int o = threadIdx.x; o < S::RW * nc * kW4Rows; o += blockDim.x) {
                    const int at = (o >> 6) * kW4Pad + (o & 63);
                    float v = sums[at];
#pragma unroll
                    for (int w = 1; w < S::KW; ++w) v += sums[w * S::RW * nc * kW4Pad + at];
                    sums[at] = v;
                }
            }
            cluster_sync();
        }
        // then over the cluster's CTAs, in order; each CTA stores its share
        const uint32_t sums_u = smem_addr(sums);
        const int n0 = tile_of(u) * S::kOut;
        for (int o = crank * blockDim.x + threadIdx.x; o < nc * S::kOut; o += csize * blockDim.x) {
            const int col = o / S::kOut, row = o % S::kOut;
            const int n = n0 + row;
            auto total = [&](int g, int rr) {  // row rr of row group g's tile
                const int at = (g * nc + col) * kW4Pad + rr;
                float v = 0.0f;
                if (csize == 1) {
#pragma unroll
                    for (int w = 0; w < S::KW; ++w) v += sums[w * S::RW * nc * kW4Pad + at];
                } else {
                    for (int c = 0; c < csize; ++c) v += ld_cluster_f32(sums_u + at * 4, c);
                }
                return v;
            };
            if (n < p.N) {
                if (MODE == kW4GateUp) {
                    const float g = total(row >> 5, row & 31), up = total(row >> 5, (row & 31) + 32);
                    const float h = g / (1.0f + expf(-g)) * up;
                    p.out[static_cast<size_t>(rt.order[rt.seg_r[cpart] + col]) * p.N + n] = __float2bfloat16_rn(h);
                } else {
                    const int m = MODE == kW4Gemv ? cpart * p.x_rows + col : col;
                    p.out[static_cast<size_t>(m) * p.N + n] = __float2bfloat16_rn(total(row >> 6, row & 63));
                }
            }
        }
        // no CTA may leave, or overwrite its sums, while another reads them
        if (csize > 1) cluster_sync();
        else __syncthreads();
    }
}

struct W4CombineArgs {
    const float* y;  // [T k, N]
    const int32_t* idx;
    bf16* out;
    const int32_t* d_T;
    int T_host, T_max, N, E, k;
    EtHeader* hdr;
};

// out[t] = the sum of a token's rows, in order: four columns a thread.  All launch and
// latency (T = 32, H = 2048, 8 rows each, 2.1 MB: 6.8 us by itself with cold caches).
__global__ void __launch_bounds__(256) w4_combine_kernel(const W4CombineArgs p) {
    grid_begin();
    bool ok;
    const int T = row_count(p.d_T, p.T_host, p.T_max, p.hdr, &ok);
    const int t = blockIdx.y, n = (blockIdx.x * 256 + threadIdx.x) * 4;
    if (!ok || t >= T || n >= p.N) return;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int j = 0; j < p.k; ++j) {
        const int r = t * p.k + j, e = p.idx[r];
        if (e < 0 || e >= p.E) continue;
        const float4 v = __ldcg(reinterpret_cast<const float4*>(p.y + static_cast<size_t>(r) * p.N + n));
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    *reinterpret_cast<uint2*>(p.out + static_cast<size_t>(t) * p.N + n) = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
}

// ---------------------------------------------------------------- conversion

constexpr int kConvRows = 8;       // rows of a CTA, one a warp: N is a multiple of 8, so they share an expert
constexpr int kConvK = 4096;       // most inputs of a row a CTA takes

struct W4ConvArgs {
    const bf16* w;
    const uint8_t* q;
    const bf16* s;
    bf16* w_out;
    uint8_t* q_out;
    bf16* s_out;
    int N, K, chunk;  // chunk: inputs a CTA takes, a multiple of 256 (or all of K)
};

// Eight inputs a lane and step (16 bytes), four steps in flight; the lanes of a
// group (4, 8 or 16) share its largest magnitude by shuffles.  The scales of the
// CTA's eight rows are collected in shared memory and stored 16 bytes a group.
//
// q = round-half-even(w / s) without a division: y = w * (1 / s), with a
// reciprocal good to 2^-22, is within 2^-19 of w / s (|y| < 7.1).  w and s have 8 significant bits, so w / s
// is either exactly half-way between two integers or at least 2^-10 away from
// that; rounding y to a multiple of 2^-13 first brings the half-way cases back
// and moves no other across.  Scales below 2^-126 (whose reciprocal overflows)
// are divided by.
//
// Bound by HBM: 470 M weights, 1.19 GB, in 178 us, 98 % of the measured copy rate.
template <int G>
__global__ void __launch_bounds__(kConvRows * 32) w4_quantize_kernel(const W4ConvArgs p) {
    __shared__ __align__(16) __nv_bfloat16 sc[kConvK / G][kConvRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_begin();
    const size_t row0 = static_cast<size_t>(blockIdx.x) * kConvRows, row = row0 + warp;
    const int k0 = blockIdx.y * p.chunk, kn = min(p.chunk, p.K - k0);
    constexpr int lanes = G / 8;
    const uint4* src = reinterpret_cast<const uint4*>(p.w + row * p.K + k0);
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.q_out + (row * p.K + k0) / 2);
    const int vecs = kn / 8;
    for (int base = 0; base < vecs; base += 128) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = base + i * 32 + lane;
            v[i] = at < vecs ? __ldcs(src + at) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = base + i * 32 + lane;
            const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            // largest magnitude; NaN wins over infinity, infinity over every number
            __nv_bfloat162 m2 = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&u[0]));
#pragma unroll
            for (int j = 1; j < 4; ++j)
                m2 = __hmax2_nan(m2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&u[j])));
#pragma unroll
            for (int off = 1; off < lanes; off <<= 1) {
                const uint32_t o = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<const uint32_t*>(&m2), off);
                m2 = __hmax2_nan(m2, *reinterpret_cast<const __nv_bfloat162*>(&o));
            }
            const float top = __bfloat162float(__hmax_nan(__low2bfloat16(m2), __high2bfloat16(m2)));
            const bool finite = top < __uint_as_float(0x7f800000u);
            // bf16(top / 7): top has 8 bits, so top / 7 is a bf16 value or at least 2^-12
            // of itself away from the middle between two; top * (1 / 7) rounds alike
            const __nv_bfloat16 sb = __float2bfloat16_rn(finite ? top * (1.0f / 7.0f) : __uint_as_float(0x7fc00000u));
            const float s = __bfloat162float(sb);
            uint32_t out = 0x88888888u;  // zeros, where the scale is zero or not a number
            if (s >= 1.17549435e-38f) {
                float inv;
                asm("rcp.approx.f32 %0, %1;" : "=f"(inv) : "f"(s));
                // t = 1536 + w / s in steps of 2^-13; adding 1.5 * 2^23 + 8 - 1536 leaves
                // round-half-even(w / s) + 8 in the sum's low bits, which are added up
                // at their places with the (known) high bits taken off at the end
                out = 0u - 0x4b400000u * 0x11111111u;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float f = (j & 1) ? bf_hi(u[j >> 1]) : bf_lo(u[j >> 1]);
                    const float t = __fmaf_rn(f, inv, 1536.0f);
                    out += __float_as_uint(__fadd_rn(t, 12582920.0f - 1536.0f)) << (4 * j);
                }
            } else if (s > 0.0f) {
                out = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float f = (j & 1) ? bf_hi(u[j >> 1]) : bf_lo(u[j >> 1]);
                    const float r = fminf(fmaxf(rintf(f / s), -8.0f), 7.0f);
                    out |= static_cast<uint32_t>(static_cast<int>(r) + 8) << (4 * j);
                }
            }
            if (at < vecs) {
                dst[at] = out;
                if ((at & (lanes - 1)) == 0) sc[at / lanes][warp] = sb;
            }
        }
    }
    __syncthreads();
    const size_t e = row0 / p.N;
    const int n0 = static_cast<int>(row0 - e * p.N), groups = p.K / G, g0 = k0 / G;
    for (int g = threadIdx.x; g < kn / G; g += blockDim.x)
        *reinterpret_cast<uint4*>(p.s_out + (e * groups + g0 + g) * p.N + n0) = *reinterpret_cast<const uint4*>(&sc[g][0]);
}

// The same split.  128 + q by or-ing the nibble into bf16, minus 136, times the
// scale: the first two are exact, the product is rounded once.  470 M weights in
// 172 us, the measured copy rate.
template <int G>
__global__ void __launch_bounds__(kConvRows * 32) w4_dequantize_kernel(const W4ConvArgs p) {
    __shared__ __align__(16) __nv_bfloat16 sc[kConvK / G][kConvRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_begin();
    const size_t row0 = static_cast<size_t>(blockIdx.x) * kConvRows, row = row0 + warp;
    const int k0 = blockIdx.y * p.chunk, kn = min(p.chunk, p.K - k0);
    constexpr int lanes = G / 8;
    const size_t e = row0 / p.N;
    const int n0 = static_cast<int>(row0 - e * p.N), groups = p.K / G, g0 = k0 / G;
    for (int g = threadIdx.x; g < kn / G; g += blockDim.x)
        *reinterpret_cast<uint4*>(&sc[g][0]) = *reinterpret_cast<const uint4*>(p.s + (e * groups + g0 + g) * p.N + n0);
    __syncthreads();
    const uint32_t* src = reinterpret_cast<const uint32_t*>(p.q + (row * p.K + k0) / 2);
    uint4* dst = reinterpret_cast<uint4*>(p.w_out + row * p.K + k0);
    const int vecs = kn / 8;
    const __nv_bfloat162 off = __floats2bfloat162_rn(136.0f, 136.0f);
    for (int base = 0; base < vecs; base += 256) {
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int at = base + i * 32 + lane;
            v[i] = at < vecs ? __ldcs(src + at) : 0u;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int at = base + i * 32 + lane;
            if (at < vecs) {
                const __nv_bfloat162 s = __bfloat162bfloat162(sc[at / lanes][warp]);
                uint32_t o[4];  // inputs (0,4) (1,5) (2,6) (3,7)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t b = ((v[i] >> (4 * j)) & 0x000f000fu) | 0x43004300u;
                    const __nv_bfloat162 d = __hmul2(__hsub2(*reinterpret_cast<const __nv_bfloat162*>(&b), off), s);
                    o[j] = *reinterpret_cast<const uint32_t*>(&d);
                }
                __stcs(dst + at, make_uint4(__byte_perm(o[0], o[1], 0x5410), __byte_perm(o[2], o[3], 0x5410),
                                            __byte_perm(o[0], o[1], 0x7632), __byte_perm(o[2], o[3], 0x7632)));
            }
        }
    }
}

// ---------------------------------------------------------------- launches

bool w4_shape_ok(int N, int K, int group, std::string* why) {
    if (group != 32 && group != 64 && group != 128) { *why = "group must be 32, 64 or 128"; return false; }
    if (K < group || K % group || K > (1 << 20)) { *why = "inputs must be a positive multiple of group (<= 2^20)"; return false; }
    if (N < 8 || N % 8 || N > (1 << 20)) { *why = "outputs must be a positive multiple of 8 (<= 2^20)"; return false; }
    return true;
}

// How many clusters of c CTAs of a kernel fit the GPU at once when n of its CTAs
// fit an SM (a cluster lies within one of the GPU's processor clusters, so some
// places stay empty).
constexpr int kW4FitMax = 32;  // most CTAs an SM
template <class K>
cudaError_t w4_query_clusters(K kernel, int threads, int c, int n, int* clusters) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(c * 1024);
    cfg.blockDim = dim3(threads);
    const int smem = kSmemSm / n / 128 * 128 - 1024;
    cfg.dynamicSmemBytes = smem < kSmemLimit ? smem : kSmemLimit;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = c;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(clusters, kernel, &cfg);
}

// Most segments of R routed rows: each has a row, an expert has one and one more for
// each full pass.
int w4_segments(int R, int E, int width) {
    const int experts = R < E ? R : E;
    return experts + R / width < R ? experts + R / width : R;
}

// How a call is spread over the GPU.
struct W4Plan {
    long long units;
    int c, per_sm, smem;  // CTAs that share a unit, CTAs an SM, dynamic shared memory of one
    long long cost;       // estimated ns (kW4Gemv)
};

// The clusters that fit device `dev`; 0 and an error in *err if the query failed.
template <int MODE, int NT, int G, int W>
int w4_fit(int dev, int c, int n, cudaError_t* err) {
    static DeviceNumbers<4 * kW4FitMax> fits;
    n = n < 1 ? 1 : n > kW4FitMax ? kW4FitMax : n;
    const int lc = c == 8 ? 3 : c == 4 ? 2 : c == 2 ? 1 : 0;
    int v = 0;
    const cudaError_t e = fits.get(dev, lc * kW4FitMax + n - 1, &v, [&](int* out) {
        return w4_query_clusters(w4_kernel<MODE, NT, G, W>, W * 32, c, n, out);
    });
    if (e != cudaSuccess) *err = e;
    return e == cudaSuccess ? v : 0;
}

// `rows` tokens at most; x_rows <= 8 NT of them (or of an expert's rows) a pass.
template <int MODE, int NT, int G, int W>
int w4_plan(const W4Args& a, int rows, int x_rows, int dev, int sms, W4Plan* pl) {
    using S = W4Shape<MODE, NT, G, W>;
    const int segs = w4_segments(rows * a.k, a.E, x_rows);
    const long long tiles = (a.N + S::kOut - 1) / S::kOut;
    constexpr bool alone = w4_is_alone(MODE);
    const long long units = tiles * (MODE == kW4Down ? 1 : MODE == kW4Gemv ? (rows + x_rows - 1) / x_rows : segs);
    const int KB = (a.K + kW4Blk - 1) / kW4Blk;
    const long long blocks = static_cast<long long>(KB) * (MODE == kW4Down ? segs : 1);
    const int routing = MODE == kW4Gemv ? 0 : W4Routing::bytes(a.T_max * a.k, a.E, W);
    const int sum_rows = MODE == kW4Down ? rows : x_rows;
    const int smem = S::ring_bytes(x_rows) + (alone ? 0 : W * sum_rows * kW4Pad * 4) + routing;
    *pl = {};
    if (smem > kSmemLimit) return ET_OK;  // no place for it
    static SmemOptIn opt;
    const cudaError_t e = api_smem_opt_in(opt, dev, w4_kernel<MODE, NT, G, W>, kSmemLimit);
    if (e != cudaSuccess) return api_fail_cuda(e, "cudaFuncSetAttribute(4-bit products)");
    static DeviceNumbers<1> kept_regs;
    int regs = 0;
    cudaError_t err = kept_regs.get(dev, 0, &regs, [](int* out) {
        cudaFuncAttributes at{};
        const cudaError_t q = cudaFuncGetAttributes(&at, w4_kernel<MODE, NT, G, W>);
        *out = at.numRegs;
        return q;
    });
    if (err != cudaSuccess) return api_fail_cuda(err, "cudaFuncGetAttributes(4-bit products)");
    const int by_smem = kSmemSm / (smem + 1024), by_regs = 65536 / (W * 32 * ((regs + 7) / 8 * 8));
    const int per_sm = W > kW4Warps ? 1 : by_smem < by_regs ? by_smem : by_regs;
    // 8, 4 or 2 CTAs share a unit's inputs if all of them fit at once and every split
    // keeps two k-blocks
    int c = alone ? 1 : kW4ClusterMax;
    while (c > 1 && (blocks < 2ll * S::KW * c || units > w4_fit<MODE, NT, G, W>(dev, c, per_sm, &err))) c /= 2;
    if (err != cudaSuccess) return api_fail_cuda(err, "cudaOccupancyMaxActiveClusters(4-bit products)");
    // The k-blocks of a warp of the busiest SM, its CTAs taken one after the other, and
    // from them the time (W4Plan::cost), which decides between 8 and 16 rows a pass.  On 120
    // calls (9 to 64 rows, 768 x 768 to 28672 x 16384) the faster side was taken in 112;
    // the others lost 9 % on average, 23 % at most (M = 9, 2032 x 14976).
    const auto items = [&](int n) { return (units * n + sms - 1) / sms * ((KB + n * S::KW - 1) / (n * S::KW)); };
    // One CTA a unit in place of two where one apiece finds an SM to itself and its warps
    // have few k-blocks: M = 25, 2368 x 2432 (148 units) 5.0 us in place of 5.7, M = 3, 7576 x
    // 2560 5.0 and 5.4.  With many, or larger clusters, the CTAs that an SM lacks cost more
    // than an even share gains: M = 3, 8424 x 15872 24.3 us with one, 19.4 with two; M = 1,
    // 2432 x 14336 10.1 with four, 9.1 with eight.
    if (MODE == kW4Gemv && c == 2 && units <= sms && KB <= 8 * S::KW && items(1) < items(2)) c = 1;
    *pl = {units, c, per_sm, smem, NT == 1 ? 3400 + 450 * items(c) : 4800 + 640 * items(c)};
    return ET_OK;
}

template <int MODE, int NT, int G, int W>
int w4_launch(W4Args a, int rows, int x_rows, const W4Plan& pl, int dev, int sms, void* stream) {
    if (!pl.per_sm) return api_fail(ET_ERR_UNSUPPORTED, "rows do not fit in shared memory");
    a.x_rows = x_rows;
    a.sum_rows = MODE == kW4Down ? rows : x_rows;
    a.magic = 0x43004300u;
    const long long fit = static_cast<long long>(sms) * pl.per_sm;
    const long long units = w4_is_alone(MODE) ? (pl.units + W - 1) / W : pl.units;  // of a CTA's size
    const bool in_turn = MODE != kW4Down && pl.c == 1 && units > fit;                // CTAs take several
    const long long grid = in_turn ? fit : units * pl.c;
    // Scheduled while the kernel before drains, which hides the launch (M = 1, 4096 x 14336
    // 11.0 -> 10.8 us in a graph).  Its CTAs then fill the places the other kernel leaves, so
    // no more of them may fit an SM than an even spread needs: without that limit M = 1
    // took 13.7 us.  CTAs that take units in turn are launched after the other: they fill
    // the GPU, and started early they lost up to 12 % (T = 16, 16 experts of 4096 x 2048,
    // k = 4, 55.1 us and 61.8; T = 64, fine-grained, 83.7 and 87.9; T = 4, Mixtral-shaped, the
    // same) and gained 5 at most (T = 32, 256 experts of 1024 x 512, 46.6 and 44.3) -- except
    // after the gate/up kernel where they are short, up to 64 items a scheduler: 32 experts
    // of 2048 x 768, k = 4, T = 64 37.7 us and 34.8; fine-grained, T = 64 88.3 and 83.7; longer
    // ones, 64 of 7168 x 2048, T = 16 255.6 and 262.5, T = 32 288.3 and 285.6.
    const long long per_scheduler = pl.units * ((a.K + kW4Blk - 1) / kW4Blk) / (4 * sms);
    const bool early = !in_turn || (MODE == kW4DownAlone && per_scheduler <= 64);
    int smem = pl.smem;
    if (early) {
        int n = static_cast<int>((grid + sms - 1) / sms);
        cudaError_t err = cudaSuccess;
        while (n < pl.per_sm && w4_fit<MODE, NT, G, W>(dev, pl.c, n, &err) * static_cast<long long>(pl.c) < grid) ++n;
        if (err != cudaSuccess) return api_fail_cuda(err, "cudaOccupancyMaxActiveClusters(4-bit products)");
        const int more = kSmemSm / (n + 1) / 128 * 128 - 1024 + 128;  // n + 1 do not fit
        smem = smem > more ? smem : more < kSmemLimit ? more : kSmemLimit;
    }
    const cudaError_t e = api_launch_cluster(w4_kernel<MODE, NT, G, W>, dim3(static_cast<unsigned>(grid)), W * 32,
                                             pl.c, early, smem, stream, a);
    if (e != cudaSuccess) return api_fail_cuda(e, "launch of the 4-bit product kernel");
    return ET_OK;
}

template <int MODE, int NT, int G>
int w4_plan_launch(const W4Args& a, int rows, int x_rows, int dev, int sms, void* stream) {
    W4Plan pl{};
    const int rc = w4_plan<MODE, NT, G, kW4Warps>(a, rows, x_rows, dev, sms, &pl);
    return rc ? rc : w4_launch<MODE, NT, G, kW4Warps>(a, rows, x_rows, pl, dev, sms, stream);
}

// With 9 rows or more: 8 a pass (one tile of columns in every product) or 16 (two),
// whichever is estimated to end first (w4_plan).  Half the passes over the weights mean
// half the unpacking, and win where there is much to do: 28672 x 8192, M = 16 37.2 us
// against 49.6; twice the CTAs win where an SM would stay empty: 14336 x 4096, M = 16
// 15.2 us against 17.1, 2048 x 2048 4.2 against 5.6.  (32 a pass, a fourth of the splits,
// lost nearly everywhere.)
template <int G>
int w4_launch_gemv(const W4Args& a, int rows, int dev, int sms, void* stream) {
    W4Plan one{}, two{};
    const int one_rows = rows < 8 ? rows : 8, two_rows = rows < 16 ? rows : 16;
    int rc = w4_plan<kW4Gemv, 1, G, kW4Warps>(a, rows, one_rows, dev, sms, &one);
    if (!rc && rows > 8) rc = w4_plan<kW4Gemv, 2, G, kW4Warps>(a, rows, two_rows, dev, sms, &two);
    if (rc) return rc;
    if (rows <= 8 || one.cost <= two.cost) return w4_launch<kW4Gemv, 1, G, kW4Warps>(a, rows, one_rows, one, dev, sms, stream);
    return w4_launch<kW4Gemv, 2, G, kW4Warps>(a, rows, two_rows, two, dev, sms, stream);
}

// A warp takes a unit alone when each at work has two or three in turn: T = 16,
// Mixtral-shaped (5376 units), in clusters and alone, 165.9 us and 159.6, T = 32, 64 experts of
// 7168 x 2048 297 and 289, T = 64, 8 of 3200 x 6400 147 and 138; with fewer some wait long
// for the last: T = 8, 64 of 7168 x 2048 (4096) 191.6 and 198.2, T = 16, 16 of 4096 x 2048
// 55.1 and 70.5.  On 43 calls it took the faster or lost 6 % at most, but for two: T = 32,
// 256 of 1024 x 512 46.6 and 42.8, T = 64, 4 of 1024 x 4096 48.0 and 44.2.
template <int G>
int w4_launch_gate_up(const W4Args& a, int rows, int width, int dev, int sms, void* stream) {
    if (width > 8) return w4_plan_launch<kW4GateUp, 2, G>(a, rows, width, dev, sms, stream);
    constexpr int kOut = kW4Rows / 2;
    const long long units = static_cast<long long>((a.N + kOut - 1) / kOut) * w4_segments(rows * a.k, a.E, width);
    if (units >= 30ll * sms) return w4_plan_launch<kW4GateUpAlone, 1, G>(a, rows, width, dev, sms, stream);
    return w4_plan_launch<kW4GateUp, 1, G>(a, rows, width, dev, sms, stream);
}

// Estimated ns of an item of a warp when `warps` are at work.
long long w4_item_ns(long long warps, int sms) {
    const long long ns = 350 * warps / (4 * sms);
    return ns > 600 ? ns : 600;
}

// Up to 8 rows a pass, three forms.
//   Clusters of 8 with about two CTAs an SM become clusters of 4 with one of twice the
//   warps.  The places the gate/up kernel leaves come free one by one, its shared memory
//   in pieces, where 8 did not always find room: then 3 of 32 clusters ran after the
//   others (fine-grained, T = 5: 34.6 us, now 31.2; T = 8 42.7, now 40.5).  Clusters of 4
//   did, and two tiles of columns (NT) did.
//   A warp takes a unit alone, and a second kernel sums a token's rows, where that is
//   estimated to end first: clusters have 64 output columns each, and their fp32 rows of
//   T tokens leave room for one CTA an SM from T = 50 on.  Estimate: items of a warp,
//   0.1 us a token for the sums of a cluster, 2.5 us for the second kernel.  Call with
//   clusters and alone, us: T = 64, E 64, k 4, 1024 x 512 38 and 26; T = 16, E 64, k 8,
//   7168 x 2048 283 and 256; T = 8, fine-grained 40.5 and 41.6; T = 8, E 16, k 4, 4096 x 2048
//   51 and 57; T = 16, Mixtral-shaped 160 and 209.  On 43 calls it took the faster or lost
//   8 % at most (T = 20, fine-grained, 67.3 and 62.4).
template <int G>
int w4_launch_down(const W4Args& a, int rows, int width, int dev, int sms, void* stream) {
    if (width > 8) return w4_plan_launch<kW4Down, 2, G>(a, rows, width, dev, sms, stream);
    W4Plan four{}, eight{};
    int rc = w4_plan<kW4Down, 1, G, kW4Warps>(a, rows, width, dev, sms, &four);
    if (!rc && four.c == kW4ClusterMax && four.units * four.c * 4 >= 5ll * sms)
        rc = w4_plan<kW4Down, 1, G, kW4WarpsMax>(a, rows, width, dev, sms, &eight);
    if (rc) return rc;
    const bool wide = eight.per_sm && 2 * eight.c >= four.c;
    const W4Plan& pl = wide ? eight : four;
    const int KB = (a.K + kW4Blk - 1) / kW4Blk, segs = w4_segments(rows * a.k, a.E, width);
    const long long splits = pl.c * (wide ? kW4WarpsMax : kW4Warps), units = pl.units * segs;
    const long long shared_ns = (static_cast<long long>(segs) * KB + splits - 1) / splits * w4_item_ns(pl.units * splits, sms) + 100 * rows;
    // alone: units at work at once are rounded up to whole ones a scheduler, of three at most
    const long long each = (units + 4 * sms - 1) / (4 * sms);
    const long long alone_ns = KB * w4_item_ns(each <= 3 ? each * 4 * sms : units, sms) + 2500;
    if (pl.per_sm && shared_ns <= alone_ns)
        return wide ? w4_launch<kW4Down, 1, G, kW4WarpsMax>(a, rows, width, pl, dev, sms, stream)
                    : w4_launch<kW4Down, 1, G, kW4Warps>(a, rows, width, pl, dev, sms, stream);
    if ((rc = w4_plan_launch<kW4DownAlone, 1, G>(a, rows, width, dev, sms, stream))) return rc;
    const W4CombineArgs ca{a.y, a.idx, a.out, a.d_T, a.T_host, a.T_max, a.N, a.E, a.k, a.hdr};
    const cudaError_t e = api_launch(w4_combine_kernel, dim3((a.N + 1023) / 1024, rows), 256, 0, stream, ca);
    if (e != cudaSuccess) return api_fail_cuda(e, "launch of the sum over a token's experts");
    return ET_OK;
}

// f with the group size as a constant.
template <class F>
int w4_by_group(int group, F&& f) {
    if (group == 32) return f(std::integral_constant<int, 32>{});
    if (group == 64) return f(std::integral_constant<int, 64>{});
    return f(std::integral_constant<int, 128>{});
}

int w4_conv_check(int E, int N, int K, int group) {
    std::string why;
    if (!w4_shape_ok(N, K, group, &why)) return api_fail(ET_ERR_UNSUPPORTED, why);
    if (E < 1 || static_cast<long long>(E) * N > (1ll << 32))
        return api_fail(ET_ERR_UNSUPPORTED, "E must be positive, E * N at most 2^32");
    return ET_OK;
}

// Rows in the grid's x (8 a CTA), inputs in chunks of 4096 in its y -- of 1024
// when that leaves fewer than two CTAs an SM.
dim3 w4_conv_grid(W4ConvArgs* a, int E, int sms) {
    const long long tiles = static_cast<long long>(E) * a->N / kConvRows;
    a->chunk = tiles * ((a->K + kConvK - 1) / kConvK) < 2ll * sms ? 1024 : kConvK;
    return dim3(static_cast<unsigned>(tiles), (a->K + a->chunk - 1) / a->chunk);
}

// Workspace: header, h [T_max k, F] bf16, a routed row's share of the output [T_max k, H]
// fp32.
size_t w4_h_end(int T_max, int F, int k) {
    return (kHeaderBytes + sizeof(uint16_t) * static_cast<size_t>(T_max) * k * F + 255) / 256 * 256;
}
size_t w4_experts_bytes(int T_max, int H, int F, int k) {
    return w4_h_end(T_max, F, k) + (sizeof(float) * static_cast<size_t>(T_max) * k * H + 255) / 256 * 256;
}

bool w4_experts_ok(int T_max, int H, int F, int E, int k, int group, std::string* why) {
    if (T_max < 1 || T_max > kW4RowsMax) { *why = "T_max must be in [1, 64]"; return false; }
    if (E < 1 || E > kW4EMax) { *why = "E must be in [1, 256]"; return false; }
    if (k < 1 || k > kW4KMax || k > E) { *why = "k must be in [1, min(E, 8)]"; return false; }
    return w4_shape_ok(H, F, group, why) && w4_shape_ok(F, H, group, why);
}

}  // namespace
}  // namespace et

using namespace et;

extern "C" {

int et_w4_quantize(const void* w, void* q, void* scale, int E, int N, int K, int group, void* stream) {
    return api_entry([&]() -> int {
        int rc = w4_conv_check(E, N, K, group);
        if (rc) return rc;
        if (!w || !q || !scale) return api_fail(ET_ERR_INVALID, "w, q and scale must be non-NULL");
        if (!api_aligned(w, 16) || !api_aligned(q, 16) || !api_aligned(scale, 16))
            return api_fail(ET_ERR_INVALID, "tensors must be 16-byte aligned");
        int dev = 0, sms = 0;
        if ((rc = api_device(&dev, &sms))) return rc;
        W4ConvArgs a{};
        a.w = static_cast<const bf16*>(w);
        a.q_out = static_cast<uint8_t*>(q);
        a.s_out = static_cast<bf16*>(scale);
        a.N = N;
        a.K = K;
        const dim3 grid = w4_conv_grid(&a, E, sms);
        const cudaError_t e = api_launch(group == 32 ? w4_quantize_kernel<32> : group == 64 ? w4_quantize_kernel<64>
                                                                   : w4_quantize_kernel<128>,
                                          grid, kConvRows * 32, 0, stream, a);
        if (e != cudaSuccess) return api_fail_cuda(e, "launch of the 4-bit quantiser");
        return ET_OK;
    });
}

int et_w4_dequantize(const void* q, const void* scale, void* w, int E, int N, int K, int group, void* stream) {
    return api_entry([&]() -> int {
        int rc = w4_conv_check(E, N, K, group);
        if (rc) return rc;
        if (!w || !q || !scale) return api_fail(ET_ERR_INVALID, "q, scale and w must be non-NULL");
        if (!api_aligned(w, 16) || !api_aligned(q, 16) || !api_aligned(scale, 16))
            return api_fail(ET_ERR_INVALID, "tensors must be 16-byte aligned");
        int dev = 0, sms = 0;
        if ((rc = api_device(&dev, &sms))) return rc;
        W4ConvArgs a{};
        a.q = static_cast<const uint8_t*>(q);
        a.s = static_cast<const bf16*>(scale);
        a.w_out = static_cast<bf16*>(w);
        a.N = N;
        a.K = K;
        const dim3 grid = w4_conv_grid(&a, E, sms);
        const cudaError_t e = api_launch(group == 32 ? w4_dequantize_kernel<32> : group == 64 ? w4_dequantize_kernel<64>
                                                                     : w4_dequantize_kernel<128>,
                                          grid, kConvRows * 32, 0, stream, a);
        if (e != cudaSuccess) return api_fail_cuda(e, "launch of the 4-bit expansion");
        return ET_OK;
    });
}

size_t et_w4_gemv_workspace_bytes(int M_max, int N, int K, int group) {
    try {
        std::string why;
        if (M_max < 1 || M_max > kW4RowsMax || !w4_shape_ok(N, K, group, &why)) return 0;
        return kHeaderBytes;
    } catch (...) {
        return 0;
    }
}

int et_w4_gemv(const void* X, const void* q, const void* scale, void* Y, int M, const int32_t* d_M,
               int M_max, int N, int K, int group, void* workspace, size_t workspace_bytes, void* stream) {
    return api_entry([&]() -> int {
        std::string why;
        if (!w4_shape_ok(N, K, group, &why)) return api_fail(ET_ERR_UNSUPPORTED, why);
        if (M_max < 1 || M_max > kW4RowsMax)
            return api_fail(ET_ERR_UNSUPPORTED, "M_max must be in [1, 64] (et_w4_dequantize and "
                                                "et_splitk_gemm serve larger batches)");
        if (!X || !q || !scale || !Y) return api_fail(ET_ERR_INVALID, "X, q, scale and Y must be non-NULL");
        if (!api_aligned(X, 16) || !api_aligned(q, 16) || !api_aligned(scale, 16) || !api_aligned(Y, 16))
            return api_fail(ET_ERR_INVALID, "tensors must be 16-byte aligned");
        if (!api_aligned(d_M, 4)) return api_fail(ET_ERR_INVALID, "d_M must be 4-byte aligned");
        if (!d_M && (M < 0 || M > M_max)) return api_fail(ET_ERR_INVALID, "M must be in [0, M_max]");
        int rc = api_check_ws(workspace, workspace_bytes, kHeaderBytes);
        if (rc) return rc;
        if (!d_M && M == 0) return ET_OK;
        int dev = 0, sms = 0;
        if ((rc = api_device(&dev, &sms))) return rc;
        W4Args a{};
        a.x = static_cast<const bf16*>(X);
        a.q0 = static_cast<const uint8_t*>(q);
        a.s0 = static_cast<const bf16*>(scale);
        a.out = static_cast<bf16*>(Y);
        a.d_T = d_M;
        a.T_host = M;
        a.T_max = M_max;
        a.N = N;
        a.K = K;
        a.E = 1;
        a.k = 1;
        a.hdr = static_cast<EtHeader*>(workspace);
        const int rows = d_M ? M_max : M;
        return w4_by_group(group, [&](auto g) { return w4_launch_gemv<decltype(g)::value>(a, rows, dev, sms, stream); });
    });
}

size_t et_w4_experts_workspace_bytes(int T_max, int H, int F, int E, int k, int group) {
    try {
        std::string why;
        if (!w4_experts_ok(T_max, H, F, E, k, group, &why)) return 0;
        return w4_experts_bytes(T_max, H, F, k);
    } catch (...) {
        return 0;
    }
}

int et_w4_experts(const void* x, const int32_t* topk_idx, const float* topk_w, const void* q_gate,
                  const void* s_gate, const void* q_up, const void* s_up, const void* q_down,
                  const void* s_down, void* out, int T, const int32_t* d_T, int T_max, int H, int F,
                  int E, int k, int group, void* workspace, size_t workspace_bytes, void* stream) {
    return api_entry([&]() -> int {
        std::string why;
        if (!w4_experts_ok(T_max, H, F, E, k, group, &why)) return api_fail(ET_ERR_UNSUPPORTED, why);
        const void* need16[] = {x, q_gate, s_gate, q_up, s_up, q_down, s_down, out};
        for (const void* v : need16) {
            if (!v) return api_fail(ET_ERR_INVALID, "x, the weights, their scales and out must be non-NULL");
            if (!api_aligned(v, 16)) return api_fail(ET_ERR_INVALID, "tensors must be 16-byte aligned");
        }
        if (!topk_idx || !topk_w) return api_fail(ET_ERR_INVALID, "topk_idx and topk_w must be non-NULL");
        if (!api_aligned(topk_idx, 4) || !api_aligned(topk_w, 4) || !api_aligned(d_T, 4))
            return api_fail(ET_ERR_INVALID, "tensors must be aligned to their element size");
        if (!d_T && (T < 0 || T > T_max)) return api_fail(ET_ERR_INVALID, "T must be in [0, T_max]");
        int rc = api_check_ws(workspace, workspace_bytes, w4_experts_bytes(T_max, H, F, k));
        if (rc) return rc;
        if (!d_T && T == 0) return ET_OK;
        int dev = 0, sms = 0;
        if ((rc = api_device(&dev, &sms))) return rc;
        uint8_t* ws = static_cast<uint8_t*>(workspace);
        bf16* h = reinterpret_cast<bf16*>(ws + kHeaderBytes);
        W4Args a{};
        a.x = static_cast<const bf16*>(x);
        a.q0 = static_cast<const uint8_t*>(q_gate);
        a.q1 = static_cast<const uint8_t*>(q_up);
        a.s0 = static_cast<const bf16*>(s_gate);
        a.s1 = static_cast<const bf16*>(s_up);
        a.out = h;
        a.idx = topk_idx;
        a.w = topk_w;
        a.d_T = d_T;
        a.T_host = T;
        a.T_max = T_max;
        a.N = F;
        a.K = H;
        a.E = E;
        a.k = k;
        a.hdr = reinterpret_cast<EtHeader*>(ws);
        const int rows = d_T ? T_max : T, R = rows * k;
        // Rows a pass takes, 4, 8 or 16, by the rows an expert has on average.  More save passes
        // over experts with many, and cost shared memory (CTAs an SM) and, from 9 on, a second
        // tile of columns in every product; long sums (H) repay that sooner.  Microseconds with
        // 4 and 8 rows at an average of 1: fine-grained, T = 5 31.2 and 32.4; of 2: T = 32 77.1
        // and 72.3, E 8, 4096 x 14336 164 and 154, 30 other calls 0 to 18 % apart, 8 never the slower by
        // more than 1; with 8 and 16 at 8: 246 and 206, E 32, 2048 x 768 34.8 and 53.8; at 16: 397
        // and 339, E 8, 2048 x 768 21.7 and 31.7 (but E 4, 1024 x 4096 at 32: 48.0 and 43.6).
        // In between the two come near: E 16, 3584 x 2560 at 8 82.8 and 81.0, 83 and 92 with
        // k = 2; E 8, 3200 x 6400 at 16 138 and 142.
        const int avg = (R + E - 1) / E;
        const bool deep = H >= 4096;
        int width = avg <= 1 ? 4 : avg < 8 || !deep ? 8 : 16;
        width = rows < width ? rows : width;
        rc = w4_by_group(group, [&](auto g) { return w4_launch_gate_up<decltype(g)::value>(a, rows, width, dev, sms, stream); });
        if (rc) return rc;
        W4Args b = a;
        b.x = h;
        b.q0 = static_cast<const uint8_t*>(q_down);
        b.s0 = static_cast<const bf16*>(s_down);
        b.q1 = nullptr;
        b.s1 = nullptr;
        b.out = static_cast<bf16*>(out);
        b.N = H;
        b.K = F;
        b.y = reinterpret_cast<float*>(ws + w4_h_end(T_max, F, k));
        return w4_by_group(group, [&](auto g) { return w4_launch_down<decltype(g)::value>(b, rows, width, dev, sms, stream); });
    });
}

}  // extern "C"
