// w4_ops.cu -- products with 4-bit weights for a few rows (decoding), the
// routed SwiGLU experts over such weights, and the weights' own conversion.
//
//   w[n, k] = scale[k / group, n] * (q[n, k] - 8),  q in 0..15
//
// q is row-major, two inputs a byte (the even one in the low half); scale is
// bf16 with the group first, so that a tile of rows reads consecutive scales.
#include <cmath>

#include "../../include/etmoe.h"
#include "et_api.h"
#include "ops_device.cuh"

namespace et {
namespace {

constexpr int kW4Rows = 64;        // weight rows of a CTA (gate/up: 32 of each)
constexpr int kW4Blk = 128;        // inputs of a stage: 64 bytes of a row
constexpr int kW4Warps = 4;
constexpr int kW4Stages = 4;
constexpr int kW4RowsMax = 64;     // most rows of x (tokens)
constexpr int kW4KMax = 8;         // experts of a token
constexpr int kW4EMax = 256;
constexpr int kW4ClusterMax = 8;
constexpr int kW4Pad = kW4Rows + 8;  // row length of a CTA's fp32 tile, padded against bank conflicts

enum W4Mode { kW4Gemv = 0, kW4GateUp = 1, kW4Down = 2 };

struct W4Args {
    const bf16* x;            // [rows, K]
    const uint8_t *q0, *q1;   // [E][N, K/2]; q1: the up projection
    const bf16 *s0, *s1;      // [E][K/group, N]
    bf16* out;                // [rows, N]
    const int32_t* idx;       // [T, k]
    const float* w;           // [T, k]
    const int32_t* d_T;
    int T_host, T_max, N, K, group, E, k;
    EtHeader* hdr;
    int x_rows;               // rows of x a stage holds = rows of a pass or segment
    int stage_bytes;
};

// The warp's own ring: each stage is [64 rows][64 B] of weights, x_rows rows of
// 256 B of x, and 128 / group rows of 64 scales.  16-byte pieces are swizzled
// so that the fragment reads below touch every bank once.
struct W4Stage {
    uint32_t w, x, s;
};

__device__ __forceinline__ W4Stage stage_at(const W4Args& p, uint32_t base, int slot) {
    const uint32_t b = base + slot * p.stage_bytes;
    return {b, b + kW4Rows * 64, b + kW4Rows * 64 + static_cast<uint32_t>(p.x_rows) * 256};
}

// Post the copies of k-block kb: weights of rows [n0, n0 + 64) (gate/up: 32 + 32),
// x rows cols[0..nc), scales.  Pieces outside the matrices are filled with zeros.
template <int MODE>
__device__ __forceinline__ void load_stage(const W4Args& p, const W4Stage& st, int e, int n0, int kb,
                                           const int* cols, int nc) {
    const int lane = threadIdx.x & 31;
    const int k0 = kb * kW4Blk;
    {
        const int c = lane & 3;
        const bool kin = k0 + c * 32 < p.K;
        const size_t ld = static_cast<size_t>(p.K) / 2;
        const size_t base = static_cast<size_t>(e) * p.N * ld + k0 / 2 + c * 16;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = (lane >> 2) + 8 * i;
            const int n = MODE == kW4GateUp ? n0 + (r & 31) : n0 + r;
            const uint8_t* q = (MODE == kW4GateUp && i >= 4) ? p.q1 : p.q0;
            const bool in = kin && n < p.N;
            cp_async16(st.w + r * 64 + ((c ^ ((r >> 1) & 3)) << 4), in ? q + base + n * ld : q, in);
        }
    }
    {
        const int c = lane & 15;
        const bool kin = k0 + c * 8 < p.K;
        for (int r = lane >> 4; r < nc; r += 2)
            cp_async16(st.x + r * 256 + ((c ^ ((r & 1) << 2)) << 4),
                       kin ? p.x + static_cast<size_t>(cols[r]) * p.K + k0 + c * 8 : p.x, kin);
    }
    {
        const int gs = kW4Blk / p.group;  // groups of a k-block: 1, 2 or 4, of 8 pieces each
        const int g = lane >> 3, c = lane & 7;
        if (g < gs) {
            const int gi = k0 / p.group + g;
            const int G = p.K / p.group;
            const int n = MODE == kW4GateUp ? n0 + (c & 3) * 8 : n0 + c * 8;
            const bf16* s = (MODE == kW4GateUp && c >= 4) ? p.s1 : p.s0;
            const bool in = gi < G && n < p.N;
            cp_async16(st.s + g * 128 + (c << 4),
                       in ? s + (static_cast<size_t>(e) * G + gi) * p.N + n : s, in);
        }
    }
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a));
    return v;
}
__device__ __forceinline__ float ld_shared_bf16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return __uint_as_float(static_cast<uint32_t>(v) << 16);
}

// Eight 4-bit values -> four packed pairs of q - 8 in bf16, pairs (0,4) (1,5)
// (2,6) (3,7).  0x4300 is 128.0 with a unit of 1 in its last place, so or-ing a
// nibble in gives 128 + q exactly, and subtracting 136 gives q - 8 exactly.
__device__ __forceinline__ void unpack8(uint32_t v, uint32_t (&o)[4]) {
    const __nv_bfloat162 off = __floats2bfloat162_rn(136.0f, 136.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t b = ((v >> (4 * i)) & 0x000f000fu) | 0x43004300u;
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&b), off);
        o[i] = *reinterpret_cast<const uint32_t*>(&d);
    }
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One k-block: acc += scale * ((q - 8) x), the bracket exact products summed in
// fp32 by the tensor core over a group, the scale applied in fp32 after it.
// A fragment: lane (r = lane / 4, t = lane % 4) holds inputs 8t .. 8t + 7 of
// each 32 (one 32-bit word) of rows r and r + 8; the order of the inputs inside
// a product is free as long as x follows it, and x is paired (0,4) (1,5) ...
// like the unpacked weights.
template <int NT>
__device__ __forceinline__ void compute_stage(const W4Args& p, const W4Stage& st, int nc,
                                              float (&acc)[4][NT][4]) {
    const int lane = threadIdx.x & 31;
    const int r = lane >> 2, t = lane & 3;
    const int per = p.group >> 5;  // 32-input pieces of a group
    float part[4][NT][4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if ((c & (per - 1)) == 0) {
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) part[m][j][i] = 0.0f;
        }
        uint32_t b[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int n = j * 8 + r;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (n < nc) v = ld_shared_v4(st.x + n * 256 + (((c * 4 + t) ^ ((n & 1) << 2)) << 4));
            b[j][0] = __byte_perm(v.x, v.z, 0x5410);
            b[j][1] = __byte_perm(v.x, v.z, 0x7632);
            b[j][2] = __byte_perm(v.y, v.w, 0x5410);
            b[j][3] = __byte_perm(v.y, v.w, 0x7632);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            uint32_t lo[4], hi[4];
            const uint32_t a = st.w + (m * 16 + r) * 64 + ((c ^ ((r >> 1) & 3)) << 4) + t * 4;
            unpack8(ld_shared_u32(a), lo);
            unpack8(ld_shared_u32(a + 8 * 64), hi);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                mma16816(part[m][j], lo[0], hi[0], lo[1], hi[1], b[j][0], b[j][1]);
                mma16816(part[m][j], lo[2], hi[2], lo[3], hi[3], b[j][2], b[j][3]);
            }
        }
        if (((c + 1) & (per - 1)) == 0) {
            const uint32_t sa = st.s + (c / per) * 128 + r * 2;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float s0 = ld_shared_bf16(sa + m * 32), s1 = ld_shared_bf16(sa + m * 32 + 16);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    acc[m][j][0] += s0 * part[m][j][0];
                    acc[m][j][1] += s0 * part[m][j][1];
                    acc[m][j][2] += s1 * part[m][j][2];
                    acc[m][j][3] += s1 * part[m][j][3];
                }
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
    int e[kW4RowsMax * kW4KMax];        // row -> expert (-1: none)
    int order[kW4RowsMax * kW4KMax];    // rows by expert, ascending within one
    int start[kW4EMax + 1];             // first entry of an expert in `order`
    int seg_e[kW4RowsMax * kW4KMax];    // segments: up to `width` rows of one expert
    int seg_r[kW4RowsMax * kW4KMax];
    int seg_n[kW4RowsMax * kW4KMax];
    int cnt[kW4EMax];
    int n_seg;
};

__device__ __forceinline__ void build_routing(const W4Args& p, W4Routing& rt, int T, int width) {
    const int R = T * p.k;
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) rt.cnt[e] = 0;
    __syncthreads();
    for (int r = threadIdx.x; r < R; r += blockDim.x) {
        int e = p.idx[r];
        if (e < -1 || e >= p.E) {
            record_status(p.hdr, ET_ERR_BOUNDS, kWhereExpertIndex);
            e = -1;
        }
        rt.e[r] = e;
        if (e >= 0) atomicAdd(&rt.cnt[e], 1);
    }
    __syncthreads();
    if (threadIdx.x < 32) {  // exclusive sums over experts: of rows and of segments
        const int lane = threadIdx.x;
        int rows = 0, segs = 0;
        for (int b = 0; b < p.E; b += 32) {
            const int e = b + lane;
            const int c = e < p.E ? rt.cnt[e] : 0;
            const int s = (c + width - 1) / width;
            int ci = c, si = s;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int a = __shfl_up_sync(0xffffffffu, ci, off), d = __shfl_up_sync(0xffffffffu, si, off);
                if (lane >= off) { ci += a; si += d; }
            }
            const int r0 = rows + ci - c;
            int s0 = segs + si - s;
            if (e < p.E) rt.start[e] = r0;
            for (int o = 0; o < c; o += width, ++s0) {
                rt.seg_e[s0] = e;
                rt.seg_r[s0] = r0 + o;
                rt.seg_n[s0] = min(width, c - o);
            }
            rows += __shfl_sync(0xffffffffu, ci, 31);
            segs += __shfl_sync(0xffffffffu, si, 31);
        }
        if (lane == 0) rt.n_seg = segs;
    }
    __syncthreads();
    for (int r = threadIdx.x; r < R; r += blockDim.x) {
        const int e = rt.e[r];
        if (e < 0) continue;
        int rank = 0;
        for (int o = 0; o < r; ++o) rank += rt.e[o] == e;
        rt.order[rt.start[e] + rank] = r;
    }
    __syncthreads();
}

// One CTA: 64 weight rows (gate/up: 32 + 32).  The inputs are split over the
// warps of the CTA and over the CTAs of its cluster; each warp streams its own
// k-blocks through its own ring, and no barrier sits in the loop.
//   kW4Gemv   x rows in chunks of x_rows <= 8 NT, all of K.
//   kW4GateUp blockIdx.y picks the segment: up to x_rows rows of one expert.
//   kW4Down   the work is the list of (segment, k-block); a warp adds what it
//             has for a segment, times the gate weight, to its own fp32 rows by
//             token, and the sum over warps and CTAs is the layer's output.
template <int MODE, int NT>
__global__ void __launch_bounds__(kW4Warps * 32) w4_kernel(const W4Args p) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int cols_s[MODE == kW4Down ? 1 : NT * 8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int csize = static_cast<int>(cluster_size()), crank = static_cast<int>(cluster_rank());
    const int unit = crank * kW4Warps + warp, units = csize * kW4Warps;
    constexpr int kOutRows = MODE == kW4GateUp ? 32 : 64;
    const int n0 = (blockIdx.x / csize) * kOutRows;
    const int KB = (p.K + kW4Blk - 1) / kW4Blk;
    bool ok;
    const int T = row_count(p.d_T, p.T_host, p.T_max, p.hdr, &ok);
    if (!ok) return;  // the same for every CTA of the cluster

    // shared memory: [routing][fp32 sums][rings]; the sums of the first two
    // modes lie over the rings, which are empty by then
    W4Routing& rt = *reinterpret_cast<W4Routing*>(smem);
    uint8_t* rest = smem + (MODE == kW4Gemv ? 0 : (sizeof(W4Routing) + 127) / 128 * 128);
    float* sums = reinterpret_cast<float*>(rest);
    if (MODE == kW4Down) rest += (static_cast<size_t>(kW4Warps) * T * kW4Pad * 4 + 127) / 128 * 128;
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(rest)) +
                          warp * kW4Stages * p.stage_bytes;
    if (MODE != kW4Gemv) build_routing(p, rt, T, p.x_rows);

    const int passes = MODE == kW4Gemv ? (T + p.x_rows - 1) / p.x_rows : 1;
    if (MODE == kW4GateUp && static_cast<int>(blockIdx.y) >= rt.n_seg) return;
    if (MODE == kW4Down)
        for (int i = threadIdx.x; i < kW4Warps * T * kW4Pad; i += blockDim.x) sums[i] = 0.0f;

    for (int pass = 0; pass < passes; ++pass) {
        int nc0 = 0, e0 = 0;
        if (MODE == kW4Gemv) {
            nc0 = min(p.x_rows, T - pass * p.x_rows);
            if (threadIdx.x < nc0) cols_s[threadIdx.x] = pass * p.x_rows + threadIdx.x;
        } else if (MODE == kW4GateUp) {
            nc0 = rt.seg_n[blockIdx.y];
            e0 = rt.seg_e[blockIdx.y];
            if (threadIdx.x < nc0) cols_s[threadIdx.x] = rt.order[rt.seg_r[blockIdx.y] + threadIdx.x] / p.k;
        }
        __syncthreads();

        const long long items = static_cast<long long>(MODE == kW4Down ? rt.n_seg : 1) * KB;
        const int i0 = static_cast<int>(items * unit / units), i1 = static_cast<int>(items * (unit + 1) / units);
        auto post = [&](int i) {
            if (i < i1) {
                const W4Stage st = stage_at(p, ring, (i - i0) % kW4Stages);
                if (MODE == kW4Down) {
                    const int s = i / KB;
                    load_stage<MODE>(p, st, rt.seg_e[s], n0, i - s * KB, rt.order + rt.seg_r[s], rt.seg_n[s]);
                } else {
                    load_stage<MODE>(p, st, e0, n0, i, cols_s, nc0);
                }
            }
            cp_async_commit();
        };
        float acc[4][NT][4];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.0f;
#pragma unroll
        for (int s = 0; s < kW4Stages - 1; ++s) post(i0 + s);
        for (int i = i0; i < i1; ++i) {
            cp_async_wait<kW4Stages - 2>();
            __syncwarp();
            post(i + kW4Stages - 1);
            const int seg = MODE == kW4Down ? i / KB : 0;
            const int nc = MODE == kW4Down ? rt.seg_n[seg] : nc0;
            compute_stage<NT>(p, stage_at(p, ring, (i - i0) % kW4Stages), nc, acc);
            if (MODE == kW4Down && (i + 1 == i1 || (i + 1) % KB == 0)) {
                // the quarter-warps in turn: a token may hold two rows of one segment
                float* mine = sums + static_cast<size_t>(warp) * T * kW4Pad;
                const int r = lane >> 2, t = lane & 3;
                for (int q = 0; q < 4; ++q) {
                    if (t == q) {
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int col = j * 8 + 2 * t + h;
                                if (col < nc) {
                                    const int row = rt.order[rt.seg_r[seg] + col];
                                    const float wt = p.w[row];
                                    float* dst = mine + (row / p.k) * kW4Pad + r;
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
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int z = 0; z < 4; ++z) acc[m][j][z] = 0.0f;
            }
        }
        cp_async_wait<0>();
        __syncthreads();  // the rings are empty

        // sums over the CTA's warps, in order, into the first warp's tile
        const int nc = MODE == kW4Down ? T : nc0;
        if (MODE != kW4Down) {
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
            __syncthreads();
        }
        for (int o = threadIdx.x; o < nc * kW4Rows; o += blockDim.x) {
            const int at = (o >> 6) * kW4Pad + (o & 63);
            float v = sums[at];
#pragma unroll
            for (int w = 1; w < kW4Warps; ++w) v += sums[w * nc * kW4Pad + at];
            sums[at] = v;
        }
        // sums over the cluster's CTAs, in order; each CTA stores its share
        if (csize > 1) cluster_sync();
        else __syncthreads();
        const uint32_t sums_u = static_cast<uint32_t>(__cvta_generic_to_shared(sums));
        for (int o = crank * blockDim.x + threadIdx.x; o < nc * kOutRows; o += csize * blockDim.x) {
            const int col = o / kOutRows, row = o % kOutRows;
            const int n = n0 + row;
            auto total = [&](int rr) {
                const uint32_t at = sums_u + (col * kW4Pad + rr) * 4;
                if (csize == 1) return sums[col * kW4Pad + rr];
                float v = 0.0f;
                for (int c = 0; c < csize; ++c) v += ld_cluster_f32(at, c);
                return v;
            };
            if (n < p.N) {
                if (MODE == kW4GateUp) {
                    const float g = total(row), u = total(row + 32);
                    const float h = g / (1.0f + expf(-g)) * u;
                    const int rr = rt.order[rt.seg_r[blockIdx.y] + col];
                    p.out[static_cast<size_t>(rr) * p.N + n] = __float2bfloat16_rn(h);
                } else {
                    const int m = MODE == kW4Gemv ? pass * p.x_rows + col : col;
                    p.out[static_cast<size_t>(m) * p.N + n] = __float2bfloat16_rn(total(row));
                }
            }
        }
        // no CTA may leave, or overwrite its sums, while another reads them
        if (csize > 1) cluster_sync();
        else __syncthreads();
    }
}

// ---------------------------------------------------------------- conversion

struct W4ConvArgs {
    const bf16* w;
    const uint8_t* q;
    const bf16* s;
    bf16* w_out;
    uint8_t* q_out;
    bf16* s_out;
    int N, K, group;
    long long rows;  // E * N
};

// Eight inputs a thread: 16 bytes in, 4 bytes out; the lanes of a group (4, 8 or
// 16) share its largest magnitude by shuffles.
__global__ void __launch_bounds__(256) w4_quantize_kernel(const W4ConvArgs p) {
    const int per = p.K / 8;  // vectors of a row: a multiple of 4, groups never cross a row
    const long long total = p.rows * per;
    const int lanes = p.group / 8;
    const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
    // whole warps run to the last vector, so that every shuffle has its partners
    const long long end = (total + 31) / 32 * 32;
    for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < end; i += stride) {
        const bool in = i < total;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (in) v = reinterpret_cast<const uint4*>(p.w)[i];
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
        float f[8];
        uint32_t top = 0;  // largest magnitude as bits: NaN above infinity above all numbers
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            f[j] = (j & 1) ? bf_hi(u[j >> 1]) : bf_lo(u[j >> 1]);
            top = max(top, __float_as_uint(f[j]) & 0x7fffffffu);
        }
        for (int off = 1; off < lanes; off <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
        const bool finite = top < 0x7f800000u;
        const __nv_bfloat16 sb = finite ? __float2bfloat16_rn(__uint_as_float(top) / 7.0f)
                                        : __float2bfloat16_rn(__uint_as_float(0x7fc00000u));
        const float s = __bfloat162float(sb);
        uint32_t out = 0x88888888u;  // zeros, where the scale is zero or not a number
        if (s > 0.0f) {
            out = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float r = fminf(fmaxf(rintf(f[j] / s), -8.0f), 7.0f);
                out |= static_cast<uint32_t>(static_cast<int>(r) + 8) << (4 * j);
            }
        }
        if (in) {
            reinterpret_cast<uint32_t*>(p.q_out)[i] = out;
            if ((i & (lanes - 1)) == 0) {
                const long long row = i / per;
                const int g = static_cast<int>(i - row * per) / lanes;
                const long long e = row / p.N;
                const int n = static_cast<int>(row - e * p.N);
                p.s_out[(e * (p.K / p.group) + g) * p.N + n] = sb;
            }
        }
    }
}

__global__ void __launch_bounds__(256) w4_dequantize_kernel(const W4ConvArgs p) {
    const int per = p.K / 8;
    const long long total = p.rows * per;
    const int lanes = p.group / 8;
    const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
    for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += stride) {
        const uint32_t q = reinterpret_cast<const uint32_t*>(p.q)[i];
        const long long row = i / per;
        const int g = static_cast<int>(i - row * per) / lanes;
        const long long e = row / p.N;
        const int n = static_cast<int>(row - e * p.N);
        const float s = __bfloat162float(p.s[(e * (p.K / p.group) + g) * p.N + n]);
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o[j] = pack_bf16(s * (static_cast<int>((q >> (8 * j)) & 15u) - 8),
                             s * (static_cast<int>((q >> (8 * j + 4)) & 15u) - 8));
        reinterpret_cast<uint4*>(p.w_out)[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// ---------------------------------------------------------------- launches

bool w4_shape_ok(int N, int K, int group, std::string* why) {
    if (group != 32 && group != 64 && group != 128) { *why = "group must be 32, 64 or 128"; return false; }
    if (K < group || K % group || K > (1 << 20)) { *why = "inputs must be a positive multiple of group (<= 2^20)"; return false; }
    if (N < 8 || N % 8 || N > (1 << 20)) { *why = "outputs must be a positive multiple of 8 (<= 2^20)"; return false; }
    return true;
}

// CTAs that share a tile's inputs: doubled while the grid stays below two CTAs
// an SM and every warp keeps two k-blocks.
int w4_cluster(long long ctas, long long blocks, int sms) {
    int c = 1;
    while (c < kW4ClusterMax && ctas * c * 2 <= 2 * sms && blocks >= 2ll * kW4Warps * c * 2) c *= 2;
    return c;
}

SmemOptIn g_w4_opt[3][3];

// `rows` tokens at most; x_rows <= 8 NT of them (or of an expert's rows) a pass.
template <int MODE, int NT>
int w4_launch(W4Args a, int rows, int x_rows, int dev, int sms, void* stream) {
    constexpr int kOutRows = MODE == kW4GateUp ? 32 : 64;
    constexpr int kSmemMost = kSmemLimit - 1024;  // the column list is static
    a.x_rows = x_rows;
    a.stage_bytes = kW4Rows * 64 + x_rows * 256 + (kW4Blk / a.group) * 128;
    const size_t rings = static_cast<size_t>(kW4Warps) * kW4Stages * a.stage_bytes;
    const int sum_rows = MODE == kW4Down ? rows : x_rows;
    const size_t sums = (static_cast<size_t>(kW4Warps) * sum_rows * kW4Pad * 4 + 127) / 128 * 128;
    const size_t routing = MODE == kW4Gemv ? 0 : (sizeof(W4Routing) + 127) / 128 * 128;
    const size_t smem = routing + (MODE == kW4Down ? sums + rings : (sums > rings ? sums : rings));
    if (smem > kSmemMost) return api_fail(ET_ERR_UNSUPPORTED, "rows do not fit in shared memory");
    constexpr int kNi = NT == 1 ? 0 : NT == 2 ? 1 : 2;
    cudaError_t e = api_smem_opt_in(g_w4_opt[MODE][kNi], dev, w4_kernel<MODE, NT>, kSmemMost);
    if (e != cudaSuccess) return api_fail_cuda(e, "cudaFuncSetAttribute(4-bit products)");
    // segments of a call: each has a row, an expert has one and one more for each full pass
    const int R = rows * a.k, experts = R < a.E ? R : a.E;
    const int slots = MODE == kW4Gemv ? 1 : (experts + R / x_rows < R ? experts + R / x_rows : R);
    const int tiles = (a.N + kOutRows - 1) / kOutRows;
    const long long blocks = static_cast<long long>((a.K + kW4Blk - 1) / kW4Blk) * (MODE == kW4Down ? slots : 1);
    const int c = w4_cluster(static_cast<long long>(tiles) * (MODE == kW4GateUp ? slots : 1), blocks, sms);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(tiles * c, MODE == kW4GateUp ? slots : 1);
    cfg.blockDim = dim3(kW4Warps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = c;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, w4_kernel<MODE, NT>, a);
    if (e != cudaSuccess) return api_fail_cuda(e, "launch of the 4-bit product kernel");
    return ET_OK;
}

template <int MODE>
int w4_launch_nt(const W4Args& a, int rows, int x_rows, int dev, int sms, void* stream) {
    if (x_rows <= 8) return w4_launch<MODE, 1>(a, rows, x_rows, dev, sms, stream);
    if (x_rows <= 16) return w4_launch<MODE, 2>(a, rows, x_rows, dev, sms, stream);
    return w4_launch<MODE, 4>(a, rows, x_rows, dev, sms, stream);
}

int w4_conv_check(int E, int N, int K, int group) {
    std::string why;
    if (!w4_shape_ok(N, K, group, &why)) return api_fail(ET_ERR_UNSUPPORTED, why);
    if (E < 1 || E > 65536) return api_fail(ET_ERR_UNSUPPORTED, "E must be in [1, 65536]");
    return ET_OK;
}

int w4_conv_grid(const W4ConvArgs& a, int sms) {
    const long long ctas = (a.rows * (a.K / 8) + 255) / 256;
    return static_cast<int>(ctas < 32ll * sms ? ctas : 32ll * sms);
}

size_t w4_experts_bytes(int T_max, int F, int k) {
    return (kHeaderBytes + sizeof(uint16_t) * static_cast<size_t>(T_max) * k * F + 255) / 256 * 256;
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
        a.group = group;
        a.rows = static_cast<long long>(E) * N;
        const cudaError_t e = api_launch(w4_quantize_kernel, w4_conv_grid(a, sms), 256, 0, stream, a);
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
        a.group = group;
        a.rows = static_cast<long long>(E) * N;
        const cudaError_t e = api_launch(w4_dequantize_kernel, w4_conv_grid(a, sms), 256, 0, stream, a);
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
        a.group = group;
        a.E = 1;
        a.k = 1;
        a.hdr = static_cast<EtHeader*>(workspace);
        const int rows = d_M ? M_max : M;
        return w4_launch_nt<kW4Gemv>(a, rows, rows < 32 ? rows : 32, dev, sms, stream);
    });
}

size_t et_w4_experts_workspace_bytes(int T_max, int H, int F, int E, int k, int group) {
    try {
        std::string why;
        if (!w4_experts_ok(T_max, H, F, E, k, group, &why)) return 0;
        return w4_experts_bytes(T_max, F, k);
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
        int rc = api_check_ws(workspace, workspace_bytes, w4_experts_bytes(T_max, F, k));
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
        a.group = group;
        a.E = E;
        a.k = k;
        a.hdr = reinterpret_cast<EtHeader*>(ws);
        const int rows = d_T ? T_max : T, R = rows * k;
        // a pass takes the rows an expert has on average, with room for twice as many;
        // the down products also keep fp32 rows by token, which leaves room for 16
        const int avg = (R + E - 1) / E;
        const int width = avg <= 4 ? 8 : avg <= 8 ? 16 : 32;
        const int up_rows = rows < width ? rows : width, down_rows = up_rows < 16 ? up_rows : 16;
        if ((rc = w4_launch_nt<kW4GateUp>(a, rows, up_rows, dev, sms, stream))) return rc;
        W4Args b = a;
        b.x = h;
        b.q0 = static_cast<const uint8_t*>(q_down);
        b.s0 = static_cast<const bf16*>(s_down);
        b.q1 = nullptr;
        b.s1 = nullptr;
        b.out = static_cast<bf16*>(out);
        b.N = H;
        b.K = F;
        return w4_launch_nt<kW4Down>(b, rows, down_rows, dev, sms, stream);
    });
}

}  // extern "C"
