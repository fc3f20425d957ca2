// layer_norm_ops.cu -- a block's residual with dropout and the layer norm before
// the next block, in one pass; their gradient; dropout by itself.
//
//   z = x + dropout(y);  n = (z - mean z) / sqrt(var z + eps);  x_hat = n gamma + beta
//
// The mask is never stored: forward and backward draw it again from a counter
// (Philox4x32-10: Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy
// as 1, 2, 3", SC 2011).  Sixteen bits an element serve eight elements, one
// 16-byte access, with one block of the generator.
#include <cmath>

#include "../../include/etmoe.h"
#include "et_api.h"
#include "row_ops.cuh"

namespace et {
namespace {

constexpr int kLnParts = 304;   // most CTAs of the backward kernel = rows of partial sums
constexpr int kLnChain = 256;   // rows that a thread adds up before it puts the sums away

// ---------------------------------------------------------------- the mask

struct DropArgs {
    uint64_t seed, offset;
    const uint64_t* d_rng;  // {seed, offset} on the device, or null
    uint32_t thr;           // kept: 16 random bits >= thr; 0: everything is
    float mul;              // 65536 / (65536 - thr)
};

struct DropKey {
    uint32_t k0, k1, o0, o1;
    // What every lane holds, by a warp reduction: the ten rounds' keys stay in uniform registers.
    static __device__ __forceinline__ uint32_t same(uint32_t v) { return __reduce_or_sync(0xffffffffu, v); }
    __device__ __forceinline__ explicit DropKey(const DropArgs& d) : k0(0), k1(0), o0(0), o1(0) {
        if (!d.thr) return;
        uint64_t s = d.seed, o = d.offset;
        if (d.d_rng) {
            s = d.d_rng[0];
            o = d.d_rng[1];
        }
        k0 = same(static_cast<uint32_t>(s));
        k1 = same(static_cast<uint32_t>(s >> 32));
        o0 = same(static_cast<uint32_t>(o));
        o1 = same(static_cast<uint32_t>(o >> 32));
    }
};

// 16 random bits for each of the elements 8 h8 .. 8 h8 + 7 of row t: element i has the
// low (even i) or high half of word i / 2.
__device__ __forceinline__ uint4 drop_bits(const DropKey& k, uint32_t h8, uint32_t t) {
    uint32_t a = h8, b = t, c = k.o0, d = k.o1, k0 = k.k0, k1 = k.k1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p = static_cast<uint64_t>(a) * 0xD2511F53u, q = static_cast<uint64_t>(c) * 0xCD9E8D57u;
        a = static_cast<uint32_t>(q >> 32) ^ b ^ k0;
        c = static_cast<uint32_t>(p >> 32) ^ d ^ k1;
        b = static_cast<uint32_t>(q);
        d = static_cast<uint32_t>(p);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(a, b, c, d);
}

// What is kept of eight packed bf16: ones over the elements whose 16 bits are at least thr
// (> 0), two at a time: max(bits, thr - 1) - (thr - 1), then at most 1.
struct Mask8 { uint32_t u[4]; };
__device__ __forceinline__ Mask8 keep_all() { return Mask8{{~0u, ~0u, ~0u, ~0u}}; }
__device__ __forceinline__ Mask8 keep_mask8(const DropKey& k, uint32_t thr, uint32_t h8, uint32_t t) {
    const uint4 w = drop_bits(k, h8, t);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    const uint32_t below = (thr - 1) * 0x10001u, minus = ((1 - thr) & 0xffffu) * 0x10001u;
    Mask8 m;
#pragma unroll
    for (int i = 0; i < 4; ++i) m.u[i] = __viaddmin_u16x2(__vmaxu2(u[i], below), minus, 0x10001u) * 0xffffu;
    return m;
}

// Bit i: element i of the eight is dropped.
__device__ __forceinline__ uint32_t dropped_bits(const Mask8& m) {
    uint32_t b = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) b |= (m.u[i] & 1u) << (2 * i) | (m.u[i] >> 31) << (2 * i + 1);
    return b ^ 0xffu;
}

// ---------------------------------------------------------------- dropout by itself

struct DropoutArgs {
    const bf16* x;  // [T, H] or null
    const bf16* y;  // [T, H]
    bf16* out;
    DropArgs drop;
    const int32_t* d_T;
    int T_host, T_max, H;
    int rows;        // of a CTA
    uint32_t magic;  // i / H8 = umulhi(i, magic) for i below rows * H8 (H8 > 1)
    EtHeader* hdr;
};

constexpr int kDropThreads = 256;
constexpr int kDropCols = 2048;  // columns of a CTA without VEC

// Eight elements of one 16-byte access each, four accesses of a thread on their way.  Bound
// by HBM with x (8192 x 4096: 30 us, 6.7 TB/s, the rate of a copy); without it (23 us, 5.8
// TB/s) the mask's 7.6 of some 14 instructions an element show.
__global__ void __launch_bounds__(kDropThreads) dropout_vec_kernel(const DropoutArgs p) {
    grid_begin();
    bool ok;
    const int T = row_count(p.d_T, p.T_host, p.T_max, p.hdr, &ok);
    const int t0 = blockIdx.x * p.rows;
    if (t0 >= T) return;
    const int H8 = p.H >> 3;
    const int n = min(p.rows, T - t0) * H8;
    const size_t base = static_cast<size_t>(t0) * H8;
    const uint4* y = reinterpret_cast<const uint4*>(p.y) + base;
    const uint4* x = p.x ? reinterpret_cast<const uint4*>(p.x) + base : nullptr;
    uint4* out = reinterpret_cast<uint4*>(p.out) + base;
    const DropKey key(p.drop);
    constexpr int U = 4;
    for (int i0 = threadIdx.x; i0 < n; i0 += U * kDropThreads) {
        uint4 yv[U], xv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kDropThreads;
            yv[u] = xv[u] = make_uint4(0, 0, 0, 0);
            if (i < n) {
                yv[u] = y[i];
                if (x) xv[u] = x[i];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kDropThreads;
            if (i >= n) break;
            const uint32_t row = H8 > 1 ? __umulhi(i, p.magic) : i;
            const Mask8 m = p.drop.thr ? keep_mask8(key, p.drop.thr, i - row * H8, t0 + row) : keep_all();
            const uint32_t yw[4] = {yv[u].x, yv[u].y, yv[u].z, yv[u].w}, xw[4] = {xv[u].x, xv[u].y, xv[u].z, xv[u].w};
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // (one rounding, as in the norm; without x its zeros)
                const float2 v = __ffma2_rn(unpack2(yw[j] & m.u[j]), both(p.drop.mul), unpack2(xw[j]));
                o[j] = pack_bf16(v.x, v.y);
            }
            out[i] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// Any H and alignment: a CTA takes 2048 columns of a row, draws their mask into
// shared memory, then neighbouring threads take neighbouring elements.  Bound by its
// 2-byte accesses and its short CTAs (8000 x 1001: 21 us, 2.3 TB/s).
__global__ void __launch_bounds__(kDropThreads) dropout_any_kernel(const DropoutArgs p) {
    __shared__ uint8_t dropped[kDropCols / 8];
    grid_begin();
    bool ok;
    const int T = row_count(p.d_T, p.T_host, p.T_max, p.hdr, &ok);
    const int pieces = (p.H + kDropCols - 1) / kDropCols;
    const int t = blockIdx.x / pieces, c0 = (blockIdx.x - t * pieces) * kDropCols;
    if (t >= T) return;
    const int n = min(kDropCols, p.H - c0);
    const DropKey key(p.drop);
    static_assert(kDropCols / 8 == kDropThreads, "a thread draws eight elements");
    dropped[threadIdx.x] = p.drop.thr ? dropped_bits(keep_mask8(key, p.drop.thr, c0 / 8 + threadIdx.x, t)) : 0u;
    __syncthreads();
    const size_t off = static_cast<size_t>(t) * p.H + c0;
    bf16 yv[8], xv[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = threadIdx.x + i * kDropThreads;
        yv[i] = xv[i] = __float2bfloat16_rn(0.0f);
        if (c < n) {
            yv[i] = p.y[off + c];
            if (p.x) xv[i] = p.x[off + c];
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = threadIdx.x + i * kDropThreads;
        if (c < n) {
            const float y = dropped[c >> 3] >> (c & 7) & 1 ? 0.0f : __bfloat162float(yv[i]);
            p.out[off + c] = __float2bfloat16_rn(fmaf(y, p.drop.mul, __bfloat162float(xv[i])));
        }
    }
}

// ---------------------------------------------------------------- layer norm

struct LnArgs {
    const bf16* x;        // [T, H]
    const bf16* y;        // [T, H] or null
    const bf16* gamma;    // [H] or null (1)
    const bf16* beta;     // [H] or null (0)
    DropArgs drop;
    float eps, inv_H;
    int row_threads;      // threads of a row
    const int32_t* d_T;
    int T_host, T_max, H;
    EtHeader* hdr;
    bf16* x_out;          // [T, H] or null
    bf16* x_hat;          // [T, H]
    // backward
    const bf16* d_x_out;  // [T, H] or null
    const bf16* d_x_hat;  // [T, H]
    bf16* dx;
    bf16* dy;             // [T, H] or null
    int want;             // parameter gradients: bit 0 gamma, 1 beta
    int bufs;             // staged rows a group: 2 (the next one is copied ahead) or 1
    float* part;          // [CTAs][2][H]
};

// One or three sums over the row's threads, the same bits in every one of them, with the
// slots of row_sum.  The warps' sums are added in their order: eight at most are read by
// every thread (zeros behind the row's last warp), more are added by a warp's lanes.
template <int N>
struct RowSums {
    float red[2][N][64];  // eight warps of up to eight rows, or a row's 32
    __device__ __forceinline__ void clear() {  // by the whole CTA, a barrier behind it
        for (int i = threadIdx.x; i < 2 * N * 64; i += blockDim.x) (&red[0][0][0])[i] = 0.0f;
    }
    template <int MODE, int MAXT>
    __device__ __forceinline__ void sum(float (&v)[N], const RowGroup<MODE>& g, int& n) {
        static_assert(N == 1 || N == 3, "");
        const int lane = threadIdx.x & 31;
        auto in_warp = [&]() { return N == 1 ? warp_sum(v[0]) : warp_sum3(reinterpret_cast<const float (&)[3]>(v)); };
        auto spread = [&](float s) {
            if (N == 1) { v[0] = s; return; }
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, s, i == 0 ? 0 : i == 1 ? 16 : 8);
        };
        float s = in_warp();
        if (MODE == kRowsWarp) {
            spread(s);
            return;
        }
        const int slot = n++ & 1, warps = g.th() >> 5, warp = (threadIdx.x >> 5) - g.id() * warps;
        const int first = MAXT <= 256 ? g.id() * 8 : 0;
        if (N == 1 ? lane == 0 : (lane & 7) == 0 && lane < 24) red[slot][N == 1 ? 0 : lane == 0 ? 0 : lane == 16 ? 1 : 2][first + warp] = s;
        g.sync();
        if (MAXT <= 256) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float4 a = *reinterpret_cast<const float4*>(&red[slot][i][first]), b = *reinterpret_cast<const float4*>(&red[slot][i][first + 4]);
                const float2 t = __fadd2_rn(__fadd2_rn(make_float2(a.x, a.y), make_float2(a.z, a.w)),
                                            __fadd2_rn(make_float2(b.x, b.y), make_float2(b.z, b.w)));
                v[i] = t.x + t.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = lane < warps ? red[slot][i][lane] : 0.0f;
            s = in_warp();
            spread(s);
        }
    }
};

// s / H, exactly where that is a float (a row of equal values: no deviation is made up).
__device__ __forceinline__ float row_mean(float s, float H, float inv_H) {
    const float q = s * inv_H;
    return fmaf(fmaf(-q, H, s), inv_H, q);
}

// A parameter vector as floats in shared memory, each thread's own values where only it
// reads them (the groups of a CTA write the same ones); `none` where there is no vector.
template <bool VEC, int MODE>
__device__ __forceinline__ void stage_param(float4* to, const bf16* from, float none, const RowGroup<MODE>& g, int H) {
#pragma unroll
    for (int j = 0; j < norm_v(MODE); ++j) {
        const Vec8 v = from ? load8<VEC>(from, g, j, H) : Vec8{};
        float4 f[2] = {make_float4(v[0], v[1], v[2], v[3]), make_float4(v[4], v[5], v[6], v[7])};
        if (!from) f[0] = f[1] = make_float4(none, none, none, none);
        to[2 * j * g.th() + g.lane()] = f[0];
        to[(2 * j + 1) * g.th() + g.lane()] = f[1];
    }
}
// Its pairs i and i + 1 (i even) of vector j.
template <int MODE>
__device__ __forceinline__ float4 param4(const float4* from, const RowGroup<MODE>& g, int j, int i) {
    return from[(2 * j + (i >> 1)) * g.th() + g.lane()];
}

// The mask of this thread's columns.  VEC: drawn here.  Else the row's threads draw the
// row's mask into `bytes` first (8 columns a byte).
template <bool VEC, int MODE>
__device__ __forceinline__ void row_mask(Mask8 (&m)[norm_v(MODE)], const DropArgs& d, const DropKey& key,
                                         const RowGroup<MODE>& g, uint8_t* bytes, int t, int H) {
#pragma unroll
    for (int j = 0; j < norm_v(MODE); ++j) m[j] = keep_all();
    if (!d.thr) return;
    if (VEC) {
#pragma unroll
        for (int j = 0; j < norm_v(MODE); ++j) m[j] = keep_mask8(key, d.thr, g.template col<true>(j, 0) >> 3, t);
    } else {
        g.sync();  // the last row's mask has been read
        for (int q = g.lane(); q < (H + 7) >> 3; q += g.th()) bytes[q] = dropped_bits(keep_mask8(key, d.thr, q, t));
        g.sync();
#pragma unroll
        for (int j = 0; j < norm_v(MODE); ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = g.template col<false>(j, i);
                if (c < H && (bytes[c >> 3] >> (c & 7) & 1)) m[j].u[i >> 1] &= i & 1 ? 0xffffu : 0xffff0000u;
            }
    }
}

__host__ __device__ constexpr int ln_mask_bytes(int H) { return (H + 7) / 8; }
// Bytes of a staged row; with VEC whole vectors of all its threads (threads V).
__host__ __device__ constexpr int ln_row_bytes(int H, bool vec, int vectors) { return vec ? vectors * 16 : norm_row_bytes(H, false); }

// The mean first, then the squares of the distances from it: one pass over memory,
// two sums over the row's threads, the next row on its way meanwhile.  gamma and beta
// are floats in shared memory (unpacked anew for each row they were two of 33 instructions
// an element).  T = H = 4096: 20.5 us, 6.5 TB/s without dropout, bound by HBM; 23.3 us, 5.8
// TB/s with it, by issue slots too (30 instructions an element, 62 % of the slots).
// Without VEC by its 2-byte accesses: 4096 x 1001 11.8 us, 2.8 TB/s; with dropout 14.9.
template <bool VEC, int MODE, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT > 256 ? 1 : VEC ? 4 : 3) ln_fwd_kernel(const LnArgs p) {
    constexpr int V = norm_v(MODE);
    __shared__ RowSums<1> sums;
    extern __shared__ __align__(16) uint8_t dyn[];  // gamma, beta; without VEC [groups][H / 8] mask bytes
    int n_sums = 0;
    const RowGroup<MODE> g(p.row_threads);
    sums.clear();
    grid_begin();
    bool ok;
    const int T = row_count(p.d_T, p.T_host, p.T_max, p.hdr, &ok);
    const int H = p.H;
    float4* const gam = reinterpret_cast<float4*>(dyn);
    float4* const bet = gam + 2 * V * g.th();
    uint8_t* bytes = reinterpret_cast<uint8_t*>(bet + 2 * V * g.th()) + g.id() * ln_mask_bytes(H);
    Vec8 xv[V], yv[V];
    auto fetch = [&](int t) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            xv[j] = t < T ? load8<VEC>(p.x + static_cast<size_t>(t) * H, g, j, H) : Vec8{};
            yv[j] = p.y && t < T ? load8<VEC>(p.y + static_cast<size_t>(t) * H, g, j, H) : Vec8{};
        }
    };
    int t = blockIdx.x * g.groups() + g.id();
    fetch(t);
    const DropKey key(p.drop);
    stage_param<VEC>(gam, p.gamma, 1.0f, g, H);
    stage_param<VEC>(bet, p.beta, 0.0f, g, H);
    __syncthreads();  // (for the cleared sums)
    for (; t < T; t += gridDim.x * g.groups()) {
        const size_t off = static_cast<size_t>(t) * H;
        float2 z[V][4], s2 = both(0.0f);
        if (p.y) {
            Mask8 m[V];
            row_mask<VEC>(m, p.drop, key, g, bytes, t, H);
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) z[j][i] = __ffma2_rn(unpack2(yv[j].u[i] & m[j].u[i]), both(p.drop.mul), unpack2(xv[j].u[i]));
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) z[j][i] = unpack2(xv[j].u[i]);
        }
        fetch(t + gridDim.x * g.groups());
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (p.x_out) store8<VEC>(p.x_out + off, g, j, H, &z[j][0].x);
#pragma unroll
            for (int i = 0; i < 4; ++i) s2 = __fadd2_rn(s2, z[j][i]);  // 0 past H
        }
        float s[1] = {s2.x + s2.y};
        sums.template sum<MODE, MAXT>(s, g, n_sums);
        const float mean = row_mean(s[0], static_cast<float>(H), p.inv_H);
        s2 = both(0.0f);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float mj = VEC && g.template col<VEC>(j, 0) >= H ? 0.0f : mean;  // 0 behind H, as z
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                z[j][i] = __fadd2_rn(z[j][i], both(-mj));
                if (!VEC) {
                    if (g.template col<VEC>(j, 2 * i) >= H) z[j][i].x = 0.0f;
                    if (g.template col<VEC>(j, 2 * i + 1) >= H) z[j][i].y = 0.0f;
                }
                s2 = __ffma2_rn(z[j][i], z[j][i], s2);
            }
        }
        s[0] = s2.x + s2.y;
        sums.template sum<MODE, MAXT>(s, g, n_sums);
        const float r = rsqrtf(s[0] * p.inv_H + p.eps);
#pragma unroll
        for (int j = 0; j < V; ++j) {
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const float4 gv = param4(gam, g, j, i), bv = param4(bet, g, j, i);
                z[j][i] = __ffma2_rn(__fmul2_rn(z[j][i], both(r)), make_float2(gv.x, gv.y), make_float2(bv.x, bv.y));
                z[j][i + 1] = __ffma2_rn(__fmul2_rn(z[j][i + 1], both(r)), make_float2(gv.z, gv.w), make_float2(bv.z, bv.w));
            }
            store8<VEC>(p.x_hat + off, g, j, H, &z[j][0].x);
        }
    }
}

// The gradient.  With d = z - mean z, r = 1 / sqrt(var + eps), a = d_x_hat gamma:
//   D = d_x_out + r (a - mean a - d r^2 mean(a d)),   dx = D,  dy = dropout(D),
//   d_gamma = sum_t d_x_hat d r,  d_beta = sum_t d_x_hat.
// z, its statistics and the mask are made again from x and y, which costs no more
// bytes than reading z would.  Two sums over a row's threads: z; d^2, a and a d.
//
// Bound by HBM if a row's latencies are hidden: the input rows of a group's next
// row are copied to shared memory while the current one is worked on, each thread
// reading back only what it copied itself, so that the copies need no barrier.
// Without VEC a row is copied by the 16-byte pieces that hold it (the first of a
// tensor element by element, the last cut to its end) and read back by element,
// with a barrier on either side.  Rows of H > 8192 do not fit twice and are copied
// one at a time, and their 1024 threads have 64 registers, of which they spill 354 bytes (428
// without VEC): T = 1000, H = 16384 84 us, a third of the copy rate.  T = H = 4096 with
// dropout: 33 us, 6.1 TB/s, and 39 us with the parameter gradients: 304 rows of partial sums
// are written and read again, and a second kernel starts.
// (512-thread CTAs of two rows, half the partial sums, took 44.)  The parameter gradients
// are added up in registers, for 256 rows
// at most, then in this CTA's row of partial sums, then by ln_sum_kernel: a fixed
// order, no atomics.
template <bool VEC, int MODE, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT > 512 ? 1 : 512 / MAXT) ln_bwd_kernel(const LnArgs p) {
    constexpr int V = norm_v(MODE);
    __shared__ RowSums<1> sums1;
    __shared__ RowSums<3> sums3;
    // [groups][bufs][A] rows; gamma as floats; [groups][2][H]
    // floats where several groups' sums meet; without VEC [groups][H / 8] mask bytes
    extern __shared__ __align__(16) uint8_t dyn[];
    int n1 = 0, n3 = 0;
    const RowGroup<MODE> grp(p.row_threads);
    sums1.clear();
    sums3.clear();
    grid_begin();
    bool ok;
    const int T = row_count(p.d_T, p.T_host, p.T_max, p.hdr, &ok);
    if (!ok) return;
    const int H = p.H, H2 = H * 2, groups = grp.groups(), bufs = p.bufs;
    const int row_b = ln_row_bytes(H, VEC, grp.th() * V), par_b = grp.th() * V * 32;
    const int ny = p.y ? 1 : 0, nd = p.d_x_out ? 1 : 0, A = 2 + ny + nd;  // staged: x, d_x_hat, y, d_x_out
    const int c0 = grp.template col<true>(0, 0), c1 = grp.template col<true>(1, 0);
    const bool in0 = c0 < H, in1 = V > 1 && c1 < H;  // VEC only
    uint8_t* mine = dyn + static_cast<size_t>(grp.id()) * bufs * A * row_b;
    uint8_t* par = dyn + static_cast<size_t>(groups) * bufs * A * row_b;
    float* merge = reinterpret_cast<float*>(par + par_b);
    uint8_t* bytes = par + par_b + (MODE != kRowsOne && groups > 1 ? groups * 2 * H * 4 : 0) + grp.id() * ln_mask_bytes(H);
    float4* const gam = reinterpret_cast<float4*>(par);
    const DropKey key(p.drop);

    const bf16* const src[4] = {p.x, p.d_x_hat, ny ? p.y : p.d_x_out, p.d_x_out};
    auto stage = [&](int t, int buf) {
        if (t < T) {
            const size_t off = static_cast<size_t>(t) * H;
            const uint32_t dst = smem_addr(mine) + buf * A * row_b;
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                if (a >= A) break;
                if (VEC) {
                    if (in0) cp_async16(dst + a * row_b + c0 * 2, src[a] + off + c0);
                    if (in1) cp_async16(dst + a * row_b + c1 * 2, src[a] + off + c1);
                } else {
                    const uint8_t* base = reinterpret_cast<const uint8_t*>(src[a]);
                    const uint8_t* row = base + off * 2;
                    const uint8_t* first = row - (reinterpret_cast<uintptr_t>(row) & 15);
                    const int pieces = static_cast<int>((row + H2 - first + 15) >> 4);
                    const uint8_t* end = base + static_cast<size_t>(p.T_max) * H2;
                    for (int k = grp.lane(); k < pieces; k += grp.th()) {
                        const uint8_t* c = first + k * 16;
                        if (c < base) {
                            for (int i = 0; i < 8; ++i)
                                if (c + 2 * i >= base && c + 2 * i < end)
                                    *reinterpret_cast<uint16_t*>(mine + (buf * A + a) * row_b + k * 16 + 2 * i) =
                                        *reinterpret_cast<const uint16_t*>(c + 2 * i);
                        } else {
                            cp_async16_part(dst + a * row_b + k * 16, c, end - c < 16 ? static_cast<int>(end - c) : 16);
                        }
                    }
                }
            }
        }
        cp_async_commit();
    };
    int buf = 0;
    const int step = gridDim.x * groups, t0 = blockIdx.x * groups;
    if (VEC)  // what a thread has behind H stays zero
        for (int a = 0; a < bufs * A; ++a) {
            if (!in0) *reinterpret_cast<uint4*>(mine + a * row_b + c0 * 2) = make_uint4(0, 0, 0, 0);
            if (V > 1 && !in1) *reinterpret_cast<uint4*>(mine + a * row_b + c1 * 2) = make_uint4(0, 0, 0, 0);
        }
    if (bufs == 2) stage(t0 + grp.id(), 0);
    stage_param<VEC>(gam, p.gamma, 1.0f, grp, H);
    __syncthreads();  // (for the cleared sums)
    float2 a_g[V][4], a_b[V][4];
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) a_g[j][i] = a_b[j][i] = both(0.0f);

    // This CTA's sums so far to its row of partial sums; `more`: added to what is there.
    // Reached by the whole CTA.
    auto put_away = [&](bool more) {
        float* part = p.part + static_cast<size_t>(blockIdx.x) * 2 * H;
        const bool meet = MODE != kRowsOne && groups > 1;
        float* to = meet ? merge + static_cast<size_t>(grp.id()) * 2 * H : part;
#pragma unroll
        for (int arr = 0; arr < 2; ++arr)
            if (p.want >> arr & 1)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if (VEC) {
                        float4* o = reinterpret_cast<float4*>(to + arr * H + (j ? c1 : c0));
                        if (j ? in1 : in0)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const float2 v = arr ? a_b[j][2 * i] : a_g[j][2 * i], u = arr ? a_b[j][2 * i + 1] : a_g[j][2 * i + 1];
                                float4 q = make_float4(v.x, v.y, u.x, u.y);
                                if (!meet && more) {
                                    const float4 was = o[i];
                                    q = make_float4(q.x + was.x, q.y + was.y, q.z + was.z, q.w + was.w);
                                }
                                o[i] = q;
                            }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 v = arr ? a_b[j][i >> 1] : a_g[j][i >> 1];
                            const int c = grp.template col<VEC>(j, i);
                            if (c < H) to[arr * H + c] = (i & 1 ? v.y : v.x) + (!meet && more ? to[arr * H + c] : 0.0f);
                        }
                    }
                }
        if (meet) {
            __syncthreads();
            for (int o = threadIdx.x; o < 2 * H; o += blockDim.x)
                if (p.want >> (o >= H ? 1 : 0) & 1) {
                    float s = 0.0f;
                    for (int k = 0; k < groups; ++k) s += merge[static_cast<size_t>(k) * 2 * H + o];
                    part[o] = s + (more ? part[o] : 0.0f);
                }
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) a_g[j][i] = a_b[j][i] = both(0.0f);
    };

    bool more = false;
    int chain = 0;
    for (int r0 = t0; r0 < T; r0 += step) {  // the same rounds for every group of the CTA
        const int t = r0 + grp.id();
        if (bufs == 2) {
            stage(t + step, buf ^ 1);  // this thread has read that buffer's last row
            cp_async_wait<1>();
        } else {
            stage(t, 0);
            cp_async_wait<0>();
        }
        if (!VEC) grp.sync();  // the other threads' pieces
        if (t < T) {
            const uint8_t* rows = mine + buf * A * row_b;
            const size_t off = static_cast<size_t>(t) * H;
            auto get = [&](int a, int j) -> uint4 {  // vector j of staged row a; zeros past H
                if (VEC) return *reinterpret_cast<const uint4*>(rows + a * row_b + (j ? c1 : c0) * 2);
                const uint16_t* r = reinterpret_cast<const uint16_t*>(rows + a * row_b + (reinterpret_cast<uintptr_t>(src[a] + off) & 15));
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int lo = grp.template col<VEC>(j, 2 * i), hi = grp.template col<VEC>(j, 2 * i + 1);
                    w[i] = (lo < H ? r[lo] : 0u) | (hi < H ? static_cast<uint32_t>(r[hi]) << 16 : 0u);
                }
                return make_uint4(w[0], w[1], w[2], w[3]);
            };
            auto put_row = [&](bf16* to, int j, const uint32_t (&w)[4]) {
                if (VEC) {
                    if (j ? in1 : in0) *reinterpret_cast<uint4*>(to + off + (j ? c1 : c0)) = make_uint4(w[0], w[1], w[2], w[3]);
                } else {
                    uint16_t* o = reinterpret_cast<uint16_t*>(to + off);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int c = grp.template col<VEC>(j, i);
                        if (c < H) o[c] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
                    }
                }
            };
            auto word = [](const uint4& v, int i) -> uint32_t { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; };
            Mask8 m[V];
            float2 z[V][4], s2 = both(0.0f);
            if (ny) row_mask<VEC>(m, p.drop, key, grp, bytes, t, H);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const uint4 x = get(0, j);
#pragma unroll
                for (int i = 0; i < 4; ++i) z[j][i] = unpack2(word(x, i));
            }
            if (ny) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const uint4 y = get(2, j);
#pragma unroll
                    for (int i = 0; i < 4; ++i) z[j][i] = __ffma2_rn(unpack2(word(y, i) & m[j].u[i]), both(p.drop.mul), z[j][i]);
                }
            }
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) s2 = __fadd2_rn(s2, z[j][i]);
            float s1[1] = {s2.x + s2.y};
            sums1.template sum<MODE, MAXT>(s1, grp, n1);
            const float mean = row_mean(s1[0], static_cast<float>(H), p.inv_H);
            float2 dd = both(0.0f), sa = both(0.0f), sad = both(0.0f);
            float2 h[V][4];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const uint4 dh = get(1, j);
                const float mj = VEC && !(j ? in1 : in0) ? 0.0f : mean;  // 0 behind H, as z
                float4 gm{};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i % 2 == 0) gm = param4(gam, grp, j, i);
                    h[j][i] = unpack2(word(dh, i));
                    z[j][i] = __fadd2_rn(z[j][i], both(-mj));
                    if (!VEC) {
                        if (grp.template col<VEC>(j, 2 * i) >= H) z[j][i].x = 0.0f;
                        if (grp.template col<VEC>(j, 2 * i + 1) >= H) z[j][i].y = 0.0f;
                    }
                    const float2 a = __fmul2_rn(h[j][i], i % 2 ? make_float2(gm.z, gm.w) : make_float2(gm.x, gm.y));
                    dd = __ffma2_rn(z[j][i], z[j][i], dd);
                    sa = __fadd2_rn(sa, a);
                    sad = __ffma2_rn(a, z[j][i], sad);
                }
            }
            float s3[3] = {dd.x + dd.y, sa.x + sa.y, sad.x + sad.y};
            sums3.template sum<MODE, MAXT>(s3, grp, n3);
            const float r = rsqrtf(s3[0] * p.inv_H + p.eps);
            const float ra = -r * (s3[1] * p.inv_H), k = -r * r * (s3[2] * p.inv_H);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const uint4 dz = nd ? get(2 + ny, j) : make_uint4(0, 0, 0, 0);
                uint32_t odx[4];
                float2 D[4];
                float4 gm{};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i % 2 == 0) gm = param4(gam, grp, j, i);
                    const float2 n = __fmul2_rn(z[j][i], both(r));
                    D[i] = __fadd2_rn(unpack2(word(dz, i)), both(ra));
                    D[i] = __ffma2_rn(__fmul2_rn(h[j][i], i % 2 ? make_float2(gm.z, gm.w) : make_float2(gm.x, gm.y)), both(r), D[i]);
                    D[i] = __ffma2_rn(n, both(k), D[i]);
                    a_g[j][i] = __ffma2_rn(h[j][i], n, a_g[j][i]);
                    a_b[j][i] = __fadd2_rn(a_b[j][i], h[j][i]);
                    odx[i] = pack_bf16(D[i].x, D[i].y);
                }
                put_row(p.dx, j, odx);
                if (p.dy) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        D[i] = __fmul2_rn(D[i], both(p.drop.mul));
                        odx[i] = pack_bf16(D[i].x, D[i].y) & m[j].u[i];
                    }
                    put_row(p.dy, j, odx);
                }
            }
        }
        if (!VEC) grp.sync();  // this buffer and the mask's bytes are written again
        if (bufs == 2) buf ^= 1;
        if (p.want && (++chain == kLnChain || r0 + step >= T)) {
            put_away(more);
            more = true;
            chain = 0;
        }
    }
    cp_async_wait<0>();
    if (p.want && !more) {  // no rows: zeros
        float* part = p.part + static_cast<size_t>(blockIdx.x) * 2 * H;
        for (int o = threadIdx.x; o < 2 * H; o += blockDim.x) part[o] = 0.0f;
    }
}

struct LnSumArgs {
    const float* part;
    float* out[2];  // the wanted ones of d_gamma, d_beta
    int arr[2];     // which
    int H, parts;
    const int32_t* d_T;
    int T_max;
};

// Column sums of the partial rows: 32 columns x kSumGroups row groups a CTA, a thread's loads
// all on their way at once.  Bound by latency: with its launch 3 us for one row, 6 for 304 of
// H = 4096.  (8 groups 6.4 of a call of one row and 11.6 of one of 304, 16 6.0 and 10.0, 32
// 6.7 and 10.5.)
constexpr int kSumGroups = 16;
__global__ void __launch_bounds__(kSumGroups * 32) ln_sum_kernel(const LnSumArgs p) {
    __shared__ float red[kSumGroups][32];
    grid_begin();
    if (p.d_T && (*p.d_T < 0 || *p.d_T > p.T_max)) return;
    float* out = p.out[blockIdx.y];
    const int arr = p.arr[blockIdx.y];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    constexpr int kLoads = (kLnParts + kSumGroups - 1) / kSumGroups;
    float v[kLoads], s = 0.0f, u = 0.0f;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int g = grp + kSumGroups * i;
        v[i] = g < p.parts && c < p.H ? __ldcg(p.part + (static_cast<size_t>(g) * 2 + arr) * p.H + c) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) (i & 1 ? u : s) += v[i];
    red[grp][lane] = s + u;
    __syncthreads();
    if (grp == 0 && c < p.H) {
        s = u = 0.0f;
#pragma unroll
        for (int i = 0; i < kSumGroups; ++i) (i & 1 ? u : s) += red[i][lane];
        out[c] = s + u;
    }
}

// ---------------------------------------------------------------- host

constexpr int kDropHMax = 1 << 18;

size_t ln_ws_bytes(int T_max, int H) {
    const size_t parts = T_max < kLnParts ? T_max : kLnParts;
    return (kHeaderBytes + parts * 2 * H * sizeof(float) + 255) / 256 * 256;
}

bool ln_shape_ok(int T_max, int H, int H_max, std::string* why) {
    if (T_max < 1 || T_max > (1 << 24)) { *why = "T_max must be in [1, 2^24]"; return false; }
    if (H < 1 || H > H_max) { *why = "H must be in [1, " + std::to_string(H_max) + "]"; return false; }
    return true;
}

// The mask's threshold and factor; false where p is no probability below 1.
bool drop_args(float p, uint64_t seed, uint64_t offset, const uint64_t* d_rng, DropArgs* d) {
    if (!(p >= 0.0f) || !(p <= 65535.0f / 65536.0f)) return false;
    const double thr = std::nearbyint(static_cast<double>(p) * 65536.0);
    d->seed = seed;
    d->offset = offset;
    d->d_rng = d_rng;
    d->thr = static_cast<uint32_t>(thr);
    d->mul = static_cast<float>(65536.0 / (65536.0 - thr));
    return true;
}

const char* const kDropRange = "p must be in [0, 65535/65536]";

int ln_check(const void* x, const void* y, const void* gamma, const void* beta, float eps, float p, const uint64_t* d_rng,
             int T, const int32_t* d_T, int T_max, int H) {
    std::string why;
    if (!ln_shape_ok(T_max, H, kNormHMax, &why)) return api_fail(ET_ERR_UNSUPPORTED, why);
    if (!x) return api_fail(ET_ERR_INVALID, "x must be non-NULL");
    if (!y && p != 0.0f) return api_fail(ET_ERR_INVALID, "dropout (p > 0) needs y");
    if (!(eps > 0.0f) || !std::isfinite(eps)) return api_fail(ET_ERR_INVALID, "eps must be > 0 and finite");
    const void* need2[] = {x, y, gamma, beta};
    for (const void* q : need2)
        if (!api_aligned(q, 2)) return api_fail(ET_ERR_INVALID, "tensors must be aligned to their element size");
    if (!api_aligned(d_T, 4) || !api_aligned(d_rng, 8))
        return api_fail(ET_ERR_INVALID, "tensors must be aligned to their element size");
    if (!d_T && (T < 0 || T > T_max)) return api_fail(ET_ERR_INVALID, "T must be in [0, T_max]");
    return ET_OK;
}

struct LnLaunch {
    int dev, sms, rows, parts_max;
    int* parts;
    void* stream;
};

template <bool VEC, int MODE, int MAXT>
cudaError_t launch_ln_fwd_rows(LnArgs a, const LnLaunch& l) {
    static SmemOptIn opt;
    auto kernel = ln_fwd_kernel<VEC, MODE, MAXT>;
    const cudaError_t e = api_smem_opt_in(opt, l.dev, kernel, kSmemLimit - 4096);
    if (e != cudaSuccess) return e;
    const int groups = norm_groups(a.row_threads, l.rows), th = a.row_threads * groups;
    const int need = (l.rows + groups - 1) / groups, most = l.sms * (1024 / th);
    const int smem = a.row_threads * norm_v(MODE) * 64 + (!VEC && a.drop.thr ? groups * ln_mask_bytes(a.H) : 0);
    return api_launch(kernel, need < most ? need : most, th, smem, l.stream, a);
}

template <bool VEC>
cudaError_t launch_ln_fwd(LnArgs a, const LnLaunch& l) {
    a.row_threads = norm_threads(a.H);
    const RowMode mode = norm_mode(a.H, a.row_threads);
    if (mode == kRowsWarp) return launch_ln_fwd_rows<VEC, kRowsWarp, 256>(a, l);
    if (mode == kRowsGroup) return launch_ln_fwd_rows<VEC, kRowsGroup, 256>(a, l);
    if (a.row_threads <= 256) return launch_ln_fwd_rows<VEC, kRowsOne, 256>(a, l);
    return launch_ln_fwd_rows<VEC, kRowsOne, 1024>(a, l);
}

template <bool VEC, int MODE, int MAXT>
cudaError_t launch_ln_bwd_rows(LnArgs a, const LnLaunch& l) {
    static SmemOptIn opt;
    auto kernel = ln_bwd_kernel<VEC, MODE, MAXT>;
    const cudaError_t e = api_smem_opt_in(opt, l.dev, kernel, kSmemLimit - 4096);
    if (e != cudaSuccess) return e;
    const int groups = norm_groups(a.row_threads, l.rows), th = a.row_threads * groups;
    const int need = (l.rows + groups - 1) / groups, most = th <= kNormCtaThreads ? 2 * l.sms : l.sms;
    int n = need < l.parts_max ? need : l.parts_max;
    *l.parts = n = n < most ? n : most;
    const int A = 2 + (a.y ? 1 : 0) + (a.d_x_out ? 1 : 0);
    a.bufs = a.H <= 8192 ? 2 : 1;
    const int smem = groups * a.bufs * A * ln_row_bytes(a.H, VEC, a.row_threads * norm_v(MODE)) + a.row_threads * norm_v(MODE) * 32 +
                     (MODE != kRowsOne && groups > 1 ? groups * 2 * a.H * 4 : 0) +
                     (!VEC && a.drop.thr ? groups * ln_mask_bytes(a.H) : 0);
    return api_launch(kernel, n, th, smem, l.stream, a);
}

template <bool VEC>
cudaError_t launch_ln_bwd(LnArgs a, const LnLaunch& l) {
    a.row_threads = norm_threads(a.H);
    const RowMode mode = norm_mode(a.H, a.row_threads);
    if (mode == kRowsWarp) return launch_ln_bwd_rows<VEC, kRowsWarp, 256>(a, l);
    if (mode == kRowsGroup) return launch_ln_bwd_rows<VEC, kRowsGroup, 256>(a, l);
    if (a.row_threads <= 256) return launch_ln_bwd_rows<VEC, kRowsOne, 256>(a, l);
    if (a.row_threads <= 512) return launch_ln_bwd_rows<VEC, kRowsOne, 512>(a, l);
    return launch_ln_bwd_rows<VEC, kRowsOne, 1024>(a, l);
}

}  // namespace
}  // namespace et

using namespace et;

extern "C" {

size_t et_dropout_workspace_bytes(int T_max, int H) {
    return T_max < 1 || T_max > (1 << 24) || H < 1 || H > kDropHMax ? 0 : kHeaderBytes;
}

int et_dropout(const void* x, const void* y, void* out, float p, uint64_t seed, uint64_t offset,
               const uint64_t* d_rng, int T, const int32_t* d_T, int T_max, int H, void* workspace,
               size_t workspace_bytes, void* stream) {
    return api_entry([&]() -> int {
        std::string why;
        if (!ln_shape_ok(T_max, H, kDropHMax, &why)) return api_fail(ET_ERR_UNSUPPORTED, why);
        if (!y || !out) return api_fail(ET_ERR_INVALID, "y and out must be non-NULL");
        const void* need2[] = {x, y, out};
        for (const void* q : need2)
            if (!api_aligned(q, 2)) return api_fail(ET_ERR_INVALID, "tensors must be aligned to their element size");
        if (!api_aligned(d_T, 4) || !api_aligned(d_rng, 8))
            return api_fail(ET_ERR_INVALID, "tensors must be aligned to their element size");
        if (!d_T && (T < 0 || T > T_max)) return api_fail(ET_ERR_INVALID, "T must be in [0, T_max]");
        DropoutArgs a{};
        if (!drop_args(p, seed, offset, d_rng, &a.drop)) return api_fail(ET_ERR_INVALID, kDropRange);
        int rc = api_check_ws(workspace, workspace_bytes, kHeaderBytes);
        if (rc) return rc;
        if (!d_T && T == 0) return ET_OK;
        int dev = 0, sms = 0;
        if ((rc = api_device(&dev, &sms))) return rc;
        a.x = static_cast<const bf16*>(x);
        a.y = static_cast<const bf16*>(y);
        a.out = static_cast<bf16*>(out);
        a.d_T = d_T;
        a.T_host = T;
        a.T_max = T_max;
        a.H = H;
        a.hdr = static_cast<EtHeader*>(workspace);
        const int rows = d_T ? T_max : T;
        cudaError_t e;
        if (norm_vec(H, {x, y, out})) {
            const int H8 = H / 8;
            // 1024 vectors a CTA, four a thread; fewer where that leaves SMs without work
            a.rows = H8 >= 1024 ? 1 : 1024 / H8;
            while (a.rows > 1 && (rows + a.rows - 1) / a.rows < 2 * sms) a.rows = (a.rows + 1) / 2;
            // exact for i < 2^18 / 8 + 1024: i (magic H8 - 2^32) < 2^32 as i H8 < 2^32
            a.magic = static_cast<uint32_t>(((1ull << 32) + H8 - 1) / H8);
            e = api_launch(dropout_vec_kernel, (rows + a.rows - 1) / a.rows, kDropThreads, 0, stream, a);
        } else {
            const long long grid = static_cast<long long>(rows) * ((H + kDropCols - 1) / kDropCols);
            if (grid > 0x7fffffffll) return api_fail(ET_ERR_UNSUPPORTED, "T_max * H is too large for an unaligned or odd H");
            e = api_launch(dropout_any_kernel, static_cast<int>(grid), kDropThreads, 0, stream, a);
        }
        if (e != cudaSuccess) return api_fail_cuda(e, "launch of the dropout kernel");
        return ET_OK;
    });
}

size_t et_layer_norm_workspace_bytes(int T_max, int H) {
    if (T_max < 1 || T_max > (1 << 24) || H < 1 || H > kNormHMax) return 0;
    return ln_ws_bytes(T_max, H);
}

int et_layer_norm(const void* x, const void* y, const void* gamma, const void* beta, float eps, float p,
                  uint64_t seed, uint64_t offset, const uint64_t* d_rng, void* x_out, void* x_hat, int T,
                  const int32_t* d_T, int T_max, int H, void* workspace, size_t workspace_bytes, void* stream) {
    return api_entry([&]() -> int {
        int rc = ln_check(x, y, gamma, beta, eps, p, d_rng, T, d_T, T_max, H);
        if (rc) return rc;
        if (!x_hat) return api_fail(ET_ERR_INVALID, "x_hat must be non-NULL");
        if (!api_aligned(x_out, 2) || !api_aligned(x_hat, 2))
            return api_fail(ET_ERR_INVALID, "tensors must be aligned to their element size");
        LnArgs a{};
        if (!drop_args(p, seed, offset, d_rng, &a.drop)) return api_fail(ET_ERR_INVALID, kDropRange);
        if ((rc = api_check_ws(workspace, workspace_bytes, kHeaderBytes))) return rc;
        if (!d_T && T == 0) return ET_OK;
        int dev = 0, sms = 0;
        if ((rc = api_device(&dev, &sms))) return rc;
        a.x = static_cast<const bf16*>(x);
        a.y = static_cast<const bf16*>(y);
        a.gamma = static_cast<const bf16*>(gamma);
        a.beta = static_cast<const bf16*>(beta);
        a.eps = eps;
        a.inv_H = 1.0f / static_cast<float>(H);
        a.d_T = d_T;
        a.T_host = T;
        a.T_max = T_max;
        a.H = H;
        a.hdr = static_cast<EtHeader*>(workspace);
        a.x_out = static_cast<bf16*>(x_out);
        a.x_hat = static_cast<bf16*>(x_hat);
        const int rows = d_T ? T_max : T;
        const LnLaunch l{dev, sms, rows, 0, nullptr, stream};
        const cudaError_t e = norm_vec(H, {x, y, gamma, beta, x_out, x_hat}) ? launch_ln_fwd<true>(a, l) : launch_ln_fwd<false>(a, l);
        if (e != cudaSuccess) return api_fail_cuda(e, "launch of the layer norm kernel");
        return ET_OK;
    });
}

int et_layer_norm_bwd(const void* x, const void* y, const void* gamma, float eps, float p, uint64_t seed,
                      uint64_t offset, const uint64_t* d_rng, const void* d_x_out, const void* d_x_hat, void* dx,
                      void* dy, float* d_gamma, float* d_beta, int T, const int32_t* d_T, int T_max, int H,
                      void* workspace, size_t workspace_bytes, void* stream) {
    return api_entry([&]() -> int {
        int rc = ln_check(x, y, gamma, nullptr, eps, p, d_rng, T, d_T, T_max, H);
        if (rc) return rc;
        if (!d_x_hat || !dx) return api_fail(ET_ERR_INVALID, "d_x_hat and dx must be non-NULL");
        if (dy && !y) return api_fail(ET_ERR_INVALID, "dy needs y");
        if (d_gamma && !gamma) return api_fail(ET_ERR_INVALID, "a parameter's gradient needs the parameter");
        const void* need2[] = {d_x_out, d_x_hat, dx, dy};
        for (const void* q : need2)
            if (!api_aligned(q, 2)) return api_fail(ET_ERR_INVALID, "tensors must be aligned to their element size");
        if (!api_aligned(d_gamma, 4) || !api_aligned(d_beta, 4))
            return api_fail(ET_ERR_INVALID, "tensors must be aligned to their element size");
        LnArgs a{};
        if (!drop_args(p, seed, offset, d_rng, &a.drop)) return api_fail(ET_ERR_INVALID, kDropRange);
        if ((rc = api_check_ws(workspace, workspace_bytes, ln_ws_bytes(T_max, H)))) return rc;
        int dev = 0, sms = 0;
        if ((rc = api_device(&dev, &sms))) return rc;
        a.x = static_cast<const bf16*>(x);
        a.y = static_cast<const bf16*>(y);
        a.gamma = static_cast<const bf16*>(gamma);
        a.eps = eps;
        a.inv_H = 1.0f / static_cast<float>(H);
        a.d_T = d_T;
        a.T_host = T;
        a.T_max = T_max;
        a.H = H;
        a.hdr = static_cast<EtHeader*>(workspace);
        a.d_x_out = static_cast<const bf16*>(d_x_out);
        a.d_x_hat = static_cast<const bf16*>(d_x_hat);
        a.dx = static_cast<bf16*>(dx);
        a.dy = static_cast<bf16*>(dy);
        a.want = (d_gamma ? 1 : 0) | (d_beta ? 2 : 0);
        a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kHeaderBytes);
        const int rows = d_T ? T_max : T;
        LnSumArgs s{a.part, {}, {}, H, 0, d_T, T_max};
        int n = 0;
        if (d_gamma) { s.out[n] = d_gamma; s.arr[n++] = 0; }
        if (d_beta) { s.out[n] = d_beta; s.arr[n++] = 1; }
        if (rows > 0) {
            const LnLaunch l{dev, sms, rows, T_max < kLnParts ? T_max : kLnParts, &s.parts, stream};
            const cudaError_t e = norm_vec(H, {x, y, gamma, d_x_out, d_x_hat, dx, dy}) ? launch_ln_bwd<true>(a, l)
                                                                                      : launch_ln_bwd<false>(a, l);
            if (e != cudaSuccess) return api_fail_cuda(e, "launch of the layer norm's backward kernel");
        }
        if (n) {
            const cudaError_t e = api_launch(ln_sum_kernel, dim3((H + 31) / 32, n), kSumGroups * 32, 0, stream, s);
            if (e != cudaSuccess) return api_fail_cuda(e, "launch of the layer norm's parameter sums");
        }
        return ET_OK;
    });
}

}  // extern "C"
