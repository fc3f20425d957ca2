// router_ops.cu -- the router's selection over given logits, with the balance
// and z losses of a training step, and the gradient of all of them.
#include <cmath>

#include "../../include/etmoe.h"
#include "et_api.h"
#include "ops_device.cuh"

namespace et {
namespace {

constexpr int kRouterWarpsMax = 32;
constexpr int kRouterEMax = 256;
constexpr int kRouterParts = 152;  // most CTAs of the forward kernel = rows of partial sums

struct RouterArgs {
    const float* logits;     // [T, E]
    const uint8_t* mask;     // [T] or null
    int32_t* idx;            // [T, k]
    float* w;                // [T, k]
    int32_t* counts;         // [E]
    int32_t* n_routed;       // [1]
    float* mean_prob;        // [E]
    float* losses;           // [2]
    const int32_t* d_T;
    int T_host, T_max, E, k;
    EtHeader* hdr;
    float2* part;            // [kRouterParts, E]: a CTA's sum of probabilities; its count, as an integer
    float* part_z;           // [kRouterParts]
    int32_t* part_n;         // [kRouterParts]
};

// Order-preserving key of a logit.  Adding +0 makes -0.0 tie with +0.0 and gives
// every NaN the one positive NaN, which ranks above all (it then shows in the
// weights and losses).  Every key is > 0.
__device__ __forceinline__ uint32_t logit_key(float v) {
    const int b = __float_as_int(__fadd_rn(v, 0.0f));
    return static_cast<uint32_t>(b ^ ((b >> 31) | static_cast<int>(0x80000000u)));
}

// The logit of a key (+0.0 for both zeros, a NaN for any NaN).
__device__ __forceinline__ float key_logit(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}

// The selection on whole keys, two reductions a round (the largest key, the lowest
// expert that has it): lane j < k gets the j-th.
template <int EPL>
__device__ __forceinline__ void select_whole(const float (&v)[EPL], int E, int k, int lane, uint32_t& mykey, uint32_t& myE) {
    uint32_t key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = lane + 32 * i < E ? logit_key(v[i]) : 0u;
#pragma unroll 1
    for (int j = 0; j < k; ++j) {
        uint32_t bk = key[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) bk = max(bk, key[i]);
        const uint32_t kmax = __reduce_max_sync(0xffffffffu, bk);
        uint32_t low = 0xffffffffu;  // this lane's lowest expert that holds it
#pragma unroll
        for (int i = EPL - 1; i >= 0; --i)
            if (key[i] == kmax) low = static_cast<uint32_t>(lane + 32 * i);
        const uint32_t e = __reduce_min_sync(0xffffffffu, low);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (static_cast<uint32_t>(lane + 32 * i) == e) key[i] = 0u;
        if (lane == j) { mykey = kmax; myE = e; }
    }
}

// (key, expert), out of line: it is seldom needed.
template <int EPL>
struct RowLogits { float v[EPL]; };
template <int EPL>
__device__ __noinline__ uint2 select_again(RowLogits<EPL> row, int E, int k, int lane) {
    uint32_t key = 0, e = 0;
    select_whole<EPL>(row.v, E, k, lane, key, e);
    return make_uint2(key, e);
}

// The same where a lane has four experts or eight.  Keys are cut above kLow, with the
// expert below, lower experts larger: one reduction a round finds both.  A lane's keys
// are sorted, so that a round looks at the heads alone.  Round k + 1 tells whether the
// cut decided who is chosen; if it may have, the row is selected again on whole keys.
// T = 65536, E = 128, k = 8 37.0 -> 32.5 us, T = 16384, E = 256 25.6 -> 20.7; with one
// or two experts a lane whole keys are faster (T = 16384, E = 8, k = 2 9.1 us and 10.4).
template <int EPL>
__device__ __forceinline__ void select_cut(const float (&v)[EPL], const float* logits, int E, int k, int lane,
                                           uint32_t& mykey, uint32_t& myE) {
    constexpr uint32_t kLow = 32 * EPL - 1, kNegInfKey = 0x007fffffu;
    uint32_t pk[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const uint32_t e = lane + 32 * i;
        pk[i] = e < static_cast<uint32_t>(E) ? (logit_key(v[i]) & ~kLow) | (kLow - e) : 0u;
    }
#pragma unroll
    for (int m = EPL - 1; m > 0; --m)
#pragma unroll
        for (int i = 0; i < m; ++i) {
            const uint32_t hi = max(pk[i], pk[i + 1]);
            pk[i + 1] = min(pk[i], pk[i + 1]);
            pk[i] = hi;
        }
    uint32_t mine = 0;  // lane j: the j-th, 0 when there is none
#pragma unroll 1
    for (int j = 0; j <= k; ++j) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, pk[0]);
        const bool win = pk[0] == top;
#pragma unroll
        for (int i = 0; i < EPL; ++i) pk[i] = win ? (i + 1 < EPL ? pk[(i + 1) % EPL] : 0u) : pk[i];
        if (lane == j) mine = top;
    }
    myE = kLow - (mine & kLow);
    mykey = 0;
    if (mine) mykey = logit_key(logits[myE]);
    // Experts with one cut key come in the order of their number: right unless a later
    // one's whole key is larger, or the cut key goes on behind the k-th (-inf may: none
    // of its kind is chosen).
    const uint32_t after = __shfl_down_sync(0xffffffffu, mykey, 1);
    const uint32_t next = __shfl_down_sync(0xffffffffu, mine, 1);
    const bool same = ((mine ^ next) & ~kLow) == 0 && mykey != kNegInfKey;
    const bool doubt = lane < k && same && (mykey < after || lane == k - 1);
    if (__any_sync(0xffffffffu, doubt)) {
        RowLogits<EPL> row;
#pragma unroll
        for (int i = 0; i < EPL; ++i) row.v[i] = v[i];
        const uint2 r = select_again<EPL>(row, E, k, lane);
        mykey = r.x;
        myE = r.y;
    }
}

// One row a warp, expert e = lane + 32 i in register i; the next row's logits are
// loaded while the current one is worked on.  The k rounds of the selection also
// give the row's largest logit, so the softmax needs no max pass.  Sums over
// rows: per warp in registers (32 rows, then once more, so that long sums stay
// short), per CTA in shared memory, over CTAs by the last one to finish -- each
// in a fixed order, so that losses and mean probabilities are the same bits on
// every run.  All in fp32: fp64 runs at 1/64 of it here.  The gate weights, which a
// program uses as they are, take expf and a true quotient (T = 65536, E = 128 32.4 us ->
// 34.0; the fast ones moved a weight of e^-60 by 40 x 2^-24).  The probabilities and the
// losses, averaged over tokens, take the fast ones: exp within 2 + 1.2 |L - L0| ulp
// (rounding L - L0 moves it by half of |L - L0| ulp already), a quotient within 2 ulp,
// log(s) within 2^-21.4 for s <= 2 and 3 ulp above.  With expf, logf and true quotients
// there too the means and losses were as far from 64 bits as before (5 x 10^-8; the order
// of the sums), for 35.1 us, and with the gradient T = 65536, E = 16 36.2 in place of 31.6.
//
// T = 16384, E = 128, k = 8: 13.8 us for 9.4 MB, which HBM would bring in 1.4.  About
// 7 us are fixed -- the launch, the first loads, and the way through memory to the
// last CTA's sums -- and the rest is instructions: 27 rows a scheduler, 450 cycles
// each, the selection most of them.
template <int EPL>
__global__ void __launch_bounds__(kRouterWarpsMax * 32) router_topk_kernel(const RouterArgs p) {
    extern __shared__ __align__(16) float sm[];  // [warps][E], then the last CTA's sums
    __shared__ int hist[kRouterEMax];
    __shared__ float zsum[kRouterWarpsMax];
    __shared__ int nsum[kRouterWarpsMax];
    __shared__ int last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    const int E = p.E, k = p.k;
    grid_begin();
    bool ok;
    const int T = row_count(p.d_T, p.T_host, p.T_max, p.hdr, &ok);
    if (!ok) return;
    // rows to CTAs in turn, so that the last round is spread over all of them
    const int t0 = blockIdx.x + gridDim.x * warp, step = gridDim.x * nwarps;
    auto load = [&](int t, float (&v)[EPL], int& on) {
        const float* L = p.logits + static_cast<size_t>(t) * E;
        on = t < T && (!p.mask || p.mask[t] != 0);
#pragma unroll
        for (int i = 0; i < EPL; ++i) v[i] = t < T && lane + 32 * i < E ? L[lane + 32 * i] : -INFINITY;
    };
    float nv[EPL];
    int non;
    load(t0, nv, non);
    for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
    __syncthreads();

    float accp[EPL], bigp[EPL], accz = 0.0f, bigz = 0.0f;
    int accn = 0, rows32 = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) accp[i] = bigp[i] = 0.0f;

    for (int t = t0; t < T; t += step) {
        float v[EPL];
        const int masked_in = non;
#pragma unroll
        for (int i = 0; i < EPL; ++i) v[i] = nv[i];
        load(t + step, nv, non);
        uint32_t mykey = 0, myE = 0;
        if (EPL <= 2) select_whole<EPL>(v, E, k, lane, mykey, myE);
        else select_cut<EPL>(v, p.logits + static_cast<size_t>(t) * E, E, k, lane, mykey, myE);
        const float myL = lane < k ? key_logit(mykey) : -INFINITY;
        const float L0 = __shfl_sync(0xffffffffu, myL, 0);
        const bool live = masked_in && !(L0 == -INFINITY);
        const bool on = live && lane < k && !(myL == -INFINITY);
        const float ex = on ? expf(myL - L0) : 0.0f;
        float pe[EPL], s = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            pe[i] = live && lane + 32 * i < E ? __expf(v[i] - L0) : 0.0f;
            s += pe[i];
        }
        float z = ex;
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) {  // both sums, interleaved
            z += __shfl_xor_sync(0xffffffffu, z, off);
            s += __shfl_xor_sync(0xffffffffu, s, off);
        }
        if (lane < k) {
            p.idx[static_cast<size_t>(t) * k + lane] = on ? static_cast<int>(myE) : -1;
            p.w[static_cast<size_t>(t) * k + lane] = on ? ex / z : 0.0f;
        }
        if (on) atomicAdd(&hist[myE], 1);
        if (live) {
            const float inv = __fdividef(1.0f, s);
            const float lse = L0 + __logf(s);
#pragma unroll
            for (int i = 0; i < EPL; ++i) accp[i] += pe[i] * inv;
            accz += lse * lse;
            ++accn;
        }
        if (++rows32 == 32) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) { bigp[i] += accp[i]; accp[i] = 0.0f; }
            bigz += accz;
            accz = 0.0f;
            rows32 = 0;
        }
    }

    // CTA sums, warps in order
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (lane + 32 * i < E) sm[warp * E + lane + 32 * i] = bigp[i] + accp[i];
    if (lane == 0) { zsum[warp] = bigz + accz; nsum[warp] = accn; }
    __syncthreads();
    const int b = blockIdx.x, G = gridDim.x;
    const bool one = G == 1;  // one CTA: its sums are the call's
    if (warp == 0) {
        float s = warp_sum(lane < nwarps ? zsum[lane] : 0.0f);
        const int n = __reduce_add_sync(0xffffffffu, lane < nwarps ? nsum[lane] : 0);
        __syncwarp();
        if (lane == 0) {
            if (one) { zsum[0] = s; nsum[0] = n; }
            else { p.part_z[b] = s; p.part_n[b] = n; }
        }
    }
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        float s = 0.0f;
#pragma unroll 8
        for (int w = 0; w < nwarps; ++w) s += sm[w * E + e];
        if (one) {
            sm[e] = s;
        } else {
            p.part[b * E + e] = make_float2(s, __int_as_float(hist[e]));
        }
    }
    __syncthreads();
    if (!one) {
        if (threadIdx.x == 0) {  // after what this CTA wrote, before what the last one reads
            int n;
            asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(n) : "l"(&p.hdr->exit_count) : "memory");
            last = n == G - 1;
            if (last) p.hdr->exit_count = 0;
        }
        __syncthreads();
        if (!last) return;
        // The last CTA: sums over CTAs.  As many threads as fit share an expert's
        // parts (thread group x expert), so that all their loads are in flight.
        if (warp == 0) {
            int n = 0;
            float z = 0.0f;
            for (int g = lane; g < G; g += 32) {
                n += __ldcg(p.part_n + g);
                z += __ldcg(p.part_z + g);
            }
            z = warp_sum(z);
            n = __reduce_add_sync(0xffffffffu, n);
            if (lane == 0) { zsum[0] = z; nsum[0] = n; }
        }
        const int groups = max(1, static_cast<int>(blockDim.x) / E);
        int* csum = reinterpret_cast<int*>(sm + groups * E);
        for (int o = threadIdx.x; o < groups * E; o += blockDim.x) {
            const int e = o % E;
            float s = 0.0f;
            int c = 0;
            constexpr int kBatch = 19;  // all of 152 CTAs' in flight with eight groups
            for (int g0 = o / E; g0 < G; g0 += kBatch * groups) {
                float2 v[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int g = g0 + i * groups;
                    v[i] = g < G ? __ldcg(p.part + g * E + e) : make_float2(0.0f, 0.0f);
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) { s += v[i].x; c += __float_as_int(v[i].y); }
            }
            sm[o] = s;
            csum[o] = c;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < E; e += blockDim.x) {
            float s = 0.0f;
            int c = 0;
#pragma unroll 8
            for (int g = 0; g < groups; ++g) {
                s += sm[g * E + e];
                c += csum[g * E + e];
            }
            sm[e] = s;  // this thread's column alone reads group 0's entry
            hist[e] = c;
        }
        __syncthreads();
    }
    // sm[e], hist[e], zsum[0], nsum[0] are the sums of the call
    if (warp == 0) {
        const int n = nsum[0];
        const float rows = n > 0 ? static_cast<float>(n) : 1.0f;
        float bal = 0.0f;
        for (int e = lane; e < E; e += 32) {
            const float P = sm[e] / rows;
            if (p.counts) p.counts[e] = hist[e];
            if (p.mean_prob) p.mean_prob[e] = P;
            bal += static_cast<float>(hist[e]) / (rows * k) * P;
        }
        bal = warp_sum(bal);
        if (lane == 0) {
            if (p.n_routed) *p.n_routed = n;
            if (p.losses) {
                p.losses[0] = E * bal;
                p.losses[1] = zsum[0] / rows;
            }
        }
    }
}

struct RouterBwdArgs {
    const float* logits;
    const uint8_t* mask;
    const int32_t* idx;
    const float* w;
    const int32_t* counts;
    const int32_t* n_routed;
    const float* d_losses;  // [2] or null
    const float* d_w;       // [T, k] or null
    float* d_logits;
    const int32_t* d_T;
    int T_host, T_max, E, k;
    EtHeader* hdr;
};

// One row a warp; the softmax is recomputed from the logits (4 bytes an entry
// read, 4 written: storing the probabilities would add as much again).  The
// next row's loads go out before the current row's work, and before the first
// row's the loads of the counts, so that one memory latency is paid a warp.
// T = 16384, E = 128, k = 8: 7.4 us after the forward, 10.8 by itself with cold caches, for
// 18 MB (2.7 us of HBM), the larger part of it launch and latency: a warp has one or two rows.
template <int EPL>
__global__ void __launch_bounds__(256) router_bwd_kernel(const RouterBwdArgs p) {
    __shared__ float add_s[8][32 * EPL];  // a row's gradients through the gate weights, by expert
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    const int E = p.E, k = p.k;
    grid_begin();
    bool ok;
    const int T = row_count(p.d_T, p.T_host, p.T_max, p.hdr, &ok);
    if (!ok) return;
    float* add = add_s[warp];
#pragma unroll
    for (int i = 0; i < EPL; ++i) add[lane + 32 * i] = 0.0f;
    __syncwarp();
    const int t0 = blockIdx.x * nwarps + warp, step = gridDim.x * nwarps;
    struct Row {
        float v[EPL], w, dw;
        int e, on;
    };
    auto load = [&](int t, Row& r) {
        const bool in = t < T, sel = in && lane < k && p.d_w;
        const float* L = p.logits + static_cast<size_t>(t) * E;
        const size_t o = static_cast<size_t>(t) * k + lane;
#pragma unroll
        for (int i = 0; i < EPL; ++i) r.v[i] = in && lane + 32 * i < E ? L[lane + 32 * i] : -INFINITY;
        r.on = in && (!p.mask || p.mask[t] != 0);
        r.e = sel ? p.idx[o] : -1;
        r.w = sel ? p.w[o] : 0.0f;
        r.dw = sel ? p.d_w[o] : 0.0f;
    };
    Row nx;
    load(t0, nx);
    const int n = *p.n_routed;
    const float rows = n > 0 ? static_cast<float>(n) : 1.0f;
    const float db = p.d_losses ? p.d_losses[0] : 0.0f;
    const float dz = p.d_losses ? 2.0f * p.d_losses[1] / rows : 0.0f;
    float cost[EPL];  // E f_e / n: what a unit of probability on expert e costs
    const float per = static_cast<float>(E) / (rows * k) / rows;
#pragma unroll
    for (int i = 0; i < EPL; ++i) cost[i] = lane + 32 * i < E ? per * static_cast<float>(p.counts[lane + 32 * i]) : 0.0f;
    for (int t = t0; t < T; t += step) {
        const Row c = nx;
        load(t + step, nx);
        float m = c.v[0];
        bool nan = c.v[0] != c.v[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) {
            m = fmaxf(m, c.v[i]);
            nan |= c.v[i] != c.v[i];
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        nan = __any_sync(0xffffffffu, nan);
        const bool live = c.on && (nan || !(m == -INFINITY));
        float d[EPL];
        if (live) {
            // where the index is -1 neither weight nor gradient is used
            const float w = c.e >= 0 ? c.w : 0.0f, dw = c.e >= 0 ? c.dw : 0.0f;
            float pe[EPL], s = 0.0f, cp = 0.0f, dot = w * dw;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                pe[i] = lane + 32 * i < E ? __expf(c.v[i] - m) : 0.0f;
                s += pe[i];
                cp += pe[i] * cost[i];
            }
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) {  // three sums, interleaved
                s += __shfl_xor_sync(0xffffffffu, s, off);
                cp += __shfl_xor_sync(0xffffffffu, cp, off);
                dot += __shfl_xor_sync(0xffffffffu, dot, off);
            }
            const float inv = __fdividef(1.0f, s);
            cp *= inv;
            const float zl = dz * (m + __logf(s));
            if (p.d_w) {
                // an index outside [0, E) adds nothing; one that comes twice adds twice
                const bool sel = c.e >= 0 && c.e < E;
                if (sel) atomicAdd(add + c.e, w * (dw - dot));
                __syncwarp();
#pragma unroll
                for (int i = 0; i < EPL; ++i) d[i] = add[lane + 32 * i];
                __syncwarp();
                if (sel) add[c.e] = 0.0f;
                __syncwarp();
            } else {
#pragma unroll
                for (int i = 0; i < EPL; ++i) d[i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const float pr = pe[i] * inv;
                d[i] += db * pr * (cost[i] - cp) + zl * pr;
            }
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) d[i] = 0.0f;
        }
        float* out = p.d_logits + static_cast<size_t>(t) * E;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (lane + 32 * i < E) out[lane + 32 * i] = d[i];
    }
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

struct RouterLayout {
    size_t part, part_z, part_n, total;
};

RouterLayout router_layout(int E) {
    RouterLayout L{};
    size_t off = kHeaderBytes;
    L.part = off;
    off = align256(off + sizeof(float2) * kRouterParts * E);
    L.part_z = off;
    off = align256(off + sizeof(float) * kRouterParts);
    L.part_n = off;
    L.total = align256(off + sizeof(int) * kRouterParts);
    return L;
}

bool router_shape_ok(int T_max, int E, int k, std::string* why) {
    if (T_max < 1 || T_max > (1 << 24)) { *why = "T_max must be in [1, 2^24]"; return false; }
    if (E < 1 || E > kRouterEMax) { *why = "E must be in [1, 256]"; return false; }
    if (k < 1 || k > 8 || k > E) { *why = "k must be in [1, min(E, 8)]"; return false; }
    return true;
}

int ceil_div_i(int a, int b) { return a / b + (a % b != 0); }

}  // namespace
}  // namespace et

using namespace et;

extern "C" {

size_t et_router_topk_workspace_bytes(int T_max, int E, int k) {
    if (T_max < 1 || T_max > (1 << 24) || E < 1 || E > kRouterEMax || k < 1 || k > 8 || k > E) return 0;
    return router_layout(E).total;
}

int et_router_topk(const float* logits, const uint8_t* token_mask, int32_t* topk_idx, float* topk_w,
                   int32_t* expert_counts, int32_t* n_routed, float* mean_prob, float* losses, int T,
                   const int32_t* d_T, int T_max, int E, int k, void* workspace,
                   size_t workspace_bytes, void* stream) {
    return api_entry([&]() -> int {
        std::string why;
        if (!router_shape_ok(T_max, E, k, &why)) return api_fail(ET_ERR_UNSUPPORTED, why);
        if (!logits || !topk_idx || !topk_w)
            return api_fail(ET_ERR_INVALID, "logits, topk_idx and topk_w must be non-NULL");
        const void* need4[] = {logits, topk_idx, topk_w, expert_counts, n_routed, mean_prob, losses, d_T};
        for (const void* q : need4)
            if (!api_aligned(q, 4)) return api_fail(ET_ERR_INVALID, "tensors must be aligned to their element size");
        if (!d_T && (T < 0 || T > T_max)) return api_fail(ET_ERR_INVALID, "T must be in [0, T_max]");
        const RouterLayout L = router_layout(E);
        int rc = api_check_ws(workspace, workspace_bytes, L.total);
        if (rc) return rc;
        int dev = 0, sms = 0;
        if ((rc = api_device(&dev, &sms))) return rc;
        uint8_t* ws = static_cast<uint8_t*>(workspace);
        RouterArgs a{logits, token_mask, topk_idx, topk_w, expert_counts, n_routed, mean_prob, losses,
                     d_T, T, T_max, E, k, reinterpret_cast<EtHeader*>(ws),
                     reinterpret_cast<float2*>(ws + L.part),
                     reinterpret_cast<float*>(ws + L.part_z), reinterpret_cast<int32_t*>(ws + L.part_n)};
        const int rows = d_T ? T_max : (T > 0 ? T : 1);
        // One CTA up to 32 rows: nothing to sum over CTAs.  Beyond, as few warps as let the
        // last CTA read all sums in one batch (32 warps / E groups of 19): rows share fewer SMs.
        int warps = rows < kRouterWarpsMax ? rows : kRouterWarpsMax;
        if (rows > kRouterWarpsMax)
            while (warps > 8 && 4ll * rows * E <= 608ll * warps * warps) warps /= 2;
        int grid = ceil_div_i(rows, warps);
        grid = grid < kRouterParts ? grid : kRouterParts;
        // [warps][E] floats; the last CTA: max(1, threads / E) x E of a float and an int
        const size_t sums = static_cast<size_t>(warps * 32 / E > 1 ? warps * 32 / E : 1) * E * 8;
        const size_t rows_p = sizeof(float) * warps * E;
        const size_t smem = rows_p > sums ? rows_p : sums;
        auto kernel = E <= 32 ? router_topk_kernel<1> : E <= 64 ? router_topk_kernel<2>
                    : E <= 128 ? router_topk_kernel<4> : router_topk_kernel<8>;
        const cudaError_t e = api_launch(kernel, grid, warps * 32, smem, stream, a);
        if (e != cudaSuccess) return api_fail_cuda(e, "launch of the router kernel");
        return ET_OK;
    });
}

int et_router_topk_bwd(const float* logits, const uint8_t* token_mask, const int32_t* topk_idx,
                       const float* topk_w, const int32_t* expert_counts, const int32_t* n_routed,
                       const float* d_losses, const float* d_topk_w, float* d_logits, int T,
                       const int32_t* d_T, int T_max, int E, int k, void* workspace,
                       size_t workspace_bytes, void* stream) {
    return api_entry([&]() -> int {
        std::string why;
        if (!router_shape_ok(T_max, E, k, &why)) return api_fail(ET_ERR_UNSUPPORTED, why);
        if (!logits || !topk_idx || !topk_w || !expert_counts || !n_routed || !d_logits)
            return api_fail(ET_ERR_INVALID, "logits, topk_idx, topk_w, expert_counts, n_routed and d_logits "
                                            "must be non-NULL");
        const void* need4[] = {logits, topk_idx, topk_w, expert_counts, n_routed, d_losses, d_topk_w, d_logits, d_T};
        for (const void* q : need4)
            if (!api_aligned(q, 4)) return api_fail(ET_ERR_INVALID, "tensors must be aligned to their element size");
        if (!d_T && (T < 0 || T > T_max)) return api_fail(ET_ERR_INVALID, "T must be in [0, T_max]");
        int rc = api_check_ws(workspace, workspace_bytes, kHeaderBytes);
        if (rc) return rc;
        if (!d_T && T == 0) return ET_OK;
        int dev = 0, sms = 0;
        if ((rc = api_device(&dev, &sms))) return rc;
        RouterBwdArgs a{logits, token_mask, topk_idx, topk_w, expert_counts, n_routed, d_losses, d_topk_w,
                        d_logits, d_T, T, T_max, E, k, static_cast<EtHeader*>(workspace)};
        const int rows = d_T ? T_max : T;
        int grid = ceil_div_i(rows, 8);
        grid = grid < 8 * sms ? grid : 8 * sms;
        auto kernel = E <= 32 ? router_bwd_kernel<1> : E <= 64 ? router_bwd_kernel<2>
                    : E <= 128 ? router_bwd_kernel<4> : router_bwd_kernel<8>;
        const cudaError_t e = api_launch(kernel, grid, 256, 0, stream, a);
        if (e != cudaSuccess) return api_fail_cuda(e, "launch of the router's backward kernel");
        return ET_OK;
    });
}

}  // extern "C"
