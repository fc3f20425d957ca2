// router_sums.cuh -- what the router kernels share: the order of logits, and the
// sums over tokens (counts, mean probabilities, losses) that a call ends with.
#pragma once

#include "et_api.h"
#include "ops_device.cuh"

namespace et {
namespace {

constexpr int kRouterWarpsMax = 32;
constexpr int kRouterEMax = 256;
constexpr int kRouterParts = 152;  // most CTAs of a forward kernel = rows of partial sums

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

}  // namespace

// Where the sums go (each output may be null) and meet.
struct RouterSums {
    int32_t* counts;         // [E]
    int32_t* n_routed;       // [1]
    float* mean_prob;        // [E]
    float* losses;           // [2], balance and z; without z_loss [1]
    bool z_loss;
    EtHeader* hdr;
    float2* part;            // [kRouterParts, E]: a CTA's sum of probabilities; its count, as an integer
    float* part_z;           // [kRouterParts]
    int32_t* part_n;         // [kRouterParts]
};

namespace {

struct RouterShared {
    int hist[kRouterEMax];   // how often this CTA's tokens chose an expert
    float zsum[kRouterWarpsMax];
    int nsum[kRouterWarpsMax];
    int last;
};

// The end of a forward kernel, reached by the whole CTA: each warp has stored its sums
// of probabilities as sm[warp][E]; accz and accn are its sum of squared log(sum exp)
// and its routed tokens.  Sums run over warps, then (in the last CTA to finish) over
// CTAs, each in a fixed order.
__device__ __forceinline__ void router_sums(const RouterSums& p, float* sm, RouterShared& sh, int E, int k, float accz, int accn) {
    // CTA sums, warps in order
    int* hist = sh.hist;
    float* zsum = sh.zsum;
    int* nsum = sh.nsum;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    if (lane == 0) { zsum[warp] = accz; nsum[warp] = accn; }
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
            sh.last = n == G - 1;
            if (sh.last) p.hdr->exit_count = 0;
        }
        __syncthreads();
        if (!sh.last) return;
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
                if (p.z_loss) p.losses[1] = zsum[0] / rows;
            }
        }
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

RouterSums router_sums_args(void* workspace, const RouterLayout& L, int32_t* counts, int32_t* n_routed, float* mean_prob,
                            float* losses, bool z_loss) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    return {counts, n_routed, mean_prob, losses, z_loss, reinterpret_cast<EtHeader*>(ws), reinterpret_cast<float2*>(ws + L.part),
            reinterpret_cast<float*>(ws + L.part_z), reinterpret_cast<int32_t*>(ws + L.part_n)};
}

struct RouterGrid {
    int ctas, warps;
    size_t smem;
};

// A forward kernel's launch for this many rows, one a warp.
RouterGrid router_grid_of(int rows, int E, int warps) {
    RouterGrid g;
    g.warps = warps;
    g.ctas = ceil_div_i(rows, g.warps);
    g.ctas = g.ctas < kRouterParts ? g.ctas : kRouterParts;
    // [warps][E] floats; the last CTA: max(1, threads / E) x E of a float and an int
    const size_t sums = static_cast<size_t>(g.warps * 32 / E > 1 ? g.warps * 32 / E : 1) * E * 8;
    const size_t rows_p = sizeof(float) * g.warps * E;
    g.smem = rows_p > sums ? rows_p : sums;
    return g;
}

// One CTA up to 32 rows: nothing to sum over CTAs.  Beyond, as few warps as let the last
// CTA read all sums in one batch (32 warps / E groups of 19): rows share fewer SMs.
RouterGrid router_grid(int rows, int E) {
    int warps = rows < kRouterWarpsMax ? rows : kRouterWarpsMax;
    if (rows > kRouterWarpsMax)
        while (warps > 8 && 4ll * rows * E <= 608ll * warps * warps) warps /= 2;
    return router_grid_of(rows, E, warps);
}

}  // namespace
}  // namespace et
