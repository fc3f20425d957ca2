// router_groups.cu -- the router with scores by softmax or sigmoid, a bias that
// only the choice sees, and groups of experts of which the best take part; its
// balance loss, and the gradient.
#include <cmath>

#include "../../include/etmoe.h"
#include "router_sums.cuh"

namespace et {
namespace {

constexpr int kGroupsMax = 32;

struct GroupArgs {
    const float* logits;     // [T, E]
    const float* bias;       // [E] or null
    const uint8_t* mask;     // [T] or null
    int32_t* idx;            // [T, k]
    float* w;                // [T, k]
    const int32_t* d_T;
    int T_host, T_max, E, k;
    int G, kg, best;         // groups, how many take part, whose `best` experts rank them
    int gs;                  // experts a group
    int lanes;               // lanes that hold a group where that is a power of two, else 0
    int renorm, vec;
    float scale;
    RouterSums sums;
};

__device__ __forceinline__ double key_value(unsigned long long key) {
    return __longlong_as_double(static_cast<long long>(key >> 63 ? key ^ 0x8000000000000000ull : ~key));
}

// logit_key of a 64-bit value; NaN above all, > 0 everywhere.
__device__ __forceinline__ unsigned long long value_key(double v) {
    if (v != v) return ~0ull;
    const long long b = __double_as_longlong(v + 0.0);
    return static_cast<unsigned long long>(b) ^ (static_cast<unsigned long long>(b >> 63) | 0x8000000000000000ull);
}

// The whole choice in 64 bits, for the rows where 32 cannot tell.  Lane `lane` has the
// experts lane * EPL + i.  Returns lane j's expert, the j-th, or -1.
// Out of line and in plain loops: one row in some hundreds comes here.
template <int EPL>
__device__ __noinline__ int choose64(const float* row, const float* bias, int E, int k, int G, int kg, int best, int gs,
                                     int sigmoid, int lane) {
    constexpr uint32_t kAll = 0xffffffffu;
    unsigned long long key[EPL];  // of score + bias; 0: not available
    float v[EPL];
    double m = 0.0, Z = 1.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = lane * EPL + i < E ? row[lane * EPL + i] : -INFINITY;
    if (!sigmoid) {
        float top = v[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) top = fmaxf(top, v[i]);
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, off));
        m = top;
        Z = 0.0;
#pragma unroll 1
        for (int i = 0; i < EPL; ++i) Z += exp(static_cast<double>(v[i]) - m);  // 0 past E
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) Z += __shfl_xor_sync(kAll, Z, off);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const double x = v[i];
        key[i] = 0;
        if (!(v[i] == -INFINITY)) {
            double c = sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - m) / Z;
            if (bias) c += static_cast<double>(bias[lane * EPL + i]);
            if (!(c == -INFINITY)) key[i] = value_key(c);
        }
    }
    if (kg < G) {
        double score = -INFINITY;  // lane g: of group g
#pragma unroll 1
        for (int g = 0; g < G; ++g) {
            unsigned long long hi = 0, lo = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int e = lane * EPL + i;
                if (e >= g * gs && e < g * gs + gs) {
                    lo = max(lo, min(hi, key[i]));
                    hi = max(hi, key[i]);
                }
            }
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) {
                const unsigned long long h = __shfl_xor_sync(kAll, hi, off), l = __shfl_xor_sync(kAll, lo, off);
                lo = max(max(lo, l), min(hi, h));
                hi = max(hi, h);
            }
            double s = hi ? key_value(hi) : -INFINITY;
            if (best > 1 && lo) s += key_value(lo);
            if (lane == g) score = s;
        }
        const unsigned long long mine = value_key(score);
        int rank = 0;
#pragma unroll 1
        for (int g = 0; g < G; ++g) {
            const unsigned long long other = __shfl_sync(kAll, mine, g);
            rank += other > mine || (other == mine && g < lane);
        }
        const uint32_t in = __ballot_sync(kAll, lane < G && rank < kg);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane * EPL + i;
            if (e >= E || !(in >> (e / gs) & 1)) key[i] = 0;
        }
    }
    int mineE = -1;
#pragma unroll 1
    for (int j = 0; j < k; ++j) {
        unsigned long long hi = 0;
        int at = E;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (key[i] > hi) {
                hi = key[i];
                at = lane * EPL + i;
            }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) {
            const unsigned long long h = __shfl_xor_sync(kAll, hi, off);
            const int a = __shfl_xor_sync(kAll, at, off);
            if (h > hi || (h == hi && a < at)) {
                hi = h;
                at = a;
            }
        }
        if (hi && lane == j) mineE = at;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (lane * EPL + i == at) key[i] = 0;
    }
    return mineE;
}

constexpr uint32_t kNegInfKey = 0x007fffffu;  // logit_key(-inf); nothing available has it or less

__device__ __forceinline__ float rcp_fast(float x) {  // within 1 ulp; 0 for +inf
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float sigmoid_fast(float v) { return rcp_fast(1.0f + __expf(-v)); }  // 0 for -inf

// The float of a key, -inf where nothing is available.
__device__ __forceinline__ float key_or_none(uint32_t key) { return key > kNegInfKey ? key_logit(key) : -INFINITY; }

// logit_key of a score (>= 0 or NaN).  In assembly: as C++ it became a negation, which makes
// the one positive NaN of -NaN.
__device__ __forceinline__ uint32_t score_key(float s) {
    uint32_t k;
    asm("or.b32 %0, %1, 0x80000000;" : "=r"(k) : "r"(__float_as_uint(s)));
    return k;
}

// Sorts a lane's keys, the largest first.
template <int EPL>
__device__ __forceinline__ void sort_keys(uint32_t (&k)[EPL]) {
    auto swap = [&](int a, int b) {
        const uint32_t hi = max(k[a], k[b]);
        k[b] = min(k[a], k[b]);
        k[a] = hi;
    };
    // odd-even merge sort
    if (EPL == 2) swap(0, 1);
    if (EPL >= 4) {
#pragma unroll
        for (int o = 0; o + 3 < EPL; o += 4) {
            swap(o, o + 1); swap(o + 2, o + 3);
            swap(o, o + 2); swap(o + 1, o + 3);
            swap(o + 1, o + 2);
        }
    }
    if (EPL == 8) {
        swap(0, 4 % EPL); swap(1 % EPL, 5 % EPL); swap(2 % EPL, 6 % EPL); swap(3 % EPL, 7 % EPL);
        swap(2 % EPL, 4 % EPL); swap(3 % EPL, 5 % EPL);
        swap(1 % EPL, 2 % EPL); swap(3 % EPL, 4 % EPL); swap(5 % EPL, 6 % EPL);
    }
}

constexpr int kCandidates = 16;  // experts whose order is looked at again at most

// score + bias in 64 bits, without a bias and with softmax scores the logit, which orders alike.
__device__ __forceinline__ double value64(float x, float b, bool sigmoid) {
    return sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(x))) + static_cast<double>(b) : static_cast<double>(x);
}

// Two groups whose scores 32 bits cannot tell apart: 1 if the first has the larger, or the
// same and the lower number, 0 if the second, -1 if it takes more than their best two to
// say.  Sigmoid scores.  floor_a, floor_b: what the experts that count are not below;
// want_a, want_b: how many those are.  slots: 16 places of shared memory.
template <int EPL>
__device__ __noinline__ int compare_groups(const float* row, const float* bias_s, int E, int gs, int a, int b, float floor_a,
                                           float floor_b, int want_a, int want_b, uint32_t* slots, int lane) {
    constexpr uint32_t kAll = 0xffffffffu;
    int na = 0, nb = 0;
#pragma unroll 1
    for (int i = 0; i < EPL; ++i) {
        const int e = lane * EPL + i, g = e / gs;
        const float x = e < E ? row[e] : -INFINITY;
        const float c = x == -INFINITY ? x : __fadd_rn(sigmoid_fast(x), bias_s[min(e, E - 1)]);
        const uint32_t in_a = __ballot_sync(kAll, e < E && g == a && c >= floor_a);
        const uint32_t in_b = __ballot_sync(kAll, e < E && g == b && c >= floor_b);
        const uint32_t bit = 1u << lane, below = bit - 1;
        if ((in_a & bit) && na + __popc(in_a & below) < 8) slots[na + __popc(in_a & below)] = e;
        if ((in_b & bit) && nb + __popc(in_b & below) < 8) slots[8 + nb + __popc(in_b & below)] = e;
        na += __popc(in_a);
        nb += __popc(in_b);
    }
    __syncwarp();
    if (na != want_a || nb != want_b) return -1;
    const bool mine = lane < na || (lane >= 8 && lane < 8 + nb);
    const int e = mine ? static_cast<int>(slots[lane]) : 0;
    double c = mine ? value64(row[e], bias_s[e], true) : 0.0;
    c += __shfl_xor_sync(kAll, c, 1);  // two at most
    const double sa = __shfl_sync(kAll, c, 0), sb = __shfl_sync(kAll, c, 8);
    return sa > sb || (sa == sb && a < b) ? 1 : 0;
}

// The order of n candidates (n <= kCandidates, their experts in slots) in 64 bits: puts the
// best k there in their order.
__device__ __noinline__ void order_again(const float* row, const float* bias_s, bool sigmoid, int n, int k, uint32_t* slots, int lane) {
    constexpr uint32_t kAll = 0xffffffffu;
    const int e = lane < n ? static_cast<int>(slots[lane]) : 0;
    const double c = lane < n ? value64(row[e], bias_s[e], sigmoid) : 0.0;
    const unsigned long long key = value_key(c);
    int rank = 0;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const unsigned long long other = __shfl_sync(kAll, key, i);
        const int oe = __shfl_sync(kAll, e, i);
        rank += other > key || (other == key && oe < e);
    }
    __syncwarp();
    if (lane < n && rank < k) slots[rank] = e;
    __syncwarp();
}

// One row a warp, experts lane * EPL + i in register i, so that a group is a few
// neighbouring lanes.  The choice runs on 32-bit values: without a bias on the logits,
// which order as the scores do and are exact; with one on score + bias, whose error has a
// bound.  A lane's keys, cut by the bits that name its experts, are sorted once; a round
// of the choice looks at the heads alone, and takes the lowest lane of those with the
// largest cut key.  Where two neighbours in the order are no farther apart than the cut
// and both errors, or the last group that takes part and the next than theirs, 64 bits
// decide: on the candidates alone (a lane each: 1.3 us where a whole row takes 14), and on
// the whole row if they are too many, or softmax scores with a bias.
template <int EPL, bool SIGMOID>
__global__ void __launch_bounds__(kRouterWarpsMax * 32) router_groups_kernel(const GroupArgs p) {
    constexpr uint32_t kAll = 0xffffffffu, kLow = EPL - 1;
    constexpr float kU = 1.0f / (1 << 24);
    extern __shared__ __align__(16) float sm[];  // [warps][E], then the last CTA's sums
    __shared__ RouterShared sh;
    __shared__ uint32_t chosen[kRouterWarpsMax][kCandidates];
    __shared__ float bias_s[kRouterEMax];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    const int E = p.E, k = p.k, e0 = lane * EPL;
    const uint32_t below = (1u << lane) - 1;
    grid_begin();
    bool ok;
    const int T = row_count(p.d_T, p.T_host, p.T_max, p.sums.hdr, &ok);
    if (!ok) return;
    const int t0 = blockIdx.x + gridDim.x * warp, step = gridDim.x * nwarps;
    auto load = [&](int t, float (&v)[EPL], int& on) {
        const float* L = p.logits + static_cast<size_t>(t) * E + e0;
        on = t < T && (!p.mask || p.mask[t] != 0);
        if (EPL >= 4 && p.vec) {  // E a multiple of 4, rows 16-byte aligned
#pragma unroll
            for (int i = 0; i < EPL; i += 4) {
                float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                if (t < T && e0 + i < E) q = *reinterpret_cast<const float4*>(L + i);
                v[i] = q.x;
                v[(i + 1) % EPL] = q.y;
                v[(i + 2) % EPL] = q.z;
                v[(i + 3) % EPL] = q.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) v[i] = t < T && e0 + i < E ? L[i] : -INFINITY;
        }
    };
    float nv[EPL];
    int non;
    load(t0, nv, non);
    for (int e = threadIdx.x; e < kRouterEMax; e += blockDim.x) {
        if (e < E) sh.hist[e] = 0;
        bias_s[e] = p.bias && e < E ? p.bias[e] : 0.0f;
    }
    float* const big = sm + warp * E + e0;  // this lane's sums of whole batches of 32 rows
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (e0 + i < E) big[i] = 0.0f;
    __syncthreads();

    float accp[EPL];
    int accn = 0, rows32 = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) accp[i] = 0.0f;

    for (int t = t0; t < T; t += step) {
        float v[EPL], s[EPL], S = 0.0f, top = 0.0f;
        const int masked_in = non;
#pragma unroll
        for (int i = 0; i < EPL; ++i) v[i] = nv[i];
        load(t + step, nv, non);

        // scores s, their sum S
        if (!SIGMOID) {
            top = v[0];
#pragma unroll
            for (int i = 1; i < EPL; ++i) top = fmaxf(top, v[i]);
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, off));
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            s[i] = SIGMOID ? sigmoid_fast(v[i]) : v[i] == -INFINITY ? 0.0f : __expf(v[i] - top);
            S += s[i];
        }
        S = warp_sum(S);
        const float inv = __fdividef(1.0f, S);
        if (!SIGMOID) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) s[i] *= inv;
        }
        // How far a score can be off: sigmoid 6 x 2^-24 (exp within 2 + 1.2 |x| ulp, times the
        // slope e^x / (1 + e^x)^2 <= 1/4; an add; a reciprocal within 1 ulp), softmax 40 x 2^-24
        // of the largest, 1 / S (its sum's terms are off by 8.5 ulp on average at most, as their
        // mean |x - top| is below log 256).
        const float err = (SIGMOID ? 10.0f : 48.0f * inv) * kU;

        uint32_t key[EPL];  // kNegInfKey or 0: not available
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            float c = v[i];
            if (p.bias) c = v[i] == -INFINITY ? v[i] : __fadd_rn(s[i], bias_s[e0 + i]);
            key[i] = logit_key(c);
        }
        bool again = false;  // the whole row in 64 bits
        if (p.kg < p.G) {
            float score = -INFINITY, mag = 0.0f;  // lane g: of group g
            auto group_score = [&](uint32_t hi, uint32_t lo) {  // from its best two values of score + bias
                const float h = key_or_none(hi), l = lo > kNegInfKey ? key_logit(lo) : 0.0f;
                score = h + (p.best > 1 ? l : 0.0f);
                mag = fabsf(h) + fabsf(l);
            };
            uint32_t hi = 0, lo = 0;
            if (p.lanes) {
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const uint32_t c = p.bias || key[i] <= kNegInfKey ? key[i] : score_key(s[i]);
                    lo = max(lo, min(hi, c));
                    hi = max(hi, c);
                }
                for (int off = 1; off < p.lanes; off <<= 1) {
                    const uint32_t h = __shfl_xor_sync(kAll, hi, off), l = __shfl_xor_sync(kAll, lo, off);
                    lo = max(max(lo, l), min(hi, h));
                    hi = max(hi, h);
                }
                const int from = min(lane * p.lanes, 31);
                hi = __shfl_sync(kAll, hi, from);
                lo = __shfl_sync(kAll, lo, from);
            } else {
#pragma unroll 1
                for (int g = 0; g < p.G; ++g) {
                    uint32_t h = 0, l = 0;
#pragma unroll
                    for (int i = 0; i < EPL; ++i) {
                        const bool in = e0 + i >= g * p.gs && e0 + i < g * p.gs + p.gs;
                        const uint32_t c = !in ? 0u : p.bias || key[i] <= kNegInfKey ? key[i] : score_key(s[i]);
                        l = max(l, min(h, c));
                        h = max(h, c);
                    }
                    const uint32_t H = __reduce_max_sync(kAll, h);
                    // its holder's second best (the first holder's, where several hold it)
                    const uint32_t who = __ballot_sync(kAll, h == H);
                    const uint32_t L = __reduce_max_sync(kAll, lane == __ffs(who) - 1 ? l : h);
                    if (lane == g) {
                        hi = H;
                        lo = L;
                    }
                }
            }
            if (lane < p.G) group_score(hi, lo);
            const uint32_t mine = logit_key(score);
            int rank = 0;
#pragma unroll 4
            for (int g = 0; g < p.G; ++g) {
                const uint32_t other = __shfl_sync(kAll, mine, g);
                rank += other > mine || (other == mine && g < lane);
            }
            uint32_t in = __ballot_sync(kAll, lane < p.G && rank < p.kg);
            // the last that takes part and the next: apart by more than any two may be off
            const uint32_t last_in = __ballot_sync(kAll, lane < p.G && rank == p.kg - 1);
            const uint32_t next = __ballot_sync(kAll, lane < p.G && rank == p.kg);
            const float off_by = 2.0f * err + 2.0f * kU * mag;
            const float a = __shfl_sync(kAll, score, __ffs(last_in) - 1), b = __shfl_sync(kAll, score, __ffs(next) - 1);
            const float tol = 2.0f * __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(off_by)));
            if (!(a - b > tol) && !(b == -INFINITY)) {
                const int ga = __ffs(last_in) - 1, gb = __ffs(next) - 1;
                // between these two alone?
                const bool other = lane < p.G && !(rank < p.kg - 1 ? score - b > tol : rank > p.kg ? a - score > tol : true);
                again = !SIGMOID || !(tol < 1.0f) || __any_sync(kAll, other);
                if (!again) {
                    const uint32_t last = p.best > 1 && lo > kNegInfKey ? lo : hi;  // the last that counts
                    const float floor = key_or_none(last) - tol;
                    const int want = last == hi && (p.best == 1 || lo <= kNegInfKey) ? 1 : 2;
                    const int r = compare_groups<EPL>(p.logits + static_cast<size_t>(t) * E, bias_s, E, p.gs, ga, gb,
                                                      __shfl_sync(kAll, floor, ga), __shfl_sync(kAll, floor, gb),
                                                      __shfl_sync(kAll, want, ga), __shfl_sync(kAll, want, gb), chosen[warp], lane);
                    again = r < 0;
                    if (r == 0) in ^= 1u << ga | 1u << gb;
                    __syncwarp();
                }
            }
            if (p.lanes) {
                const bool out = !(in >> (lane / p.lanes & 31) & 1);
#pragma unroll
                for (int i = 0; i < EPL; ++i) key[i] = out ? 0u : key[i];
            } else {
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (!(in >> ((e0 + i) / p.gs & 31) & 1)) key[i] = 0u;
            }
        }

        // the best k and the next one; lane j: the j-th
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = (key[i] & ~kLow) | (kLow - i);
        sort_keys<EPL>(key);
        auto take = [&](int j) -> uint32_t {  // the largest cut key; its expert goes to chosen[j]
            const uint32_t best = __reduce_max_sync(kAll, key[0]);
            const bool mine = (key[0] ^ best) <= kLow;
            const uint32_t who = __ballot_sync(kAll, mine);
            if (mine && !(who & below)) {
                chosen[warp][j] = e0 + (kLow - (key[0] & kLow));
#pragma unroll
                for (int i = 0; i < EPL; ++i) key[i] = i + 1 < EPL ? key[(i + 1) % EPL] : 0u;
            }
            return best;
        };
        uint32_t mykey = 0;
#pragma unroll 1
        for (int j = 0; j <= k; ++j) {
            const uint32_t best = take(j);
            if (lane == j) mykey = best;
        }
        __syncwarp();
        const float* row = p.logits + static_cast<size_t>(t) * E;
        const bool there = lane <= k && mykey > (kNegInfKey | kLow);
        bool on = lane < k && there;
        int myE = there ? static_cast<int>(chosen[warp][lane & 15]) : 0;
        float myL = there ? row[myE] : -INFINITY;
        {
            const float b = there ? bias_s[myE] : 0.0f;
            // score + bias as above
            const float c = !there ? -INFINITY : !p.bias ? myL : __fadd_rn(SIGMOID ? sigmoid_fast(myL) : __expf(myL - top) * inv, b);
            const float cn = __shfl_down_sync(kAll, c, 1), bn = __shfl_down_sync(kAll, b, 1), Ln = __shfl_down_sync(kAll, myL, 1);
            const uint32_t keyn = __shfl_down_sync(kAll, mykey, 1);
            const bool equal = b == bn && myL == Ln;  // a true tie, in the order of the experts already
            // with a bias: both errors and the cut; without: the order is the whole key's unless
            // the cut key is one, or the scores meet at 1 or 0 in 64 bits
            const float tol = 2.0f * err + (kU + 2.0f * EPL * kU) * (fabsf(c) + fabsf(cn));
            const bool meet = SIGMOID ? Ln > 16.0f || Ln < -700.0f : Ln - top < -700.0f;
            const bool close = p.bias ? !(c - cn > tol) : meet || ((mykey ^ keyn) <= kLow && (c < cn || c != c || lane == k - 1));
            const bool pair = on && keyn > (kNegInfKey | kLow);
            bool doubt = __any_sync(kAll, pair && !equal && close);
            const bool met = __any_sync(kAll, pair && !equal && meet);
            // after a true tie across the k-th place, whoever comes next must be apart from it, too
            bool tie = __ballot_sync(kAll, pair && equal) >> (k - 1) & 1;
            const float ck = __shfl_sync(kAll, c, k - 1), tk = __shfl_sync(kAll, tol, k - 1);
            int n = k + 1;  // experts taken so far
            while (tie && !doubt && !again) {
                const float Lk = __shfl_sync(kAll, myL, k - 1), bk = __shfl_sync(kAll, b, k - 1);
                const uint32_t keyk = __shfl_sync(kAll, mykey, k - 1);
                const uint32_t best = take(k);
                __syncwarp();
                const int e = static_cast<int>(chosen[warp][k]);
                __syncwarp();
                tie = false;
                if (best > (kNegInfKey | kLow)) {
                    const float L = row[e];
                    tie = L == Lk && bias_s[e] == bk;
                    // (experts equal to the k-th are lost to the list of candidates)
                    if (!tie) again = p.bias ? !(ck - key_logit(best | kLow) > tk) : (keyk ^ best) <= kLow;
                }
            }
            if (doubt && !again) {
                // candidates until the next one is apart from the k-th, the least of the first k
                float ckmin = lane < k ? c : INFINITY;
#pragma unroll
                for (int off = 8; off >= 1; off >>= 1) ckmin = fminf(ckmin, __shfl_xor_sync(kAll, ckmin, off));
                ckmin = __shfl_sync(kAll, ckmin, 0);
                const float t2 = p.bias ? 2.0f * err + (4.0f * EPL + 2.0f) * kU * fabsf(ckmin) : 0.0f;
                uint32_t last = __shfl_sync(kAll, mykey, k);
                while (n < kCandidates && last > (kNegInfKey | kLow) && !(ckmin - key_logit(last | kLow) > t2)) last = take(n++);
                again = (!SIGMOID && p.bias) || (!SIGMOID && met) || !(ckmin == ckmin) ||
                        (n == kCandidates && last > (kNegInfKey | kLow) && !(ckmin - key_logit(last | kLow) > t2));
                if (!again) {
                    __syncwarp();
                    // (the last taken may be none, and of the first ones too)
                    const int base = __popc(__ballot_sync(kAll, there));
                    const int have = base <= k ? base : last > (kNegInfKey | kLow) ? n : n - 1;
                    order_again(row, bias_s, SIGMOID, have, k, chosen[warp], lane);
                    myE = lane < k && lane < have ? static_cast<int>(chosen[warp][lane & 15]) : 0;
                    on = lane < k && lane < have;
                    myL = on ? row[myE] : -INFINITY;
                }
            }
        }
        if (again) {
            myE = choose64<EPL>(row, p.bias, E, k, p.G, p.kg, p.best, p.gs, SIGMOID, lane);
            on = lane < k && myE >= 0;
            myL = on ? row[myE] : -INFINITY;
        }
        const bool any = __any_sync(kAll, on), live = masked_in && any;
        on = on && live;

        // the weights, to full precision: by ratios of e^L where all scores are tiny
        float Lm = on ? myL : -INFINITY;
#pragma unroll
        for (int off = 4; off >= 1; off >>= 1) Lm = fmaxf(Lm, __shfl_xor_sync(kAll, Lm, off));
        Lm = __shfl_sync(kAll, Lm, 0);
        float x = 0.0f, z = 1.0f;
        if (on) {
            if (p.renorm) x = !SIGMOID || Lm < -60.0f ? expf(myL - Lm) : 1.0f / (1.0f + expf(-myL));
            else x = SIGMOID ? 1.0f / (1.0f + expf(-myL)) : expf(myL - top);
            if (!SIGMOID && S != S) x = S;  // a NaN or infinite logit shows, chosen or not
        }
        if (p.renorm) {
            z = x;
#pragma unroll
            for (int off = 4; off >= 1; off >>= 1) z += __shfl_xor_sync(kAll, z, off);
        } else if (!SIGMOID) {
            z = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) z += v[i] == -INFINITY ? 0.0f : expf(v[i] - top);
            z = warp_sum(z);
        }
        if (lane < k) {
            p.idx[static_cast<size_t>(t) * k + lane] = on ? myE : -1;
            p.w[static_cast<size_t>(t) * k + lane] = on ? p.scale * (x / z) : 0.0f;
        }
        if (on) atomicAdd(&sh.hist[myE], 1);
        if (live) {
            float q = SIGMOID ? inv : 1.0f;
            if (SIGMOID && !(S >= 1e-24f) && S == S) {  // scores as small as that (all below e^-55): their ratios
                top = v[0];
#pragma unroll
                for (int i = 1; i < EPL; ++i) top = fmaxf(top, v[i]);
#pragma unroll
                for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, off));
                q = 0.0f;
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    s[i] = v[i] == -INFINITY ? 0.0f : __expf(v[i] - top);
                    q += s[i];
                }
                q = __fdividef(1.0f, warp_sum(q));
            }
#pragma unroll
            for (int i = 0; i < EPL; ++i) accp[i] += s[i] * q;
            ++accn;
        }
        if (++rows32 == 32) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                if (e0 + i < E) big[i] += accp[i];
                accp[i] = 0.0f;
            }
            rows32 = 0;
        }
        __syncwarp();  // `chosen` is written again
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (e0 + i < E) big[i] += accp[i];
    router_sums(p.sums, sm, sh, E, k, 0.0f, accn);
}

struct GroupBwdArgs {
    const float* logits;
    const uint8_t* mask;
    const int32_t* idx;
    const float* w;
    const int32_t* counts;
    const int32_t* n_routed;
    const float* d_loss;    // [1] or null
    const float* d_w;       // [T, k] or null
    float* d_logits;
    const int32_t* d_T;
    int T_host, T_max, E, k;
    int sigmoid, renorm;
    float inv_scale;        // 0 where scale is
    EtHeader* hdr;
};

// One row a warp; scores are made again from the logits.  With q = 1 - s (sigmoid) or 1
// (softmax), p = s / sum s and W_j = w_j d_w_j:
//   d_L[e] = q_e (d_loss p_e (C_e - sum C p) + sum_{j: idx_j = e} (W_j - r_j)) - u p_e,
//   r_j = w_j sum W / scale with renorm; u = sum W for softmax without; else 0.
// A token is routed if it has an index that is not -1.
template <int EPL>
__global__ void __launch_bounds__(256) router_groups_bwd_kernel(const GroupBwdArgs p) {
    constexpr uint32_t kAll = 0xffffffffu;
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
        const bool in = t < T, sel = in && lane < k;
        const float* L = p.logits + static_cast<size_t>(t) * E;
        const size_t o = static_cast<size_t>(t) * k + lane;
#pragma unroll
        for (int i = 0; i < EPL; ++i) r.v[i] = in && lane + 32 * i < E ? L[lane + 32 * i] : -INFINITY;
        r.on = in && (!p.mask || p.mask[t] != 0);
        r.e = sel ? p.idx[o] : -1;
        r.w = sel ? p.w[o] : 0.0f;
        r.dw = sel && p.d_w ? p.d_w[o] : 0.0f;
    };
    Row nx;
    load(t0, nx);
    const int n = *p.n_routed;
    const float rows = n > 0 ? static_cast<float>(n) : 1.0f;
    const float dl = p.d_loss ? *p.d_loss : 0.0f;
    float cost[EPL];  // E counts / (n^2 k): what a unit of p on expert e costs
    const float per = static_cast<float>(E) / (rows * k) / rows;
#pragma unroll
    for (int i = 0; i < EPL; ++i) cost[i] = lane + 32 * i < E ? per * static_cast<float>(p.counts[lane + 32 * i]) : 0.0f;
    for (int t = t0; t < T; t += step) {
        const Row c = nx;
        load(t + step, nx);
        float top = c.v[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) top = fmaxf(top, c.v[i]);
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, off));
        const bool sel = c.e >= 0 && c.e < E;
        const bool any = __any_sync(kAll, c.e >= 0), live = c.on && any;
        float d[EPL];
        if (live) {
            const float W = c.e >= 0 ? c.w * c.dw : 0.0f;
            const bool ratio = !p.sigmoid || top < -60.0f;  // scores as ratios of e^L
            float s[EPL], q[EPL], S = 0.0f, cp = 0.0f, sum = W;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const bool there = !(c.v[i] == -INFINITY);
                const float e = __expf(-fabsf(c.v[i]));  // sigmoid of either sign without overflow
                const float h = __fdividef(1.0f, 1.0f + e);
                const float lo = e * h;
                s[i] = !there ? 0.0f : ratio ? __expf(c.v[i] - top) : c.v[i] < 0.0f ? lo : h;
                q[i] = !p.sigmoid ? 1.0f : c.v[i] < 0.0f ? h : lo;
                if (c.v[i] != c.v[i]) s[i] = q[i] = c.v[i];
                S += s[i];
                cp += s[i] * cost[i];
            }
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) {  // three sums, interleaved
                S += __shfl_xor_sync(kAll, S, off);
                cp += __shfl_xor_sync(kAll, cp, off);
                sum += __shfl_xor_sync(kAll, sum, off);
            }
            const float inv = __fdividef(1.0f, S);
            cp *= inv;
            const float u = !p.renorm && !p.sigmoid ? sum : 0.0f;
            if (p.d_w) {
                // an index outside [0, E) adds nothing; one that comes twice adds twice
                if (sel) atomicAdd(add + c.e, p.renorm ? W - c.w * p.inv_scale * sum : W);
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
                const float pr = s[i] * inv;
                d[i] = q[i] * (dl * pr * (cost[i] - cp) + d[i]) - u * pr;
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

int groups_check(int T, const int32_t* d_T, int T_max, int E, int k, int score, float scale) {
    std::string why;
    if (!router_shape_ok(T_max, E, k, &why)) return api_fail(ET_ERR_UNSUPPORTED, why);
    if (score != ET_SCORE_SOFTMAX && score != ET_SCORE_SIGMOID)
        return api_fail(ET_ERR_INVALID, "score must be ET_SCORE_SOFTMAX or ET_SCORE_SIGMOID");
    if (!std::isfinite(scale)) return api_fail(ET_ERR_INVALID, "scale must be finite");
    if (!d_T && (T < 0 || T > T_max)) return api_fail(ET_ERR_INVALID, "T must be in [0, T_max]");
    return ET_OK;
}

}  // namespace
}  // namespace et

using namespace et;

extern "C" {

size_t et_router_groups_workspace_bytes(int T_max, int E, int k) {
    std::string why;
    return router_shape_ok(T_max, E, k, &why) ? router_layout(E).total : 0;
}

int et_router_groups(const float* logits, const float* bias, const uint8_t* token_mask, int score, int n_groups, int k_groups,
                     int group_best, int renorm, float scale, int32_t* topk_idx, float* topk_w, int32_t* expert_counts,
                     int32_t* n_routed, float* mean_prob, float* loss, int T, const int32_t* d_T, int T_max, int E, int k,
                     void* workspace, size_t workspace_bytes, void* stream) {
    return api_entry([&]() -> int {
        int rc = groups_check(T, d_T, T_max, E, k, score, scale);
        if (rc) return rc;
        if (n_groups < 1 || n_groups > kGroupsMax || E % n_groups)
            return api_fail(ET_ERR_UNSUPPORTED, "n_groups must be in [1, 32] and divide E");
        if (k_groups < 1 || k_groups > n_groups || k > E / n_groups * k_groups)
            return api_fail(ET_ERR_UNSUPPORTED, "k_groups must be in [1, n_groups] and its experts at least k");
        if (group_best < 1 || group_best > 2) return api_fail(ET_ERR_UNSUPPORTED, "group_best must be 1 or 2");
        if (!logits || !topk_idx || !topk_w)
            return api_fail(ET_ERR_INVALID, "logits, topk_idx and topk_w must be non-NULL");
        const void* need4[] = {logits, bias, topk_idx, topk_w, expert_counts, n_routed, mean_prob, loss, d_T};
        for (const void* q : need4)
            if (!api_aligned(q, 4)) return api_fail(ET_ERR_INVALID, "tensors must be aligned to their element size");
        const RouterLayout L = router_layout(E);
        if ((rc = api_check_ws(workspace, workspace_bytes, L.total))) return rc;
        int dev = 0, sms = 0;
        if ((rc = api_device(&dev, &sms))) return rc;
        const int epl = E <= 32 ? 1 : E <= 64 ? 2 : E <= 128 ? 4 : 8, gs = E / n_groups;
        const int lanes = gs % epl ? 0 : gs / epl;
        const GroupArgs a{logits, bias, token_mask, topk_idx, topk_w, d_T, T, T_max, E, k, n_groups, k_groups, group_best, gs,
                          lanes & (lanes - 1) ? 0 : lanes, renorm != 0, E % 4 == 0 && api_aligned(logits, 16), scale,
                          router_sums_args(workspace, L, expert_counts, n_routed, mean_prob, loss, false)};
        const RouterGrid g = router_grid(d_T ? T_max : T > 0 ? T : 1, E);
        auto pick = [&](auto one, auto two, auto four, auto eight) { return epl == 1 ? one : epl == 2 ? two : epl == 4 ? four : eight; };
        auto kernel = score == ET_SCORE_SIGMOID
            ? pick(router_groups_kernel<1, true>, router_groups_kernel<2, true>, router_groups_kernel<4, true>, router_groups_kernel<8, true>)
            : pick(router_groups_kernel<1, false>, router_groups_kernel<2, false>, router_groups_kernel<4, false>, router_groups_kernel<8, false>);
        const cudaError_t e = api_launch(kernel, g.ctas, g.warps * 32, g.smem, stream, a);
        if (e != cudaSuccess) return api_fail_cuda(e, "launch of the grouped router kernel");
        return ET_OK;
    });
}

int et_router_groups_bwd(const float* logits, const uint8_t* token_mask, int score, int renorm, float scale,
                         const int32_t* topk_idx, const float* topk_w, const int32_t* expert_counts, const int32_t* n_routed,
                         const float* d_loss, const float* d_topk_w, float* d_logits, int T, const int32_t* d_T, int T_max,
                         int E, int k, void* workspace, size_t workspace_bytes, void* stream) {
    return api_entry([&]() -> int {
        int rc = groups_check(T, d_T, T_max, E, k, score, scale);
        if (rc) return rc;
        if (!logits || !topk_idx || !topk_w || !expert_counts || !n_routed || !d_logits)
            return api_fail(ET_ERR_INVALID, "logits, topk_idx, topk_w, expert_counts, n_routed and d_logits "
                                            "must be non-NULL");
        const void* need4[] = {logits, topk_idx, topk_w, expert_counts, n_routed, d_loss, d_topk_w, d_logits, d_T};
        for (const void* q : need4)
            if (!api_aligned(q, 4)) return api_fail(ET_ERR_INVALID, "tensors must be aligned to their element size");
        if ((rc = api_check_ws(workspace, workspace_bytes, kHeaderBytes))) return rc;
        if (!d_T && T == 0) return ET_OK;
        int dev = 0, sms = 0;
        if ((rc = api_device(&dev, &sms))) return rc;
        const GroupBwdArgs a{logits, token_mask, topk_idx, topk_w, expert_counts, n_routed, d_loss, d_topk_w, d_logits, d_T,
                             T, T_max, E, k, score == ET_SCORE_SIGMOID, renorm != 0, scale != 0.0f ? 1.0f / scale : 0.0f,
                             static_cast<EtHeader*>(workspace)};
        const int rows = d_T ? T_max : T;
        int grid = ceil_div_i(rows, 8);
        grid = grid < 8 * sms ? grid : 8 * sms;
        auto kernel = E <= 32 ? router_groups_bwd_kernel<1> : E <= 64 ? router_groups_bwd_kernel<2>
                    : E <= 128 ? router_groups_bwd_kernel<4> : router_groups_bwd_kernel<8>;
        const cudaError_t e = api_launch(kernel, grid, 256, 0, stream, a);
        if (e != cudaSuccess) return api_fail_cuda(e, "launch of the grouped router's backward kernel");
        return ET_OK;
    });
}

}  // extern "C"
