// router_choice.cuh -- the grouped router's choice: its arguments, sorted lists of keys, and
// what decides in 64 bits where 32 cannot tell.  Shared by its forms.
#pragma once

#include "router_sums.cuh"

namespace et {
namespace {

constexpr int kGroupsMax = 32;

}  // namespace

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

namespace {

__device__ __forceinline__ double key_value(unsigned long long key) {
    return __longlong_as_double(static_cast<long long>(key >> 63 ? key ^ 0x8000000000000000ull : ~key));
}

// logit_key of a 64-bit value; NaN above all, > 0 everywhere.
__device__ __forceinline__ unsigned long long value_key(double v) {
    if (v != v) return ~0ull;
    const long long b = __double_as_longlong(v + 0.0);
    return static_cast<unsigned long long>(b) ^ (static_cast<unsigned long long>(b >> 63) | 0x8000000000000000ull);
}

// What ranks experts and groups in 64 bits, everywhere (equal ones tie): scores + bias, softmax
// scores by their row's sum Z of e^(x - top); Z = 0: softmax scores without a bias, as their
// multiples e^(x - top).
__device__ __forceinline__ double value64(float x, float b, bool sigmoid, float top, double Z) {
    const double e = exp(sigmoid ? -static_cast<double>(x) : static_cast<double>(x) - static_cast<double>(top));
    return sigmoid ? 1.0 / (1.0 + e) + static_cast<double>(b) : Z == 0.0 ? e : e / Z + static_cast<double>(b);
}

// The sum of e^(x - top) over a row, in 64 bits, by the warp.
__device__ __noinline__ double softmax_sum64(const float* row, float top, int E, int lane) {
    double Z = 0.0;
#pragma unroll 1
    for (int e = lane; e < E; e += 32) Z += exp(static_cast<double>(row[e]) - static_cast<double>(top));
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) Z += __shfl_xor_sync(0xffffffffu, Z, off);
    return Z;
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
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = lane * EPL + i < E ? row[lane * EPL + i] : -INFINITY;
    if (!sigmoid) {
        top = v[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) top = fmaxf(top, v[i]);
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, off));
    }
    const double Z = !sigmoid && bias ? softmax_sum64(row, top, E, lane) : 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        key[i] = 0;
        if (!(v[i] == -INFINITY)) {
            const double c = value64(v[i], bias ? bias[lane * EPL + i] : 0.0f, sigmoid, top, Z);
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

__device__ __forceinline__ void order2(uint32_t& a, uint32_t& b) {  // the larger first
    const uint32_t hi = max(a, b);
    b = min(a, b);
    a = hi;
}

// Sorts k[0 .. N), first rising and then falling (or the other way), the largest first.
template <int N>
__device__ __forceinline__ void sort_bitonic(uint32_t* k) {
#pragma unroll
    for (int h = N / 2; h >= 1; h /= 2)
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (!(i & h)) order2(k[i], k[i + h]);
}

// The larger first, of N.
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t* k) {
    if (N == 2) order2(k[0], k[1]);
    if (N >= 4) {  // odd-even merge sort
#pragma unroll
        for (int o = 0; o < N; o += 4) {
            order2(k[o], k[o + 1]); order2(k[o + 2], k[o + 3]);
            order2(k[o], k[o + 2]); order2(k[o + 1], k[o + 3]);
            order2(k[o + 1], k[o + 2]);
        }
    }
    if (N == 8) {
        order2(k[0], k[4]); order2(k[1], k[5]); order2(k[2], k[6]); order2(k[3], k[7]);
        order2(k[2], k[4]); order2(k[3], k[5]);
        order2(k[1], k[2]); order2(k[3], k[4]); order2(k[5], k[6]);
    }
}

// The eight largest keys of LANES neighbouring lanes, sorted, in each of them; a lane has
// min(N, 8) to begin with, sorted, zeros behind them.  With a neighbour's list, turned round:
// the larger of each pair are the larger half of both lists.  Short lists grow to eight first.
template <int N, int LANES>
__device__ __forceinline__ void merge8(uint32_t (&k)[8]) {
    constexpr uint32_t kAll = 0xffffffffu;
    int n = N < 8 ? N : 8;
#pragma unroll
    for (int off = 1; off < LANES; off <<= 1) {
        if (n < 8) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) {
                    const uint32_t other = __shfl_xor_sync(kAll, k[n - 1 - i], off);
                    k[8 - 1 - i] = other;  // parked
                }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) {
                    const uint32_t other = k[8 - 1 - i];
                    const uint32_t hi = max(k[i], other), lo = min(k[i], other);
                    k[i] = hi;
                    k[8 - 1 - i] = lo;
                }
            uint32_t low[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) low[i] = k[8 - 1 - i];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) k[n + i] = low[i];
            if (n == 2) { sort_bitonic<2>(k); sort_bitonic<2>(k + 2); }
            if (n == 4) { sort_bitonic<4>(k); sort_bitonic<4>(k + 4); }
            n *= 2;
        } else {
            uint32_t other[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) other[i] = __shfl_xor_sync(kAll, k[7 - i], off);
#pragma unroll
            for (int i = 0; i < 8; ++i) k[i] = max(k[i], other[i]);
            sort_bitonic<8>(k);
        }
    }
}

// logit_key of a sum score + bias, which is never -0 and no NaN but the positive one.
__device__ __forceinline__ uint32_t sum_key(float v) {
    const int b = __float_as_int(v);
    return static_cast<uint32_t>(b ^ ((b >> 31) | static_cast<int>(0x80000000u)));
}

constexpr int kCandidates = 16;  // experts whose order is looked at again at most

// Without a bias 32 bits compare logits, which are exact.  Logits this far below x or less may
// have scores that are equal in 64 bits: a score is off by 2^-51 of itself (exp, an add, a
// quotient), and two of them are (x - y) (1 - s) apart, with 1 - s >= 1/2 below 0; above, floats
// are 2^-24 x apart, which outweighs 1 - s up to x = 20.  (A softmax score: 2^-52 and what x - top
// rounds off, 2^-53 of it.)  So only logits near 0, or far below the row's largest, are that close.
constexpr float kSigmoidOne = 20.0f;
template <bool SIGMOID>
__device__ __forceinline__ float same_score(float x, float top) {
    constexpr float kStep = 1.0f / (1ull << 49);
    return SIGMOID ? kStep : fmaf(top - x, kStep, kStep);
}

// Two groups whose scores 32 bits cannot tell apart: 1 if the first has the larger, or the
// same and the lower number, 0 if the second, -1 if it takes more than their best two to
// say.  floor_a, floor_b: what the experts that count are not below;
// want_a, want_b: how many those are.  slots: 16 places of shared memory.
template <int EPL>
__device__ __noinline__ int compare_groups(const float* row, const float* bias_s, bool sigmoid, float top, float inv, double Z, int E,
                                           int gs, int a, int b, float floor_a, float floor_b, int want_a, int want_b, uint32_t* slots, int lane) {
    constexpr uint32_t kAll = 0xffffffffu;
    int na = 0, nb = 0;
#pragma unroll 1
    for (int i = 0; i < EPL; ++i) {
        const int e = lane * EPL + i, g = e / gs;
        const float x = e < E ? row[e] : -INFINITY;
        const float c = x == -INFINITY ? x : __fadd_rn(sigmoid ? sigmoid_fast(x) : __expf(x - top) * inv, bias_s[min(e, E - 1)]);
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
    double c = mine ? value64(row[e], bias_s[e], sigmoid, top, Z) : 0.0;
    c += __shfl_xor_sync(kAll, c, 1);  // two at most
    const double sa = __shfl_sync(kAll, c, 0), sb = __shfl_sync(kAll, c, 8);
    return sa > sb || (sa == sb && a < b) ? 1 : 0;
}

// The order of n candidates (n <= kCandidates, their experts in slots) in 64 bits: puts the
// best k there in their order.
__device__ __noinline__ void order_again(const float* row, const float* bias_s, bool sigmoid, float top, double Z, int n, int k, uint32_t* slots,
                                         int lane) {
    constexpr uint32_t kAll = 0xffffffffu;
    const int e = lane < n ? static_cast<int>(slots[lane]) : 0;
    const double c = lane < n ? value64(row[e], bias_s[e], sigmoid, top, Z) : 0.0;
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

}  // namespace
}  // namespace et
