// router_groups.cu -- the router with scores by softmax or sigmoid, a bias that
// only the choice sees, and groups of experts of which the best take part; its
// balance loss, and the gradient.
#include <cmath>

#include "../../include/etmoe.h"
#include "router_rows.h"

namespace et {
namespace {

// One row a warp, experts lane * EPL + i in register i, so that a group is a few
// neighbouring lanes.  The choice runs on 32-bit values: without a bias on the logits,
// which order as the scores do and are exact; with one on score + bias, whose error has a
// bound.  Keys are cut by the bits that name their experts, sorted in each lane and merged
// over the warp, a list of eight and its neighbour's at a time.  Then the chosen are looked
// at with their whole values: where two neighbours in the order are no farther apart than
// both errors, where more than k experts are above the k-th less both errors (those that
// equal it apart), or the last group that takes part and the next than theirs, 64 bits
// decide: on the candidates alone (a lane each: 1.3 us where a whole row takes 14), and on
// the whole row if they are too many.
//
// The form for few rows, and for E and groups that eight lanes cannot share
// (router_rows4_kernel has the others).  Bound by a row's latency, T = 16, E = 128 6.0 us, then
// by instruction issue, about 1080 a row at E = 256 (with 64 registers for 32 warps a CTA, of
// which E > 64 spills 80 to 384 bytes a thread).  Groups that are no power of two of lanes are
// looked at one by one (T = 16384, E = 160 in 8 groups took 43 us this way; E = 60 in 5 21.6).
template <int EPL, bool SIGMOID, bool BIAS>
__global__ void __launch_bounds__(kRouterWarpsMax * 32) router_groups_kernel(const GroupArgs p) {
    constexpr uint32_t kAll = 0xffffffffu, kLow = 32 * EPL - 1;  // the bits that name an expert
    constexpr float kU = 1.0f / (1 << 24);
    extern __shared__ __align__(16) float sm[];  // [warps][E], then the last CTA's sums
    __shared__ RouterShared sh;
    __shared__ uint32_t chosen[kRouterWarpsMax][kCandidates];
    __shared__ __align__(16) float bias_s[kRouterEMax];
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
        bias_s[e] = BIAS && e < E ? p.bias[e] : 0.0f;
    }
    float* const big = sm + warp * E + e0;  // this lane's sums of whole batches of 32 rows
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (e0 + i < E) big[i] = 0.0f;
    __syncthreads();

    const int my_group = p.lanes ? lane / p.lanes : lane;  // whose numbers this lane has
    uint32_t group_of[(EPL + 3) / 4] = {};  // a byte an expert, where a group is not whole lanes
    if (p.kg < p.G && !p.lanes)
#pragma unroll
        for (int i = 0; i < EPL; ++i) group_of[i / 4] |= static_cast<uint32_t>((e0 + i) / p.gs & 31) << (8 * (i % 4));

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

        // What ranks an expert: with a bias score + bias, else the logit.
        const float* row = p.logits + static_cast<size_t>(t) * E;
        uint32_t key[EPL];  // kNegInfKey: not available; 0: in a group that takes no part
        {
            float b[EPL];
            if (BIAS && EPL >= 4) {
#pragma unroll
                for (int i = 0; i < EPL; i += 4) {
                    const float4 q = *reinterpret_cast<const float4*>(bias_s + e0 + i);
                    b[i] = q.x;
                    b[(i + 1) % EPL] = q.y;
                    b[(i + 2) % EPL] = q.z;
                    b[(i + 3) % EPL] = q.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < EPL; ++i) b[i] = bias_s[e0 + i];
            }
#pragma unroll
            for (int i = 0; i < EPL; ++i) key[i] = BIAS ? sum_key(v[i] == -INFINITY ? v[i] : __fadd_rn(s[i], b[i])) : logit_key(v[i]);
        }
        bool again = false;  // the whole row in 64 bits
        if (p.kg < p.G) {
            // a group's best two, by score + bias: of this lane's group, or (where groups are not
            // whole lanes, or not a power of two of them) of group number `lane`
            uint32_t hi = 0, lo = 0;
            auto score_of = [&](int i) -> uint32_t { return BIAS || key[i] <= kNegInfKey ? key[i] : score_key(s[i]); };
            if (p.lanes) {
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const uint32_t c = score_of(i);
                    lo = max(lo, min(hi, c));
                    hi = max(hi, c);
                }
                for (int off = 1; off < p.lanes; off <<= 1) {
                    const uint32_t h = __shfl_xor_sync(kAll, hi, off), l = __shfl_xor_sync(kAll, lo, off);
                    lo = max(max(lo, l), min(hi, h));
                    hi = max(hi, h);
                }
            } else {
#pragma unroll 1
                for (int g = 0; g < p.G; ++g) {
                    uint32_t h = 0, l = 0;
#pragma unroll
                    for (int i = 0; i < EPL; ++i) {
                        const uint32_t c = e0 + i >= g * p.gs && e0 + i < g * p.gs + p.gs ? score_of(i) : 0u;
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
            const int wide = p.lanes ? p.lanes : 1;  // lanes that hold a group's numbers
            const bool group = my_group < p.G;
            float score = -INFINITY, off_by = 0.0f;
            if (group) {
                const float h = key_or_none(hi), l = p.best > 1 && lo > kNegInfKey ? key_logit(lo) : 0.0f;
                score = h + l;
                if (!(h == -INFINITY)) off_by = 2.0f * err + 2.0f * kU * (fabsf(h) + fabsf(l));
            }
            const uint32_t mine = logit_key(score);
            int rank = 0;
#pragma unroll 4
            for (int g = 0; g < p.G; ++g) {
                const uint32_t other = __shfl_sync(kAll, mine, g * wide);
                rank += other > mine || (other == mine && g < my_group);
            }
            // the last that takes part and the next: apart by more than any two may be off
            const int la = __ffs(__ballot_sync(kAll, group && rank == p.kg - 1)) - 1;
            const int lb = __ffs(__ballot_sync(kAll, group && rank == p.kg)) - 1;
            const float a = __shfl_sync(kAll, score, la), b = __shfl_sync(kAll, score, lb);
            const float tol = 2.0f * __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(off_by)));
            bool part = group && rank < p.kg;
            bool close = masked_in && !(a - b > tol) && !(b == -INFINITY);
            if (close) {  // but for a row of equal logits and biases (an untrained router's): the order is the experts'
                bool flat = true;
#pragma unroll
                for (int i = 0; i < EPL; ++i) flat = flat && (e0 + i >= E || (v[i] == row[0] && (!BIAS || bias_s[e0 + i] == bias_s[0])));
                close = !__all_sync(kAll, flat);
            }
            if (close) {
                // between these two alone?
                const bool other = group && !(rank < p.kg - 1 ? score - b > tol : rank > p.kg ? a - score > tol : true);
                const bool others = __any_sync(kAll, other);
                again = !(tol < 1.0f) || others;
                if (!again) {
                    const bool two = p.best > 1 && lo > kNegInfKey;
                    const float floor = key_or_none(two ? lo : hi) - tol;  // the last that counts
                    const double Z = !SIGMOID && BIAS ? softmax_sum64(row, top, E, lane) : 0.0;
                    const int r = compare_groups<EPL>(row, bias_s, SIGMOID, top, inv, Z, E, p.gs, la / wide, lb / wide,
                                                      __shfl_sync(kAll, floor, la), __shfl_sync(kAll, floor, lb),
                                                      __shfl_sync(kAll, two ? 2 : 1, la), __shfl_sync(kAll, two ? 2 : 1, lb),
                                                      chosen[warp], lane);
                    again = r < 0;
                    if (r == 0 && group && (rank == p.kg - 1 || rank == p.kg)) part = rank == p.kg;
                    __syncwarp();
                }
            }
            if (p.lanes) {
#pragma unroll
                for (int i = 0; i < EPL; ++i) key[i] = part ? key[i] : 0u;
            } else {
                const uint32_t in = __ballot_sync(kAll, part);
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (!(in >> (group_of[i / 4] >> (8 * (i % 4)) & 31) & 1)) key[i] = 0u;
            }
        }

        // the best k by their keys, cut to name the expert, lower experts larger; lane j: the j-th
        uint32_t best[8];
        {
            uint32_t cut[EPL];
#pragma unroll
            for (int i = 0; i < EPL; ++i) cut[i] = (key[i] & ~kLow) | (kLow - (e0 + i));
            sort_keys<EPL>(cut);
#pragma unroll
            for (int i = 0; i < 8; ++i) best[i] = i < EPL ? cut[i % EPL] : 0u;
            merge8<EPL, 32>(best);
        }
        uint32_t mykey = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (lane == j) mykey = best[j];
        bool on = lane < k && mykey > kNegInfKey;
        int myE = static_cast<int>(kLow - (mykey & kLow));
        float myL = on ? row[myE] : -INFINITY;
        {
            const float b = BIAS && on ? bias_s[myE] : 0.0f;
            const float c = !on ? -INFINITY : !BIAS ? myL : __fadd_rn(SIGMOID ? sigmoid_fast(myL) : __expf(myL - top) * inv, b);
            const float cn = __shfl_down_sync(kAll, c, 1), Ln = __shfl_down_sync(kAll, myL, 1);
            const float bn = BIAS ? __shfl_down_sync(kAll, b, 1) : 0.0f;
            const int onn = __shfl_down_sync(kAll, static_cast<int>(on), 1);
            const bool pair = on && lane < k - 1 && onn;
            // (one that equals its neighbour comes in the order of the experts already)
            const float tol = BIAS ? 2.0f * err + kU * (fabsf(c) + fabsf(cn)) : same_score<SIGMOID>(cn, top);
            // (without a bias, sigmoid scores of logits above kSigmoidOne may be equal: near 1)
            constexpr bool kOne = SIGMOID && !BIAS;
            bool doubt = pair && !(b == bn && myL == Ln) && (!(c - cn > tol) || (kOne && cn > kSigmoidOne));
            // logits whose scores may be equal in 64 bits near 0, chosen or not
            const bool met = !BIAS && on && (SIGMOID ? myL < -700.0f : myL - top < -700.0f);
            // the least of the chosen, and what may be above it in truth: these experts, and they alone?
            const uint32_t lanes_on = __ballot_sync(kAll, on);
            const float ck = __shfl_sync(kAll, c, k - 1), Lk = __shfl_sync(kAll, myL, k - 1), bk = __shfl_sync(kAll, b, k - 1);
            float cmin = on ? c : INFINITY;
#pragma unroll
            for (int off = 4; off >= 1; off >>= 1) cmin = fminf(cmin, __shfl_xor_sync(kAll, cmin, off));
            cmin = __shfl_sync(kAll, cmin, 0);
            float floor = cmin - (BIAS ? 2.0f * err + 4.0f * kU * fabsf(cmin) : same_score<SIGMOID>(cmin, top));
            if (kOne) floor = fminf(floor, kSigmoidOne);
            int above = 0;
            const uint32_t floor_key = lanes_on >> (k - 1) & 1 ? logit_key(floor) : ~0u;  // else all that are available are chosen
#pragma unroll
            for (int i = 0; i < EPL; ++i) above += key[i] >= floor_key;
            const int n = __reduce_add_sync(kAll, above);
            if (n > k) {
                // as many more as equal the k-th exactly may be: they come behind it
                int ties = 0;
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (key[i] >= floor_key) ties += row[e0 + i] == Lk && (!BIAS || bias_s[e0 + i] == bk);
                const int n_ties = __reduce_add_sync(kAll, ties);
                const int chosen_ties = __popc(__ballot_sync(kAll, on && myL == Lk && b == bk));
                doubt |= n - n_ties != k - chosen_ties || !(ck == cmin);
            } else if (n < k && n > 0) {
                doubt = true;  // (a NaN)
            }
            if (__any_sync(kAll, doubt || met) && !again && masked_in) {
                again = __any_sync(kAll, met) || n > kCandidates || n == 0 || !(err < 1.0f);
                if (!again) {
                    int at = 0;
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < EPL; ++i) {
                        const uint32_t who = __ballot_sync(kAll, key[i] >= floor_key);
                        if (key[i] >= floor_key) chosen[warp][at + __popc(who & below)] = e0 + i;
                        at += __popc(who);
                    }
                    __syncwarp();
                    order_again(row, bias_s, SIGMOID, top, !SIGMOID && BIAS ? softmax_sum64(row, top, E, lane) : 0.0, n, k, chosen[warp], lane);
                    on = lane < k && lane < n;
                    myE = on ? static_cast<int>(chosen[warp][lane & (kCandidates - 1)]) : 0;
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
        __syncwarp();
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
    int renorm;
    float inv_scale;        // 0 where scale is
    EtHeader* hdr;
};

// One row a warp; scores are made again from the logits.  With q = 1 - s (sigmoid) or 1
// (softmax), p = s / sum s and W_j = w_j d_w_j:
//   d_L[e] = q_e (d_loss p_e (C_e - sum C p) + sum_{j: idx_j = e} (W_j - r_j)) - u p_e,
//   r_j = w_j sum W / scale with renorm; u = sum W for softmax without; else 0.
// A token is routed if it has an index that is not -1.
//
// VEC (E a multiple of four, tensors 16-byte aligned): a lane has four neighbours in one
// access.  T = 16384, E = 256: 7.6 us, 4.4 TB/s (11.1 with 4-byte accesses, scores told apart
// at run time, three sums one by one and 8 CTAs an SM); bound by issue slots, 64 % of them,
// and the loads of the first rows.
template <int EPL, bool SIGMOID, bool VEC>
__global__ void __launch_bounds__(256) router_groups_bwd_kernel(const GroupBwdArgs p) {
    constexpr uint32_t kAll = 0xffffffffu;
    constexpr int W4 = VEC ? 4 : 1;
    static_assert(EPL % W4 == 0, "");
    __shared__ __align__(16) float add_s[8][32 * EPL];  // a row's gradients through the gate weights, by expert
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    const int E = p.E, k = p.k;
    grid_begin();
    bool ok;
    const int T = row_count(p.d_T, p.T_host, p.T_max, p.hdr, &ok);
    if (!ok) return;
    auto expert = [&](int i) { return (lane + 32 * (i / W4)) * W4 + i % W4; };  // this lane's i-th
    auto read = [&](const float* from, float (&to)[EPL], float none) {
#pragma unroll
        for (int i = 0; i < EPL; i += W4) {
            if (VEC) {
                float4 q = make_float4(none, none, none, none);
                if (expert(i) < E) q = *reinterpret_cast<const float4*>(from + expert(i));
                to[i] = q.x; to[i + 1 < EPL ? i + 1 : i] = q.y; to[i + 2 < EPL ? i + 2 : i] = q.z; to[i + 3 < EPL ? i + 3 : i] = q.w;
            } else {
                to[i] = expert(i) < E ? from[expert(i)] : none;
            }
        }
    };
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
        const size_t o = static_cast<size_t>(t) * k + lane;
        if (in) read(p.logits + static_cast<size_t>(t) * E, r.v, -INFINITY);
        r.on = in && (!p.mask || p.mask[t] != 0);
        r.e = sel ? p.idx[o] : -1;
        r.w = sel ? p.w[o] : 0.0f;
        r.dw = sel && p.d_w ? p.d_w[o] : 0.0f;
    };
    Row nx{};
    load(t0, nx);
    const int n = *p.n_routed;
    const float rows = n > 0 ? static_cast<float>(n) : 1.0f;
    const float dl = p.d_loss ? *p.d_loss : 0.0f;
    float cost[EPL];  // E counts / (n^2 k): what a unit of p on expert e costs
    const float per = static_cast<float>(E) / (rows * k) / rows;
#pragma unroll
    for (int i = 0; i < EPL; ++i) cost[i] = expert(i) < E ? per * static_cast<float>(p.counts[expert(i)]) : 0.0f;
    for (int t = t0; t < T; t += step) {
        const Row c = nx;
        load(t + step, nx);
        const bool sel = c.e >= 0 && c.e < E;
        const bool any = __any_sync(kAll, c.e >= 0), live = c.on && any;
        float d[EPL];
        if (live) {
            float top = c.v[0];
#pragma unroll
            for (int i = 1; i < EPL; ++i) top = fmaxf(top, c.v[i]);
            // Sigmoid scores that are all tiny: as ratios of e^L, like softmax's.
            const bool ratio = !SIGMOID || __all_sync(kAll, top < -60.0f);
            if (ratio)
#pragma unroll
                for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, off));
            const float W = c.e >= 0 ? c.w * c.dw : 0.0f;
            float s[EPL], q[EPL], sums[3] = {0.0f, 0.0f, W};
            // (-inf: s = 0; NaN: s is NaN.  A row of -inf alone has no index.)
            if (SIGMOID) {
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    const float e = __expf(-fabsf(c.v[i]));  // sigmoid of either sign without overflow
                    const float h = rcp_fast(1.0f + e), lo = e * h;
                    s[i] = c.v[i] < 0.0f ? lo : h;
                    q[i] = c.v[i] < 0.0f ? h : lo;
                }
            }
            if (ratio) {
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    s[i] = c.v[i] == -INFINITY ? 0.0f : __expf(c.v[i] - top);
                }
            }
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                sums[0] += s[i];
                sums[1] += s[i] * cost[i];
            }
            const float mine = warp_sum3(sums);
            const float inv = rcp_fast(__shfl_sync(kAll, mine, 0));
            const float cp = __shfl_sync(kAll, mine, 16) * inv, sum = __shfl_sync(kAll, mine, 8);
            const float u = !p.renorm && !SIGMOID ? sum : 0.0f;
            if (p.d_w) {
                // an index outside [0, E) adds nothing; one that comes twice adds twice
                if (sel) atomicAdd(add + c.e, p.renorm ? W - c.w * p.inv_scale * sum : W);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < EPL; i += W4) {
                    if (VEC) {
                        const float4 a = *reinterpret_cast<const float4*>(add + expert(i));
                        d[i] = a.x; d[i + 1 < EPL ? i + 1 : i] = a.y; d[i + 2 < EPL ? i + 2 : i] = a.z; d[i + 3 < EPL ? i + 3 : i] = a.w;
                    } else {
                        d[i] = add[expert(i)];
                    }
                }
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
                d[i] = dl * pr * (cost[i] - cp) + d[i];
                if (SIGMOID) d[i] *= q[i];
                else d[i] -= u * pr;
            }
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) d[i] = 0.0f;
        }
        float* out = p.d_logits + static_cast<size_t>(t) * E;
#pragma unroll
        for (int i = 0; i < EPL; i += W4)
            if (expert(i) < E) {
                if (VEC) *reinterpret_cast<float4*>(out + expert(i)) = make_float4(d[i], d[i + 1 < EPL ? i + 1 : i], d[i + 2 < EPL ? i + 2 : i], d[i + 3 < EPL ? i + 3 : i]);
                else out[expert(i)] = d[i];
            }
    }
}

template <int EPL, bool VEC>
auto pick_bwd(bool sigmoid) {
    return sigmoid ? router_groups_bwd_kernel<EPL, true, VEC> : router_groups_bwd_kernel<EPL, false, VEC>;
}

template <int EPL>
auto pick_groups(bool sigmoid, bool bias) {
    return sigmoid ? (bias ? router_groups_kernel<EPL, true, true> : router_groups_kernel<EPL, true, false>)
                   : (bias ? router_groups_kernel<EPL, false, true> : router_groups_kernel<EPL, false, false>);
}

// Rows from which on four share a warp, where eight lanes can share a row's experts.  Sigmoid
// with bias, E = 256, 8 groups: T = 608 14.2 us one a warp and 14.2 four a warp, T = 1024 16.0
// and 13.2, T = 2048 16.1 and 16.0, T = 4096 19.6 and 15.3, T = 16384 33 and 25, T = 65536 82
// and 59; E = 64: T = 608 7.8 and 7.7, T = 16384 19 and 13, T = 65536 51 and 28.
constexpr int kRows4Least = 1024;

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
        const bool sig = score == ET_SCORE_SIGMOID;
        const int rows = d_T ? T_max : T > 0 ? T : 1;
        if (rows >= kRows4Least && rows4_serves(E, n_groups)) {
            const cudaError_t e = launch_router_rows4(a, sig, rows, dev, stream);
            if (e != cudaSuccess) return api_fail_cuda(e, "launch of the grouped router kernel");
            return ET_OK;
        }
        // One CTA up to 16 rows, then few warps a CTA while that puts rows on more SMs.
        const int warps = rows <= 16 ? rows : rows <= 8 * kRouterParts ? 8 : rows <= 16 * kRouterParts ? 16 : kRouterWarpsMax;
        const RouterGrid g = router_grid_of(rows, E, warps);
        auto kernel = epl == 1 ? pick_groups<1>(sig, bias) : epl == 2 ? pick_groups<2>(sig, bias)
                    : epl == 4 ? pick_groups<4>(sig, bias) : pick_groups<8>(sig, bias);
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
                             T, T_max, E, k, renorm != 0, scale != 0.0f ? 1.0f / scale : 0.0f,
                             static_cast<EtHeader*>(workspace)};
        const int rows = d_T ? T_max : T;
        // With 8 experts a lane as many CTAs as find room at once, which then hide a row's loads
        // behind the one before it (T = 16384, E = 256: 7.6 us, with 8 an SM 8.8); with fewer,
        // rows are short and more CTAs hide more (E = 128: 5.8 us, with 3 7.7).
        const int most = (E > 128 ? 3 : 8) * sms;
        int grid = ceil_div_i(rows, 8);
        grid = grid < most ? grid : most;
        const bool sig = score == ET_SCORE_SIGMOID, vec = E > 64 && E % 4 == 0 && api_aligned(logits, 16) && api_aligned(d_logits, 16);
        auto kernel = E <= 32 ? pick_bwd<1, false>(sig) : E <= 64 ? pick_bwd<2, false>(sig)
                    : E <= 128 ? (vec ? pick_bwd<4, true>(sig) : pick_bwd<4, false>(sig))
                               : (vec ? pick_bwd<8, true>(sig) : pick_bwd<8, false>(sig));
        const cudaError_t e = api_launch(kernel, grid, 256, 0, stream, a);
        if (e != cudaSuccess) return api_fail_cuda(e, "launch of the grouped router's backward kernel");
        return ET_OK;
    });
}

}  // extern "C"
