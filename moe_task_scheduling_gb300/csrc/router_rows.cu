// router_rows.cu -- the grouped router's forward for many rows, four a warp.
#include <type_traits>

#include "router_rows.h"

namespace et {
namespace {

constexpr int kRows4Warps = 16;  // of a CTA

// Floats of dynamic shared memory: [warps][E] sums of batches, then [warps][4][E] of rows.
__host__ __device__ constexpr int rows4_floats(int E) { return kRows4Warps * 5 * E; }

// For E a multiple of 32 and groups of a power of two in number.
//
// Eight lanes have a row, lane l of them experts l N .. l N + N - 1 (E = 8 N), so four rows
// share each instruction of what is a row's and not an expert's: the eight places of the
// chosen, ranks of groups, doubts, weights.  The choice and its doubts are those of
// router_groups_kernel; the warp comes together for a row that 64 bits decide.  A row's
// probabilities are added up in shared memory, each lane its own places: in registers they
// would take 32 more of them.
//
// Bound by instructions and their latency: about 500 a row at E = 256 where one row a warp
// takes 1080, 16 warps an SM with 128 registers (12 with 168 were slower from T = 1024 to
// 16384 by 5 to 20 %).  With 128 the forms for E = 192 and more spill, sigmoid with a bias at
// E = 256 the most (360 bytes out, 416 in, a thread), and 36 % of the issue slots are used: no
// limit of the chip's is reached.  T = 16384, E = 256, sigmoid with bias, 8 groups, k = 8 25-28
// us, 8 of them fixed (launch, the sums over CTAs); T = 65536 59-63 us; E = 160 19 and E = 128
// 17 us.
template <int N, bool SIGMOID, bool BIAS>
__global__ void __launch_bounds__(kRows4Warps * 32, 1) router_rows4_kernel(const GroupArgs p) {
    constexpr uint32_t kAll = 0xffffffffu;
    constexpr int E = 8 * N;
    constexpr uint32_t kLow = E <= 32 ? 31 : E <= 64 ? 63 : E <= 128 ? 127 : 255;  // the bits that name an expert
    constexpr float kU = 1.0f / (1 << 24);
    constexpr int N8 = N < 8 ? N : 8;
    extern __shared__ __align__(16) float sm[];
    __shared__ RouterShared sh;
    __shared__ uint32_t slots_s[kRows4Warps][4][kCandidates];
    __shared__ __align__(16) float bias_s[kRouterEMax], bias_q[kRouterEMax];  // by expert; as the lanes read it
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane >> 3, l8 = lane & 7, seg = lane & 24, e0 = l8 * N;
    const int k = p.k, G = p.G;
    uint32_t(*const slots)[kCandidates] = slots_s[warp];
    grid_begin();
    bool ok;
    const int T = row_count(p.d_T, p.T_host, p.T_max, p.sums.hdr, &ok);
    if (!ok) return;
    for (int e = threadIdx.x; e < kRouterEMax; e += blockDim.x) {
        const float b = BIAS && e < E ? p.bias[e] : 0.0f;
        sh.hist[e] = 0;
        bias_s[e] = b;
        if (e < E) bias_q[((e % N) / 4 * 8 + e / N) * 4 + e % 4] = b;
    }
    for (int i = threadIdx.x; i < rows4_floats(E); i += blockDim.x) sm[i] = 0.0f;
    __syncthreads();
    float* const big = sm + warp * E;
    float* const acc_w = sm + kRows4Warps * E + warp * 4 * E;  // [4][N / 4][8 lanes][4]
    float4* const acc = reinterpret_cast<float4*>(acc_w) + r * (E / 4) + l8;

    auto sum8 = [&](float v) {
#pragma unroll
        for (int off = 4; off >= 1; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
        return v;
    };
    auto max8 = [&](float v) {
#pragma unroll
        for (int off = 4; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, off));
        return v;
    };
    auto of_row = [&](uint32_t ballot) { return ballot >> seg & 0xffu; };
    auto load = [&](const float* row, bool have, float (&v)[N]) {
        if (p.vec) {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                if (have) q = *reinterpret_cast<const float4*>(row + e0 + i);
                v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = have ? row[e0 + i] : -INFINITY;
        }
    };

    const int t0 = (blockIdx.x + gridDim.x * warp) * 4, step = gridDim.x * kRows4Warps * 4;
    int accn = 0, rounds = 0;
    for (int tb = t0; tb < T; tb += step) {
        const int t = tb + r;
        const bool have = t < T;
        const float* row = p.logits + static_cast<size_t>(t) * E;
        const bool masked_in = have && (!p.mask || p.mask[t] != 0);
        if (t + step < T) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + static_cast<size_t>(step) * E + e0));
        uint32_t key[N];  // kNegInfKey: not available; 0: in a group that takes no part
        float top = 0.0f, S = 0.0f, inv, err;
        float s[N];
        {
            float v[N];
            load(row, have, v);
            if (!SIGMOID) {
                top = v[0];
#pragma unroll
                for (int i = 1; i < N; ++i) top = fmaxf(top, v[i]);
                top = max8(top);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                s[i] = SIGMOID ? sigmoid_fast(v[i]) : v[i] == -INFINITY ? 0.0f : __expf(v[i] - top);
                S += s[i];
            }
            S = sum8(S);
            inv = __fdividef(1.0f, S);
            if (!SIGMOID) {
#pragma unroll
                for (int i = 0; i < N; ++i) s[i] *= inv;
            }
            // (the errors of router_groups_kernel)
            err = (SIGMOID ? 10.0f : 48.0f * inv) * kU;
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                float4 b = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (BIAS) b = reinterpret_cast<const float4*>(bias_q)[i / 4 * 8 + l8];
                const float bb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    key[i + j] = BIAS ? sum_key(v[i + j] == -INFINITY ? v[i + j] : __fadd_rn(s[i + j], bb[j])) : logit_key(v[i + j]);
            }
        }
        uint32_t top_key = key[0];
#pragma unroll
        for (int i = 1; i < N; ++i) top_key = max(top_key, key[i]);
        // Routed: not masked, and an expert is available (then some group that takes part has one).
        const bool available = of_row(__ballot_sync(kAll, top_key > kNegInfKey)) != 0;
        const bool live = masked_in && available;
        accn += __popc(__ballot_sync(kAll, live) & 0x01010101u);
        const bool tiny = SIGMOID && live && !(S >= 1e-24f) && S == S;  // all below e^-55: their ratios
        if (live && !tiny) {
            const float q = SIGMOID ? inv : 1.0f;
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                float4 a = acc[i * 2];
                a.x += s[i] * q; a.y += s[i + 1] * q; a.z += s[i + 2] * q; a.w += s[i + 3] * q;
                acc[i * 2] = a;
            }
        }
        if (SIGMOID && __any_sync(kAll, tiny)) {
            float v[N];
            load(row, have, v);
            float m = v[0], q = 0.0f;
#pragma unroll
            for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
            m = max8(m);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                v[i] = v[i] == -INFINITY ? 0.0f : __expf(v[i] - m);
                q += v[i];
            }
            q = __fdividef(1.0f, sum8(q));
            if (tiny) {
#pragma unroll
                for (int i = 0; i < N; i += 4) {
                    float4 a = acc[i * 2];
                    a.x += v[i] * q; a.y += v[i + 1] * q; a.z += v[i + 2] * q; a.w += v[i + 3] * q;
                    acc[i * 2] = a;
                }
            }
        }

        bool again = false;  // the whole row in 64 bits
        if (p.kg < G) {
            // M groups a lane (their best two by score + bias), or a group in 8 / G lanes
            auto groups = [&](auto m_) {
                constexpr int M = decltype(m_)::value;
                const int L = M > 1 ? 1 : 8 / G;  // lanes a group
                uint32_t hi[M] = {}, lo[M] = {};
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int m = i / (N / M);
                    const uint32_t c = BIAS || key[i] <= kNegInfKey ? key[i] : score_key(s[i]);
                    lo[m] = max(lo[m], min(hi[m], c));
                    hi[m] = max(hi[m], c);
                }
                if (M == 1)
                    for (int off = 1; off < L; off <<= 1) {
                        const uint32_t h = __shfl_xor_sync(kAll, hi[0], off), l = __shfl_xor_sync(kAll, lo[0], off);
                        lo[0] = max(max(lo[0], l), min(hi[0], h));
                        hi[0] = max(hi[0], h);
                    }
                float score[M], off_by = 0.0f;
                uint32_t mine[M];
                int rank[M];
                bool two[M];
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    two[m] = p.best > 1 && lo[m] > kNegInfKey;
                    const float h = key_or_none(hi[m]), l = two[m] ? key_logit(lo[m]) : 0.0f;
                    score[m] = h + l;
                    if (!(h == -INFINITY)) off_by = fmaxf(off_by, 2.0f * err + 2.0f * kU * (fabsf(h) + fabsf(l)));
                    if (score[m] != score[m]) off_by = score[m];
                    mine[m] = logit_key(score[m]);
                    rank[m] = 0;
                }
                const int group0 = M > 1 ? l8 * M : l8 / L;  // this lane's first group
#pragma unroll 2
                for (int g = 0; g < G; g += M) {
#pragma unroll
                    for (int o = 0; o < M; ++o) {
                        const uint32_t other = __shfl_sync(kAll, mine[o], M > 1 ? g / M : g * L, 8);
#pragma unroll
                        for (int m = 0; m < M; ++m) rank[m] += other > mine[m] || (other == mine[m] && g + o < group0 + m);
                    }
                }
                // the last that takes part and the next: apart by more than any two may be off
                float a = 0.0f, b = 0.0f;
                int ga = 0, gb = 0;
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    const uint32_t wa = of_row(__ballot_sync(kAll, rank[m] == p.kg - 1)), wb = of_row(__ballot_sync(kAll, rank[m] == p.kg));
                    const int la = __ffs(wa) - 1, lb = __ffs(wb) - 1;
                    const float sa = __shfl_sync(kAll, score[m], max(la, 0), 8), sb = __shfl_sync(kAll, score[m], max(lb, 0), 8);
                    if (la >= 0) { a = sa; ga = M > 1 ? la * M + m : la / L; }
                    if (lb >= 0) { b = sb; gb = M > 1 ? lb * M + m : lb / L; }
                }
                uint32_t off_bits = __float_as_uint(off_by);  // (a NaN is above all)
#pragma unroll
                for (int off = 4; off >= 1; off >>= 1) off_bits = max(off_bits, __shfl_xor_sync(kAll, off_bits, off));
                const float tol = 2.0f * __uint_as_float(off_bits & 0x7fffffffu);
                bool part[M];
#pragma unroll
                for (int m = 0; m < M; ++m) part[m] = rank[m] < p.kg;
                bool close = masked_in && !(a - b > tol) && !(b == -INFINITY);
                if (__any_sync(kAll, close)) {
                    // a row of equal logits and biases (an untrained router's): the order is the experts'
                    float v[N];
                    load(row, have, v);
                    const float first = __shfl_sync(kAll, v[0], 0, 8);
                    bool flat = true;
#pragma unroll
                    for (int i = 0; i < N; ++i) flat = flat && v[i] == first && (!BIAS || bias_s[e0 + i] == bias_s[0]);
                    const uint32_t flat_lanes = of_row(__ballot_sync(kAll, flat));
                    close = close && flat_lanes != 0xffu;
                    bool other = false;
#pragma unroll
                    for (int m = 0; m < M; ++m)
                        other |= rank[m] < p.kg - 1 ? !(score[m] - b > tol) : rank[m] > p.kg && !(a - score[m] > tol);
                    const bool others = of_row(__ballot_sync(kAll, other)) != 0;
                    again = close && (!(tol < 1.0f) || others);
                    // between these two alone: what counts for a group is not below its floor
                    float fa = 0.0f, fb = 0.0f;
                    int na = 1, nb = 1;
#pragma unroll
                    for (int m = 0; m < M; ++m) {
                        const float floor = key_or_none(two[m] ? lo[m] : hi[m]) - tol;
                        const int at_a = M > 1 ? ga / M : ga * L, at_b = M > 1 ? gb / M : gb * L;
                        const float xa = __shfl_sync(kAll, floor, at_a, 8), xb = __shfl_sync(kAll, floor, at_b, 8);
                        const int ya = __shfl_sync(kAll, two[m] ? 2 : 1, at_a, 8), yb = __shfl_sync(kAll, two[m] ? 2 : 1, at_b, 8);
                        if (ga % M == m) { fa = xa; na = ya; }
                        if (gb % M == m) { fb = xb; nb = yb; }
                    }
                    const uint32_t rows = __ballot_sync(kAll, close && !again) & 0x01010101u;
#pragma unroll 1
                    for (int rr = 0; rr < 4; ++rr) {
                        if (!(rows >> (8 * rr) & 1)) continue;
                        const int from = 8 * rr;
                        const float* const its_row = p.logits + static_cast<size_t>(tb + rr) * E;
                        const float its_top = __shfl_sync(kAll, top, from);
                        const double Z = !SIGMOID && BIAS ? softmax_sum64(its_row, its_top, E, lane) : 0.0;
                        const int c = compare_groups<N / 4>(its_row, bias_s, SIGMOID, its_top, __shfl_sync(kAll, inv, from), Z, E, p.gs, __shfl_sync(kAll, ga, from), __shfl_sync(kAll, gb, from),
                                                            __shfl_sync(kAll, fa, from), __shfl_sync(kAll, fb, from), __shfl_sync(kAll, na, from),
                                                            __shfl_sync(kAll, nb, from), slots[rr], lane);
                        if (r == rr) {
                            again = c < 0;
#pragma unroll
                            for (int m = 0; m < M; ++m)
                                if (c == 0 && (rank[m] == p.kg - 1 || rank[m] == p.kg)) part[m] = rank[m] == p.kg;
                        }
                        __syncwarp();
                    }
                }
#pragma unroll
                for (int i = 0; i < N; ++i) key[i] = part[i / (N / M)] ? key[i] : 0u;
            };
            if (G <= 8) groups(std::integral_constant<int, 1>());
            else if (G == 16) groups(std::integral_constant<int, 2>());
            else groups(std::integral_constant<int, 4>());
        }

        // the best k by their keys, cut to name the expert, lower experts larger; lane j: the j-th
        uint32_t best[8];
#pragma unroll
        for (int o = 0; o < N; o += N8) {
            uint32_t list[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) list[i] = o + i < N ? (key[(o + i) % N] & ~kLow) | (kLow - (e0 + o + i)) : 0u;
            sort_keys<N8>(list);
            if (o == 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) best[i] = list[i];
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) best[i] = max(best[i], list[7 - i]);
                sort_bitonic<8>(best);
            }
        }
        merge8<N, 8>(best);
        uint32_t mykey = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (l8 == j) mykey = best[j];
        bool on = l8 < k && mykey > kNegInfKey;
        int myE = static_cast<int>(kLow - (mykey & kLow));
        float myL = on ? row[myE] : -INFINITY;
        {
            const float b = BIAS && on ? bias_s[myE] : 0.0f;
            const float c = !on ? -INFINITY : !BIAS ? myL : __fadd_rn(SIGMOID ? sigmoid_fast(myL) : __expf(myL - top) * inv, b);
            const float cn = __shfl_down_sync(kAll, c, 1, 8), Ln = __shfl_down_sync(kAll, myL, 1, 8);
            const float bn = BIAS ? __shfl_down_sync(kAll, b, 1, 8) : 0.0f;
            const int onn = __shfl_down_sync(kAll, static_cast<int>(on), 1, 8);
            const bool pair = on && l8 < k - 1 && onn;
            // (one that equals its neighbour comes in the order of the experts already)
            const float tol = BIAS ? 2.0f * err + kU * (fabsf(c) + fabsf(cn)) : same_score<SIGMOID>(cn, top);
            // (without a bias, sigmoid scores of logits above kSigmoidOne may be equal: near 1)
            constexpr bool kOne = SIGMOID && !BIAS;
            bool doubt = pair && !(b == bn && myL == Ln) && (!(c - cn > tol) || (kOne && cn > kSigmoidOne));
            // logits whose scores may be equal in 64 bits near 0, chosen or not
            const bool met = !BIAS && on && (SIGMOID ? myL < -700.0f : myL - top < -700.0f);
            // the least of the chosen, and what may be above it in truth: these experts, and they alone?
            const uint32_t lanes_on = of_row(__ballot_sync(kAll, on));
            const float ck = __shfl_sync(kAll, c, k - 1, 8), Lk = __shfl_sync(kAll, myL, k - 1, 8), bk = __shfl_sync(kAll, b, k - 1, 8);
            float cmin = on ? c : INFINITY;
#pragma unroll
            for (int off = 4; off >= 1; off >>= 1) cmin = fminf(cmin, __shfl_xor_sync(kAll, cmin, off));
            float floor = cmin - (BIAS ? 2.0f * err + 4.0f * kU * fabsf(cmin) : same_score<SIGMOID>(cmin, top));
            if (kOne) floor = fminf(floor, kSigmoidOne);
            int above = 0;
            const uint32_t floor_key = lanes_on >> (k - 1) & 1 ? logit_key(floor) : ~0u;  // else all that are available are chosen
#pragma unroll
            for (int i = 0; i < N; ++i) above += key[i] >= floor_key;
            int n = above;
#pragma unroll
            for (int off = 4; off >= 1; off >>= 1) n += __shfl_xor_sync(kAll, n, off);
            if (__any_sync(kAll, n > k)) {
                // as many more as equal the k-th exactly may be: they come behind it
                int ties = 0;
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (n > k && key[i] >= floor_key) ties += row[e0 + i] == Lk && (!BIAS || bias_s[e0 + i] == bk);
#pragma unroll
                for (int off = 4; off >= 1; off >>= 1) ties += __shfl_xor_sync(kAll, ties, off);
                const int chosen_ties = __popc(of_row(__ballot_sync(kAll, on && myL == Lk && b == bk)));
                doubt |= n > k && (n - ties != k - chosen_ties || !(ck == cmin));
            }
            doubt |= n < k && n > 0;  // (a NaN)
            const bool row_met = of_row(__ballot_sync(kAll, met)) != 0;
            const bool any_doubt = of_row(__ballot_sync(kAll, doubt)) != 0;
            const bool row_doubt = masked_in && (any_doubt || row_met);
            const bool whole = row_met || n > kCandidates || n == 0 || !(err < 1.0f);
            const bool few = row_doubt && !again && !whole;
            again |= row_doubt && whole;
            const uint32_t rows = __ballot_sync(kAll, few) & 0x01010101u;
            if (rows) {
                int at = above;  // of the row's lanes before this one
#pragma unroll
                for (int off = 1; off < 8; off <<= 1) {
                    const int o = __shfl_up_sync(kAll, at, off, 8);
                    if (l8 >= off) at += o;
                }
                at -= above;
                __syncwarp();
                if (few) {
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        if (key[i] >= floor_key) slots[r][at++] = e0 + i;
                }
                __syncwarp();
#pragma unroll 1
                for (int rr = 0; rr < 4; ++rr) {
                    if (!(rows >> (8 * rr) & 1)) continue;
                    const float* const its_row = p.logits + static_cast<size_t>(tb + rr) * E;
                    const float its_top = __shfl_sync(kAll, top, 8 * rr);
                    const double Z = !SIGMOID && BIAS ? softmax_sum64(its_row, its_top, E, lane) : 0.0;
                    order_again(its_row, bias_s, SIGMOID, its_top, Z, __shfl_sync(kAll, n, 8 * rr), k, slots[rr], lane);
                }
                if (few) {
                    on = l8 < k && l8 < n;
                    myE = on ? static_cast<int>(slots[r][l8]) : 0;
                    myL = on ? row[myE] : -INFINITY;
                }
                __syncwarp();
            }
        }
        const uint32_t whole_rows = __ballot_sync(kAll, again) & 0x01010101u;
        if (whole_rows) {
#pragma unroll 1
            for (int rr = 0; rr < 4; ++rr) {
                if (!(whole_rows >> (8 * rr) & 1)) continue;
                const int e = choose64<N / 4>(p.logits + static_cast<size_t>(tb + rr) * E, p.bias, E, k, G, p.kg, p.best, p.gs, SIGMOID, lane);
                const int mine = __shfl_sync(kAll, e, l8);
                if (r == rr) {
                    myE = mine;
                    on = l8 < k && myE >= 0;
                    myL = on ? row[myE] : -INFINITY;
                }
            }
        }
        on = on && live;

        // the weights, to full precision: by ratios of e^L where all scores are tiny
        const float Lm = max8(on ? myL : -INFINITY);
        float x = 0.0f, z = 1.0f;
        if (on) {
            if (p.renorm) x = !SIGMOID || Lm < -60.0f ? expf(myL - Lm) : 1.0f / (1.0f + expf(-myL));
            else x = SIGMOID ? 1.0f / (1.0f + expf(-myL)) : expf(myL - top);
            if (!SIGMOID && S != S) x = S;  // a NaN or infinite logit shows, chosen or not
        }
        if (p.renorm) {
            z = sum8(x);
        } else if (!SIGMOID) {
            float v[N];
            load(row, have, v);
            z = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) z += v[i] == -INFINITY ? 0.0f : expf(v[i] - top);
            z = sum8(z);
        }
        if (have && l8 < k) {
            p.idx[static_cast<size_t>(t) * k + l8] = on ? myE : -1;
            p.w[static_cast<size_t>(t) * k + l8] = on ? p.scale * (x / z) : 0.0f;
        }
        if (on) atomicAdd(&sh.hist[myE], 1);
        if (++rounds == 32 || tb + step >= T) {  // batches of 32 rows a lane, then the batches
            __syncwarp();
            for (int e = lane; e < E; e += 32) {
                const int at = ((e % N) / 4 * 8 + e / N) * 4 + e % 4;
                float sum = 0.0f;
#pragma unroll
                for (int rr = 0; rr < 4; ++rr) {
                    sum += acc_w[rr * E + at];
                    acc_w[rr * E + at] = 0.0f;
                }
                big[e] += sum;
            }
            rounds = 0;
        }
        __syncwarp();
    }
    router_sums(p.sums, sm, sh, E, k, 0.0f, accn);
}

template <int N>
auto pick_rows4(bool sigmoid, bool bias) {
    return sigmoid ? (bias ? router_rows4_kernel<N, true, true> : router_rows4_kernel<N, true, false>)
                   : (bias ? router_rows4_kernel<N, false, true> : router_rows4_kernel<N, false, false>);
}

}  // namespace

cudaError_t launch_router_rows4(const GroupArgs& a, bool sigmoid, int rows, int dev, void* stream) {
    static SmemOptIn opt[8][4];
    const bool bias = a.bias != nullptr;
    auto kernel = pick_rows4<4>(sigmoid, bias);
    switch (a.E / 32) {
        case 2: kernel = pick_rows4<8>(sigmoid, bias); break;
        case 3: kernel = pick_rows4<12>(sigmoid, bias); break;
        case 4: kernel = pick_rows4<16>(sigmoid, bias); break;
        case 5: kernel = pick_rows4<20>(sigmoid, bias); break;
        case 6: kernel = pick_rows4<24>(sigmoid, bias); break;
        case 7: kernel = pick_rows4<28>(sigmoid, bias); break;
        case 8: kernel = pick_rows4<32>(sigmoid, bias); break;
    }
    const int smem = rows4_floats(a.E) * 4, ctas = ceil_div_i(rows, 4);
    const cudaError_t e = api_smem_opt_in(opt[a.E / 32 - 1][2 * sigmoid + bias], dev, kernel, smem);
    if (e != cudaSuccess) return e;
    return api_launch(kernel, ctas < kRouterParts ? ctas : kRouterParts, kRows4Warps * 32, smem, stream, a);
}

}  // namespace et
