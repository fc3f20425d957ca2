// i8_ops.cu -- rows of bf16 to int8 with a scale each, and products of int8
// tokens and weights with a scale for each token and channel.
#include <cmath>
#include <type_traits>

#include "../../include/etmoe.h"
#include "et_api.h"
#include "i8_gemm.h"
#include "row_ops.cuh"

namespace et {
namespace {

constexpr int kI8KMax = 65536;
constexpr int kI8Max = 1 << 20;  // rows and channels

// ---------------------------------------------------------------- quantiser

struct I8QuantArgs {
    const bf16* x;   // [M, K]
    int8_t* q;       // [M, K]
    float* scale;    // [M]
    int row_threads;
    const int32_t* d_M;
    int M_host, M_max, K;
    EtHeader* hdr;
};

// q of eight values, packed in two words; r = 1 / s, rounded.  x = v r is within two steps of
// v / s, and x + (v - x s) r, two fused operations, is v / s correctly rounded (Markstein's
// division) for every v and s = top / 127 that bf16 has: exponents apart there are 128 x 128
// mantissas and 12 shifts, all tried.  Adding 1.5 x 2^23 rounds (half to even) and leaves
// the integer in the low bits.  Where a scale is so small that v - x s would lose bits, the
// division itself.
__device__ __forceinline__ uint2 quantize8(const Vec8& v, float s, float r, bool use_r) {
    constexpr float kMagic = 12582912.0f;
    float2 t[4];
    if (use_r) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2(v.u[i]), x = __fmul2_rn(f, both(r));
            t[i] = __fadd2_rn(__ffma2_rn(__ffma2_rn(x, both(-s), f), both(r), x), both(kMagic));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = unpack2(v.u[i]);
            t[i].x = fmaxf(-127.0f, fminf(127.0f, __fdiv_rn(x.x, s))) + kMagic;
            t[i].y = fmaxf(-127.0f, fminf(127.0f, __fdiv_rn(x.y, s))) + kMagic;
        }
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __byte_perm(__float_as_uint(t[i].x), __float_as_uint(t[i].y), 0x0040);
    return make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410));
}

// A row's largest magnitude, then its values: a row of up to sixteen columns a thread
// (16384) stays in registers, and the next one is on its way meanwhile; a longer one is
// read again (from the caches).  Bound by HBM and the wait for a row's maximum (4096 x 4096:
// 10.3 us, 4.9 TB/s; 4096 x 14336: 37 us, 4.8).
template <bool VEC, int MODE>
__global__ void __launch_bounds__(MODE == kRowsOne ? 1024 : 256) i8_quantize_kernel(const I8QuantArgs p) {
    constexpr int V = norm_v(MODE);
    __shared__ uint32_t red[2][32];
    int n = 0;
    const RowGroup<MODE> g(p.row_threads);
    grid_begin();
    bool ok;
    const int M = row_count(p.d_M, p.M_host, p.M_max, p.hdr, &ok);
    const int K = p.K, span = g.th() * 8 * V, step = gridDim.x * g.groups();
    const bool whole = K <= span;
    Vec8 v[V], next[V];
    auto fetch = [&](int m) {
#pragma unroll
        for (int j = 0; j < V; ++j) next[j] = m < M ? load8<VEC>(p.x + static_cast<size_t>(m) * K, g, j, K) : Vec8{};
    };
    int m = blockIdx.x * g.groups() + g.id();
    if (whole) fetch(m);
    for (; m < M; m += step) {
        const bf16* row = p.x + static_cast<size_t>(m) * K;
        uint32_t top = 0;  // two at once, as the bits of |x|, which order as their values do, NaN above infinity
        auto look = [&]() {
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int i = 0; i < 4; i += 2) top = __vimax3_u16x2(top, v[j].u[i] & 0x7fff7fffu, v[j].u[i + 1] & 0x7fff7fffu);
        };
        if (whole) {
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = next[j];
            fetch(m + step);
            look();
        } else {
            for (int c0 = 0; c0 < K; c0 += span) {
#pragma unroll
                for (int j = 0; j < V; ++j) v[j] = load8<VEC>(row + c0, g, j, K - c0);
                look();
            }
        }
        top = __reduce_max_sync(0xffffffffu, max(top << 16, top & 0xffff0000u));
        if (MODE != kRowsWarp) {
            const int slot = n++ & 1, lane = threadIdx.x & 31, first = g.id() * (g.th() >> 5);
            if (lane == 0) red[slot][threadIdx.x >> 5] = top;
            g.sync();
            top = __reduce_max_sync(0xffffffffu, lane < (g.th() >> 5) ? red[slot][first + lane] : 0u);
        }
        const bool finite = top < 0x7f800000u, live = finite && top != 0;
        const float s = finite ? __fdiv_rn(__uint_as_float(top), 127.0f) : __int_as_float(0x7fffffff);
        const bool use_r = s >= 1e-27f;
        const float r = use_r ? __frcp_rn(s) : 0.0f;
        if (g.lane() == 0) p.scale[m] = s;
        int8_t* out = p.q + static_cast<size_t>(m) * K;
        for (int c0 = 0; c0 < K; c0 += span)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (!whole) v[j] = load8<VEC>(row + c0, g, j, K - c0);
                uint2 q = make_uint2(0, 0);
                if (live) q = quantize8(v[j], s, r, use_r);
                if (VEC) {
                    const int c = c0 + g.template col<VEC>(j, 0);
                    if (c < K) *reinterpret_cast<uint2*>(out + c) = q;
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int c = c0 + g.template col<VEC>(j, i);
                        if (c < K) out[c] = static_cast<int8_t>((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
                    }
                }
            }
    }
}

// ---------------------------------------------------------------- products of few rows

struct I8GemmArgs {
    const int8_t* x;   // [M, K]
    const float* sx;   // [M]
    const int8_t* w;   // [N, K]
    const float* sw;   // [N]
    bf16* y;           // [M, N]
    const int32_t* d_M;
    int M_host, M_max, N, K;
    EtHeader* hdr;
};

constexpr int kGemvWarps = 8;
constexpr int kGemvRows = 16;   // channels of a CTA
constexpr int kGemvCtas = 2;    // CTAs an SM

__device__ __forceinline__ int4 load_weights(const int8_t* p) {  // streamed: the tokens keep L1
    int4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// d += A B, A 16 channels x 16 k, B 16 k x 8 tokens: fp32 sums, exact up to 2^24 for int8 values.
__device__ __forceinline__ void mma_f16_sync(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void int8x16_to_half(const int4& v, uint32_t (&h)[8]) {
    int8_to_half(v.x, h[0], h[1]);
    int8_to_half(v.y, h[2], h[3]);
    int8_to_half(v.z, h[4], h[5]);
    int8_to_half(v.w, h[6], h[7]);
}
// c += A B, A 16 channels x 32 k, B 32 k x 8 tokens: exact in int32.
__device__ __forceinline__ void mma_s8(int (&c)[4], int a0, int a1, int a2, int a3, int b0, int b1) {
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 MT tokens times 16 channels a tile, a CTA its tiles in turn; its warps take 128-byte
// pieces of K in turn, and the next pieces, of this tile or the next, are on their way
// meanwhile.  A thread's 16-byte loads are its fragments as they are: the order of k within
// a piece is the same for both operands, and no other order matters to an exact sum.  An
// integer MMA takes 16 cycles of an SM here, 32 / MT bytes of weights a cycle, where HBM
// brings 23: up to 8 tokens (14336 x 4096: 11.5 us, 5.1 TB/s from launch to end, bound by
// HBM).  HALF: both operands become fp16 in registers, whose MMAs take 2 cycles for half as
// many k; 5 instructions convert 4 bytes, and the sums of a warp, fp32, are exact up to 2^24,
// so for K up to 8192.  16 tokens 13.4 us (17.7 with integer MMAs); bound by its instructions'
// latency and by the tokens, which every tile reads again: as many bytes as its weights.
// (Three pieces ahead in place of two 14.7, the tokens one piece ahead 15.1, three CTAs an SM
// with one piece 14.1 and 20 for 4096 x 14336.)
template <int MT, bool HALF>
__global__ void __launch_bounds__(kGemvWarps * 32, kGemvCtas) i8_gemv_kernel(const I8GemmArgs p) {
    __shared__ int red[2][kGemvWarps][8 * MT][kGemvRows + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
    const int K = p.K, tiles = (p.N + kGemvRows - 1) / kGemvRows, k0 = warp * 128 + q * 16;
    constexpr int kStep = kGemvWarps * 128, kAhead = HALF ? 2 : 3;  // pieces of K that a warp has on their way
    // Where this thread's next piece is.
    int ft = blockIdx.x, fk = k0;
    auto rows_of = [&](int t, const int8_t*& w0, const int8_t*& w1) {
        w0 = p.w + static_cast<size_t>(min(t * kGemvRows + g, p.N - 1)) * K;
        w1 = p.w + static_cast<size_t>(min(t * kGemvRows + g + 8, p.N - 1)) * K;
    };
    const int8_t *w0, *w1;
    rows_of(ft, w0, w1);
    // Nothing is read before what comes before has ended, but the first pieces may be on
    // their way to L2 by then.
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (fk + i * kStep < K) {
            asm volatile("prefetch.global.L2 [%0];" ::"l"(w0 + fk + i * kStep));
            asm volatile("prefetch.global.L2 [%0];" ::"l"(w1 + fk + i * kStep));
        }
    grid_begin();
    bool ok;
    const int M = row_count(p.d_M, p.M_host, p.M_max, p.hdr, &ok);
    if (M < 1) return;
    const int8_t* x[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) x[t] = p.x + static_cast<size_t>(min(8 * t + g, M - 1)) * K;
    const int4 zero = make_int4(0, 0, 0, 0);
    int4 wv[kAhead][4];  // rows g and g + 8, bytes k and k + 64
    auto fetch = [&](int4 (&v)[4]) {
        const bool here = ft < tiles;
        v[0] = here && fk < K ? load_weights(w0 + fk) : zero;
        v[1] = here && fk < K ? load_weights(w1 + fk) : zero;
        v[2] = here && fk + 64 < K ? load_weights(w0 + fk + 64) : zero;
        v[3] = here && fk + 64 < K ? load_weights(w1 + fk + 64) : zero;
        fk += kStep;
        if (fk - q * 16 >= K) {
            fk = k0;
            ft += gridDim.x;
            rows_of(min(ft, tiles - 1), w0, w1);
        }
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(wv[i]);
    int tile = blockIdx.x, k = k0, buf = 0;
    using Acc = std::conditional_t<HALF, float, int>;
    Acc acc[MT][4] = {};
    while (tile < tiles) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (tile >= tiles) break;
            if constexpr (HALF) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t a[8], b[8];  // rows g and g + 8
                    int8x16_to_half(wv[i][2 * h], a);
                    int8x16_to_half(wv[i][2 * h + 1], b);
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        const int4 v = k + 64 * h < K ? *reinterpret_cast<const int4*>(x[t] + k + 64 * h) : zero;
                        uint32_t c[8];
                        int8x16_to_half(v, c);
#pragma unroll
                        for (int j = 0; j < 8; j += 2) mma_f16_sync(acc[t], a[j], b[j], a[j + 1], b[j + 1], c[j], c[j + 1]);
                    }
                }
            } else
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const int4 x0 = k < K ? *reinterpret_cast<const int4*>(x[t] + k) : zero;
                const int4 x1 = k + 64 < K ? *reinterpret_cast<const int4*>(x[t] + k + 64) : zero;
                mma_s8(acc[t], wv[i][0].x, wv[i][1].x, wv[i][0].y, wv[i][1].y, x0.x, x0.y);
                mma_s8(acc[t], wv[i][0].z, wv[i][1].z, wv[i][0].w, wv[i][1].w, x0.z, x0.w);
                mma_s8(acc[t], wv[i][2].x, wv[i][3].x, wv[i][2].y, wv[i][3].y, x1.x, x1.y);
                mma_s8(acc[t], wv[i][2].z, wv[i][3].z, wv[i][2].w, wv[i][3].w, x1.z, x1.w);
            }
            fetch(wv[i]);
            k += kStep;
            if (k - q * 16 >= K) {  // the tile's last piece: for the warps of K's end one or two pieces sooner
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        red[buf][warp][8 * t + 2 * q + (j & 1)][g + (j >> 1) * 8] = static_cast<int>(acc[t][j]);
                        acc[t][j] = 0;
                    }
                __syncthreads();  // (the other buffer has been read: who comes here has left it)
#pragma unroll
                for (int o = threadIdx.x; o < 8 * MT * kGemvRows; o += kGemvWarps * 32) {
                    const int m = o / kGemvRows, r = o % kGemvRows, n = tile * kGemvRows + r;
                    int s = 0;
#pragma unroll
                    for (int v = 0; v < kGemvWarps; ++v) s += red[buf][v][m][r];
                    if (m < M && n < p.N) p.y[static_cast<size_t>(m) * p.N + n] = __float2bfloat16_rn(static_cast<float>(s) * (p.sx[m] * p.sw[n]));
                }
                buf ^= 1;
                tile += gridDim.x;
                k = k0;
            }
        }
    }
}

// Which calls take the form above: up to 16 tokens, and up to 32 where the weights are few.
// Measured, 32 tokens, this form and the tcgen05 form: 1024 x 1024 2.7 and 5.6 us, 2048 x 2048
// 3.8 and 6.6, 4096 x 4096 7.8 and 9.0; 4096 x 5120 9.1 and 9.7, 8192 x 2560 10.2 and 9.8, 5120
// x 4096 12.1 and 11.4; 6144 x 4096 13.5 and 11.6, 14336 x 4096 19.8 and 15.6: they meet at 20 to
// 25 MB of weights.  (17 to 24 tokens at 25 to 34 MB: 4096 x 8192 11.2 and 11.9, 14336 x 4096
// 17.2 and 15.5.  What one limit costs them is 15 % at most, 4096 x 6144 9.1 and 10.4.)
bool i8_gemv(int M_max, int N, int K) {
    return M_max <= 16 || (M_max <= 32 && static_cast<long long>(N) * K <= 22000000);
}

bool i8_shape_ok(int M_max, int N, int K, std::string* why) {
    if (M_max < 1 || M_max > kI8Max || N < 1 || N > kI8Max) { *why = "M_max and N must be in [1, 2^20]"; return false; }
    if (K < 16 || K > kI8KMax || K % 16) { *why = "K must be a multiple of 16 in [16, 65536]"; return false; }
    return true;
}

int i8_check_rows(int M, const int32_t* d_M, int M_max) {
    if (!api_aligned(d_M, 4)) return api_fail(ET_ERR_INVALID, "tensors must be aligned to their element size");
    if (!d_M && (M < 0 || M > M_max)) return api_fail(ET_ERR_INVALID, "M must be in [0, M_max]");
    return ET_OK;
}

// How a pass of M rows runs on the tensor cores.
struct I8Plan {
    bool pair;
    int tn, nt, kblocks, grid, split;
};

int ceil_div_l(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

// Estimated cycles of a pass in one form, without what all forms have.  Numbers: measured
// over the forms of some twenty shapes; a block is 128 x 128 weights and the tile's tokens.
double i8_cost(int M, const I8Plan& p) {
    const long long tiles = static_cast<long long>(ceil_div_l(M, p.tn)) * p.nt, units = tiles * p.split;
    const int most = p.pair ? kI8Sms / 2 : kI8Sms;
    const double waves = p.split > 1 ? 1.0 : static_cast<double>(ceil_div_l(tiles, most));
    const double ctas = static_cast<double>(units < most ? units : most) * (p.pair ? 2 : 1);
    double block = 4.0 * p.tn;                                        // the MMAs,
    auto at_least = [&](double v) { if (v > block) block = v; };
    at_least(waves > 1.0 ? 600.0 : 560.0);                            // the weights' conversion,
    at_least((16384.0 + 128.0 * p.tn) / 50.0);                        // what an SM gets from L2,
    if (waves == 1.0) at_least(16384.0 * ctas / 3500.0);              // what HBM brings,
    if (!p.pair) at_least(p.tn > 128 ? 1900.0 : p.tn > 64 ? 1090.0 : p.tn > 32 ? 700.0 : 560.0);  // the tokens' conversion
    double tile = ceil_div_l(p.kblocks, p.split) * block;
    tile += p.tn > 128 || waves == 1.0 ? 9.0 * p.tn : 200.0;          // the epilogue, where nothing runs beside it
    const int cluster = p.split * (p.pair ? 2 : 1);
    if (p.split > 1) tile += 3000.0 + 10.0 * p.tn + (cluster == 8 ? 9000.0 : 0.0);  // clusters of 8 find few places
    return waves * tile + (p.pair ? 1500.0 + 3.0 * M * p.kblocks * kI8KBlock / 2600.0 : 0.0);
}

I8Plan i8_plan(int M, int N, int K) {
    I8Plan best{};
    double cost = 0.0;
    for (int pair = 0; pair < 2; ++pair)
        for (int tn = 32; tn <= kI8TokensMax; tn += 32) {
            I8Plan p{};
            p.pair = pair != 0;
            p.kblocks = ceil_div_l(K, kI8KBlock);
            p.nt = ceil_div_l(N, pair ? 256 : 128);
            const int mt = ceil_div_l(M, tn);
            p.tn = ceil_div_l(ceil_div_l(M, mt), 32) * 32;
            const long long tiles = static_cast<long long>(mt) * p.nt;
            const int most = pair ? kI8Sms / 2 : kI8Sms;
            p.grid = tiles < most ? static_cast<int>(tiles) : most;
            for (p.split = 1; p.split <= (pair ? 4 : 8); p.split *= 2) {
                if (p.split > 1 && (p.split * tiles > most || p.split > p.kblocks)) break;
                const double c = i8_cost(M, p);
                if (!best.tn || c < cost) {
                    best = p;
                    cost = c;
                }
            }
            if (tn >= M) break;
        }
    return best;
}

// Tokens that a call holds as fp16 at a time: at K = 4096 they stay in L2 with their
// weights, and the workspace of a long batch stays small.
constexpr int kI8RowsPass = 8192;

size_t i8_ws_bytes(int M_max, int N, int K) {
    const size_t rows = i8_gemv(M_max, N, K) ? 0 : M_max < kI8RowsPass ? M_max : kI8RowsPass;
    return (kHeaderBytes + 2 * rows * K + 255) / 256 * 256;
}

template <bool VEC>
cudaError_t launch_i8_quantize(I8QuantArgs a, int rows, int sms, void* stream) {
    const int cols = a.K < kNormHMax ? a.K : kNormHMax;
    a.row_threads = norm_threads(cols);
    const RowMode mode = norm_mode(cols, a.row_threads);
    const int groups = norm_groups(a.row_threads, rows), th = a.row_threads * groups;
    const int need = (rows + groups - 1) / groups, most = sms * (1024 / th);  // as many as find room at once
    return api_launch(mode == kRowsWarp ? i8_quantize_kernel<VEC, kRowsWarp> : mode == kRowsGroup ? i8_quantize_kernel<VEC, kRowsGroup>
                                                                             : i8_quantize_kernel<VEC, kRowsOne>,
                      need < most ? need : most, th, 0, stream, a);
}

}  // namespace
}  // namespace et

using namespace et;

extern "C" {

size_t et_i8_quantize_workspace_bytes(int M_max, int K) {
    std::string why;
    return i8_shape_ok(M_max, 1, K, &why) ? kHeaderBytes : 0;
}

int et_i8_quantize(const void* x, void* q, float* scale, int M, const int32_t* d_M, int M_max, int K, void* workspace,
                   size_t workspace_bytes, void* stream) {
    return api_entry([&]() -> int {
        std::string why;
        if (!i8_shape_ok(M_max, 1, K, &why)) return api_fail(ET_ERR_UNSUPPORTED, why);
        if (!x || !q || !scale) return api_fail(ET_ERR_INVALID, "x, q and scale must be non-NULL");
        if (!api_aligned(q, 16)) return api_fail(ET_ERR_INVALID, "q must be 16-byte aligned");
        if (!api_aligned(x, 2) || !api_aligned(scale, 4))
            return api_fail(ET_ERR_INVALID, "tensors must be aligned to their element size");
        int rc = i8_check_rows(M, d_M, M_max);
        if (rc) return rc;
        if ((rc = api_check_ws(workspace, workspace_bytes, kHeaderBytes))) return rc;
        if (!d_M && M == 0) return ET_OK;
        int dev = 0, sms = 0;
        if ((rc = api_device(&dev, &sms))) return rc;
        const I8QuantArgs a{static_cast<const bf16*>(x), static_cast<int8_t*>(q), scale, 0, d_M, M, M_max, K,
                            static_cast<EtHeader*>(workspace)};
        const int rows = d_M ? M_max : M;
        const cudaError_t e = api_aligned(x, 16) ? launch_i8_quantize<true>(a, rows, sms, stream)
                                                 : launch_i8_quantize<false>(a, rows, sms, stream);
        if (e != cudaSuccess) return api_fail_cuda(e, "launch of the int8 quantiser");
        return ET_OK;
    });
}

size_t et_i8_gemm_workspace_bytes(int M_max, int N, int K) {
    std::string why;
    return i8_shape_ok(M_max, N, K, &why) ? i8_ws_bytes(M_max, N, K) : 0;
}

int et_i8_gemm(const void* x_q, const float* s_x, const void* w_q, const float* s_w, void* Y, int M, const int32_t* d_M,
               int M_max, int N, int K, void* workspace, size_t workspace_bytes, void* stream) {
    return et_i8_gemm_opts(x_q, s_x, w_q, s_w, Y, M, d_M, M_max, N, K, workspace, workspace_bytes, nullptr, stream);
}

int et_i8_gemm_opts(const void* x_q, const float* s_x, const void* w_q, const float* s_w, void* Y, int M, const int32_t* d_M,
                    int M_max, int N, int K, void* workspace, size_t workspace_bytes, const et_opts* opts, void* stream) {
    return api_entry([&]() -> int {
        std::string why;
        if (!i8_shape_ok(M_max, N, K, &why)) return api_fail(ET_ERR_UNSUPPORTED, why);
        if (!x_q || !s_x || !w_q || !s_w || !Y) return api_fail(ET_ERR_INVALID, "x_q, s_x, w_q, s_w and Y must be non-NULL");
        if (!api_aligned(x_q, 16) || !api_aligned(w_q, 16)) return api_fail(ET_ERR_INVALID, "x_q and w_q must be 16-byte aligned");
        if (!api_aligned(s_x, 4) || !api_aligned(s_w, 4) || !api_aligned(Y, 2))
            return api_fail(ET_ERR_INVALID, "tensors must be aligned to their element size");
        int rc = i8_check_rows(M, d_M, M_max);
        if (rc) return rc;
        if ((rc = api_check_ws(workspace, workspace_bytes, i8_ws_bytes(M_max, N, K)))) return rc;
        if (!d_M && M == 0) return ET_OK;
        int dev = 0, sms = 0;
        if ((rc = api_device(&dev, &sms))) return rc;
        const int all = d_M ? M_max : M;
        uint8_t* ws = static_cast<uint8_t*>(workspace);
        EtHeader* hdr = reinterpret_cast<EtHeader*>(ws);
        const int8_t* x = static_cast<const int8_t*>(x_q);
        bf16* y = static_cast<bf16*>(Y);
        if (i8_gemv(all, N, K)) {
            const I8GemmArgs a{x, s_x, static_cast<const int8_t*>(w_q), s_w, y, d_M, M, all, N, K, hdr};
            const int tiles = (N + kGemvRows - 1) / kGemvRows;
            const cudaError_t e = api_launch(all <= 8 ? i8_gemv_kernel<1, false> : all <= 16 ? i8_gemv_kernel<2, true> : all <= 24 ? i8_gemv_kernel<3, true> : i8_gemv_kernel<4, true>, tiles < kGemvCtas * sms ? tiles : kGemvCtas * sms, kGemvWarps * 32, 0, stream, a);
            if (e != cudaSuccess) return api_fail_cuda(e, "launch of the int8 product");
            return ET_OK;
        }
        CUtensorMap mw;
        if ((rc = api_map128(&mw, w_q, 1, N, K, 128, "w_q"))) return rc;
        for (int m0 = 0; m0 < all; m0 += kI8RowsPass) {
            const int rows = all - m0 < kI8RowsPass ? all - m0 : kI8RowsPass;
            const I8Plan pl = i8_plan(rows, N, K);
            I8TcArgs a{};
            a.x = x + static_cast<size_t>(m0) * K;
            a.sx = s_x + m0;
            a.sw = s_w;
            a.y = y + static_cast<size_t>(m0) * N;
            a.rows = {d_M, m0, rows, all};
            a.N = N;
            a.K = K;
            a.hdr = hdr;
            a.tn = pl.tn;
            a.nt = pl.nt;
            a.kblocks = pl.kblocks;
            a.grid = pl.grid;
            a.split = pl.split;
            a.blocks = ceil_div_l(pl.kblocks, pl.split) * ceil_div_l(static_cast<long long>(ceil_div_l(rows, pl.tn)) * pl.nt, pl.grid);
            i8_tc_stages(pl.pair, pl.tn, a.blocks, &a.stages_w, &a.stages_x);
            a.timeout_ns = api_timeout_ns(opts);
            a.fault_cta = opts && opts->fault_mode == 1 ? opts->fault_arg : -1;
            cudaError_t e = cudaSuccess;
            CUtensorMap mx = mw;
            if (pl.pair) {
                void* x16 = ws + kHeaderBytes;
                if ((rc = api_map128(&mx, x16, 2, rows, K, pl.tn / 2, "x_q as fp16"))) return rc;
                e = launch_i8_expand({a.x, x16, a.rows, K, hdr}, sms, stream);
            }
            if (e == cudaSuccess) e = launch_i8_tc(a, &mw, &mx, pl.pair, dev, stream);
            if (e != cudaSuccess) return api_fail_cuda(e, "launch of the int8 product");
        }
        return ET_OK;
    });
}

}  // extern "C"
