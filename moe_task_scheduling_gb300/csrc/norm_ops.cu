// norm_ops.cu -- the norms either side of a block with its gate and residual
// scale, in one pass, and their gradient.
//
//   n = RMSNorm(y) * gamma_post (or y);  z = x + scale * gate * n;
//   x_hat = RMSNorm(z) * gamma_pre
#include <cmath>

#include "../../include/etmoe.h"
#include "et_api.h"
#include "ops_device.cuh"

namespace et {
namespace {

enum GateKind { kGateNone = 0, kGateChannel = 1, kGateToken = 2, kGateFull = 3 };

constexpr int kNormHMax = 16384;
constexpr int kNormParts = 304;  // most CTAs of the backward kernel = rows of partial sums

struct NormArgs {
    const bf16* x;           // [T, H]
    const bf16* y;           // [T, H] or null (z = x)
    const bf16* gamma_post;  // [H] or null
    const void* gate;        // bf16 [H], fp32 [T], bf16 [T, H] or null
    const bf16* gamma_pre;   // [H] or null
    float scale, eps, inv_H;
    int gate_kind;
    const int32_t* d_T;
    int T_host, T_max, H;
    EtHeader* hdr;
    bf16* x_out;             // [T, H] or null
    bf16* x_hat;             // [T, H] or null
    // backward
    const bf16* d_x_out;     // [T, H] or null
    const bf16* d_x_hat;     // [T, H] or null
    bf16* dx;
    bf16* dy;
    bf16* d_gate_full;       // [T, H]
    float* d_gate_token;     // [T]
    float* part;             // [kNormParts][3][H]: d_gamma_post, d_gamma_pre, d_gate per channel
};

// Eight consecutive bf16 of a row, packed.
struct Vec8 {
    uint32_t u[4];
    __device__ __forceinline__ float operator[](int i) const {
        return (i & 1) ? bf_hi(u[i >> 1]) : bf_lo(u[i >> 1]);
    }
};

// Columns [c, c + 8) of a row of H.  VEC: one 16-byte access (H a multiple of 8
// and the tensors 16-byte aligned); else element by element, for any H.
template <bool VEC>
__device__ __forceinline__ Vec8 load8(const bf16* row, int c, int H) {
    Vec8 v{};
    if (VEC) {
        if (c < H) {
            const uint4 q = *reinterpret_cast<const uint4*>(row + c);
            v.u[0] = q.x; v.u[1] = q.y; v.u[2] = q.z; v.u[3] = q.w;
        }
    } else {
        const uint16_t* r = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < H) v.u[i >> 1] |= static_cast<uint32_t>(r[c + i]) << (16 * (i & 1));
    }
    return v;
}

template <bool VEC>
__device__ __forceinline__ void store8(bf16* row, int c, int H, const float* f) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
    if (VEC) {
        if (c < H) *reinterpret_cast<uint4*>(row + c) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
        uint16_t* r = reinterpret_cast<uint16_t*>(row);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < H) r[c + i] = static_cast<uint16_t>(u[i >> 1] >> (16 * (i & 1)));
    }
}

// Sum over the row's threads, the same bits in every one of them.  ROW: the
// whole CTA holds one row; else a warp does.  Consecutive sums alternate
// between two slots (n counts them), so one barrier a sum is enough: who has
// passed the next sum's barrier knows that all have read this one.
template <bool ROW>
__device__ __forceinline__ float row_sum(float v, float (*red)[32], int& n) {
    v = warp_sum(v);
    if (ROW) {
        const int slot = n++ & 1;
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (lane == 0) red[slot][warp] = v;
        __syncthreads();
        v = warp_sum(lane < static_cast<int>(blockDim.x >> 5) ? red[slot][lane] : 0.0f);
    }
    return v;
}

// 1 / sqrt(sum / H + eps)
__device__ __forceinline__ float inv_rms(float sum, float inv_H, float eps) { return rsqrtf(sum * inv_H + eps); }

// V vectors of 8 columns a thread; ROW: one row a CTA, else one row a warp.
template <int V, bool VEC, bool ROW>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(const NormArgs p) {
    __shared__ float red[2][32];
    int sums = 0;
    grid_begin();
    bool ok;
    const int T = row_count(p.d_T, p.T_host, p.T_max, p.hdr, &ok);
    const int H = p.H;
    const int width = ROW ? blockDim.x : 32;
    const int lane = ROW ? threadIdx.x : threadIdx.x & 31;
    const int rows_cta = ROW ? 1 : blockDim.x >> 5;
    for (int t = blockIdx.x * rows_cta + (ROW ? 0 : threadIdx.x >> 5); t < T; t += gridDim.x * rows_cta) {
        const size_t off = static_cast<size_t>(t) * H;
        float z[V][8];
        Vec8 yv[V], gv[V];
        float ss = 0.0f;
        const bool vec_gate = p.gate_kind == kGateFull || p.gate_kind == kGateChannel;
        const bf16* grow = static_cast<const bf16*>(p.gate) + (p.gate_kind == kGateFull ? off : 0);
#pragma unroll
        for (int j = 0; j < V; ++j) {  // every load of the row before the first sum
            const int c = (j * width + lane) * 8;
            const Vec8 xv = load8<VEC>(p.x + off, c, H);
            yv[j] = p.y ? load8<VEC>(p.y + off, c, H) : Vec8{};
            gv[j] = vec_gate ? load8<VEC>(grow, c, H) : Vec8{};
#pragma unroll
            for (int i = 0; i < 8; ++i) z[j][i] = xv[i];
        }
        const float gtok = p.gate_kind == kGateToken ? static_cast<const float*>(p.gate)[t] : 1.0f;
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) ss += yv[j][i] * yv[j][i];
        float ry = 1.0f;
        if (p.y && p.gamma_post) ry = inv_rms(row_sum<ROW>(ss, red, sums), p.inv_H, p.eps);
        float zz = 0.0f;
        const float gs = p.scale * gtok;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (j * width + lane) * 8;
            if (p.y && c < H) {
                const Vec8 gp = p.gamma_post ? load8<VEC>(p.gamma_post, c, H) : Vec8{};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float n = p.gamma_post ? yv[j][i] * ry * gp[i] : yv[j][i];
                    z[j][i] += (vec_gate ? gs * gv[j][i] : gs) * n;  // 0 past H, where y is 0
                }
            }
            if (p.x_out && c < H) store8<VEC>(p.x_out + off, c, H, z[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) zz += z[j][i] * z[j][i];
        }
        if (p.x_hat) {
            const float rz = inv_rms(row_sum<ROW>(zz, red, sums), p.inv_H, p.eps);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (j * width + lane) * 8;
                if (c < H) {
                    const Vec8 gp = load8<VEC>(p.gamma_pre, c, H);
                    float o[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = z[j][i] * rz * gp[i];
                    store8<VEC>(p.x_hat + off, c, H, o);
                }
            }
        }
    }
}

// Two sums over the row's threads with one barrier (see row_sum).
template <bool ROW>
__device__ __forceinline__ float2 row_sum2(float2 v, float (*red)[32], float (*red2)[32], int& n) {
    v.x = warp_sum(v.x);
    v.y = warp_sum(v.y);
    if (ROW) {
        const int slot = n++ & 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (lane == 0) { red[slot][warp] = v.x; red2[slot][warp] = v.y; }
        __syncthreads();
        const bool in = lane < static_cast<int>(blockDim.x >> 5);
        v.x = warp_sum(in ? red[slot][lane] : 0.0f);
        v.y = warp_sum(in ? red2[slot][lane] : 0.0f);
    }
    return v;
}

// The gradient.  A row's statistics are recomputed from x and y (they are read
// anyway).  The parameter gradients are summed over this CTA's rows in
// registers, thread by thread for its own columns, then over CTAs by
// norm_sum_kernel in a fixed order.  Three sums a row: mean y^2; mean z^2 with
// the second norm's projection; the first norm's projection (with a per-token
// gate's gradient).
//
// This form serves every H, alignment and combination of the optional parts;
// norm_bwd_staged_kernel the usual one.  MAXT: most threads, which bounds the
// registers.
template <int V, bool VEC, bool ROW, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_bwd_kernel(const NormArgs p) {
    __shared__ float red[2][32], red2[2][32];
    int sums = 0;
    extern __shared__ __align__(16) uint8_t dyn[];  // !ROW: [warps][3][256] floats
    grid_begin();
    bool ok;
    const int T = row_count(p.d_T, p.T_host, p.T_max, p.hdr, &ok);
    const int H = p.H;
    const int width = ROW ? blockDim.x : 32;
    const int lane = ROW ? threadIdx.x : threadIdx.x & 31;
    const int rows_cta = ROW ? 1 : blockDim.x >> 5;
    const int step = gridDim.x * rows_cta;
    const bool post = p.y && p.gamma_post;
    const bool full = p.gate_kind == kGateFull;
    float a_post[V][8], a_pre[V][8], a_gate[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) a_post[j][i] = a_pre[j][i] = a_gate[j][i] = 0.0f;

    // columns [c, c + 8) of a row of one input (zeros where it is not given)
    auto row8 = [&](const bf16* base, int t, int c) -> Vec8 {
        return base ? load8<VEC>(base + static_cast<size_t>(t) * H, c, H) : Vec8{};
    };
    // scale * gate of columns [c, c + 8)
    auto gate_of = [&](int t, int c, float gs, float* g) {
        if (full || p.gate_kind == kGateChannel) {
            const Vec8 v = row8(static_cast<const bf16*>(p.gate), full ? t : 0, c);
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = gs * v[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = gs;
        }
    };

    for (int t = blockIdx.x * rows_cta + (ROW ? 0 : threadIdx.x >> 5); t < T; t += step) {
        const size_t off = static_cast<size_t>(t) * H;
        float ss = 0.0f;
        if (post)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const Vec8 yv = row8(p.y, t, (j * width + lane) * 8);
#pragma unroll
                for (int i = 0; i < 8; ++i) ss += yv[i] * yv[i];
            }
        const float gs = p.scale * (p.gate_kind == kGateToken ? static_cast<const float*>(p.gate)[t] : 1.0f);
        float ry = 1.0f;
        if (post) ry = inv_rms(row_sum<ROW>(ss, red, sums), p.inv_H, p.eps);
        // z, and with it the statistics of the second norm and sum(d_x_hat gamma_pre z)
        float z[V][8];
        float2 za = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (j * width + lane) * 8;
            const Vec8 xv = row8(p.x, t, c);
#pragma unroll
            for (int i = 0; i < 8; ++i) z[j][i] = xv[i];
            if (c < H) {
                if (p.y) {
                    float g[8];
                    gate_of(t, c, gs, g);
                    const Vec8 yv = row8(p.y, t, c);
                    const Vec8 gp = post ? load8<VEC>(p.gamma_post, c, H) : Vec8{};
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        z[j][i] += g[i] * (post ? yv[i] * ry * gp[i] : yv[i]);  // 0 past H, where y is 0
                }
                if (p.d_x_hat) {
                    const Vec8 dh = row8(p.d_x_hat, t, c);
                    const Vec8 gp = load8<VEC>(p.gamma_pre, c, H);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        za.x += z[j][i] * z[j][i];
                        za.y += dh[i] * gp[i] * z[j][i];
                    }
                }
            }
        }
        float rz = 0.0f, k2 = 0.0f;
        if (p.d_x_hat) {
            za = row_sum2<ROW>(za, red, red2, sums);
            rz = inv_rms(za.x, p.inv_H, p.eps);
            k2 = za.y * p.inv_H * rz * rz * rz;
        }
        // d z, the parameter gradients, and sum(d n gamma_post y)
        float2 bg = make_float2(0.0f, 0.0f);
        float d[V][8];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (j * width + lane) * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) d[j][i] = 0.0f;
            if (c < H) {
                const Vec8 dz = row8(p.d_x_out, t, c);
#pragma unroll
                for (int i = 0; i < 8; ++i) d[j][i] = dz[i];
                if (p.d_x_hat) {
                    const Vec8 dh = row8(p.d_x_hat, t, c);
                    const Vec8 gp = load8<VEC>(p.gamma_pre, c, H);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        d[j][i] += rz * (dh[i] * gp[i]) - z[j][i] * k2;
                        a_pre[j][i] += dh[i] * (z[j][i] * rz);
                    }
                }
                store8<VEC>(p.dx + off, c, H, d[j]);
                if (p.y) {
                    float g[8], dgf[8];
                    gate_of(t, c, gs, g);
                    const Vec8 yv = row8(p.y, t, c);
                    const Vec8 gp = post ? load8<VEC>(p.gamma_post, c, H) : Vec8{};
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float u = yv[i] * ry;  // the normalised value
                        const float n = post ? u * gp[i] : yv[i];
                        dgf[i] = p.scale * n * d[j][i];
                        d[j][i] *= g[i];  // d n
                        a_post[j][i] += d[j][i] * u;
                        if (post) {
                            d[j][i] *= gp[i];
                            bg.x += d[j][i] * yv[i];
                        }
                        a_gate[j][i] += dgf[i];
                        bg.y += dgf[i];
                    }
                    if (p.d_gate_full) store8<VEC>(p.d_gate_full + off, c, H, dgf);
                }
            }
        }
        if (p.y) {
            if (post || p.d_gate_token) bg = row_sum2<ROW>(bg, red, red2, sums);
            const float k1 = post ? bg.x * p.inv_H * ry * ry * ry : 0.0f;
            if (p.d_gate_token && lane == 0) p.d_gate_token[t] = bg.y;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (j * width + lane) * 8;
                if (c < H) {
                    const Vec8 yv = row8(p.y, t, c);
                    float o[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = post ? ry * d[j][i] - yv[i] * k1 : d[j][i];
                    store8<VEC>(p.dy + off, c, H, o);
                }
            }
        }
    }
    if (!ok) return;
    float* part = p.part + static_cast<size_t>(blockIdx.x) * 3 * H;
    if (ROW) {
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = (j * width + lane) * 8 + i;
                if (c < H) {
                    part[c] = a_post[j][i];
                    part[H + c] = a_pre[j][i];
                    part[2 * H + c] = a_gate[j][i];
                }
            }
    } else {  // one row a warp (H <= 256): the CTA's warps in order
        const int warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
        float* acc_sm = reinterpret_cast<float*>(dyn);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float* a = acc_sm + warp * 768 + lane * 8 + i;
            a[0] = a_post[0][i];
            a[256] = a_pre[0][i];
            a[512] = a_gate[0][i];
        }
        __syncthreads();
        for (int o = threadIdx.x; o < 3 * H; o += blockDim.x) {
            const int arr = o / H, c = o - arr * H;
            float s = 0.0f;
            for (int w = 0; w < nwarps; ++w) s += acc_sm[w * 768 + arr * 256 + c];
            part[o] = s;
        }
    }
}

// The same gradient where y, gamma_pre and both incoming gradients are given, H
// is a multiple of 8 in (512, 8192] and every tensor is 16-byte aligned.
//
// Bound by HBM (T = H = 4096 with a full gate: 268 MB) if a row's latencies are
// hidden: the input rows of this CTA's next row are copied to shared memory
// while the current one is worked on, each thread reading back only what it
// copied itself, so that the copies need no barrier; the parameters lie there
// for all rows.  Sixteen columns a thread, in pairs (fp32x2 products): the three
// sums and the addresses cost as much as the columns' arithmetic.
//   u = y r_y, a = scale gate gamma_post, z = x + a u, e = d_x_hat gamma_pre,
//   D = d_x_out + r_z e - z r_z^3 mean(e z),  b = a D,
//   dx = D, dy = r_y (b - u mean(b u)).
enum NormGate { kGScalar = 0, kGChannel = 1, kGFull = 2 };

__device__ __forceinline__ float2 unpack2(uint32_t w) { return make_float2(bf_lo(w), bf_hi(w)); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

template <int GK, int MAXT>
__global__ void __launch_bounds__(MAXT, 512 / MAXT) norm_bwd_staged_kernel(const NormArgs p) {
    constexpr int A = GK == kGFull ? 5 : 4;  // staged rows: x, y, d_x_out, d_x_hat (, gate)
    __shared__ float red[2][32], red2[2][32];
    extern __shared__ __align__(16) uint8_t dyn[];  // [2][A][H] rows; gamma_post, gamma_pre (, gate) [H]
    int sums = 0;
    grid_begin();
    bool ok;
    const int T = row_count(p.d_T, p.T_host, p.T_max, p.hdr, &ok);
    if (!ok) return;
    const int H = p.H, H2 = H * 2;
    const bool post = p.gamma_post != nullptr;
    const int c0 = threadIdx.x * 8, c1 = (blockDim.x + threadIdx.x) * 8;
    const bool in0 = c0 < H, in1 = c1 < H;
    uint8_t* par = dyn + 2 * A * H2;

    auto stage = [&](int t, int buf) {
        if (t < T) {
            const size_t off = static_cast<size_t>(t) * H;
            const bf16* src[5] = {p.x, p.y, p.d_x_out, p.d_x_hat, static_cast<const bf16*>(p.gate)};
            const uint32_t dst = smem_addr(dyn) + buf * A * H2;
#pragma unroll
            for (int a = 0; a < A; ++a) {
                if (in0) cp_async16(dst + a * H2 + c0 * 2, src[a] + off + c0);
                if (in1) cp_async16(dst + a * H2 + c1 * 2, src[a] + off + c1);
            }
        }
        cp_async_commit();
    };
    int buf = 0;
    stage(blockIdx.x, 0);
    // the parameters, 1 for a missing gamma_post
    for (int j = 0; j < 2; ++j) {
        const int c = j ? c1 : c0;
        if (c < H) {
            *reinterpret_cast<uint4*>(par + c * 2) = post ? *reinterpret_cast<const uint4*>(p.gamma_post + c)
                : make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
            *reinterpret_cast<uint4*>(par + H2 + c * 2) = *reinterpret_cast<const uint4*>(p.gamma_pre + c);
            if (GK == kGChannel)
                *reinterpret_cast<uint4*>(par + 2 * H2 + c * 2) =
                    *reinterpret_cast<const uint4*>(static_cast<const bf16*>(p.gate) + c);
        }
    }
    float2 a_post[2][4], a_pre[2][4], a_gate[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) a_post[j][i] = a_pre[j][i] = a_gate[j][i] = both(0.0f);

    for (int t = blockIdx.x; t < T; t += gridDim.x, buf ^= 1) {
        stage(t + gridDim.x, buf ^ 1);  // this thread has read that buffer's last row
        cp_async_wait<1>();
        const uint8_t* rows = dyn + buf * A * H2;
        auto get = [&](const uint8_t* base, int j) -> uint4 {  // zeros past H
            return (j ? in1 : in0) ? *reinterpret_cast<const uint4*>(base + (j ? c1 : c0) * 2) : make_uint4(0, 0, 0, 0);
        };
        auto word = [](const uint4& v, int i) -> uint32_t { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; };
        const float gs = p.scale * (GK == kGScalar && p.gate ? static_cast<const float*>(p.gate)[t] : 1.0f);
        float2 u[2][4], z[2][4];
        float2 ss = both(0.0f);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint4 y = get(rows + H2, j);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                u[j][i] = unpack2(word(y, i));
                ss = __ffma2_rn(u[j][i], u[j][i], ss);
            }
        }
        const float ry = post ? inv_rms(row_sum<true>(ss.x + ss.y, red, sums), p.inv_H, p.eps) : 1.0f;
        float2 zz = both(0.0f), ez = both(0.0f);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint4 x = get(rows, j), dh = get(rows + 3 * H2, j), gp = get(par, j), gr = get(par + H2, j);
            const uint4 g = GK == kGFull ? get(rows + 4 * H2, j) : GK == kGChannel ? get(par + 2 * H2, j) : uint4{};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                u[j][i] = __fmul2_rn(u[j][i], both(ry));
                float2 a = __fmul2_rn(unpack2(word(gp, i)), both(gs));
                if (GK != kGScalar) a = __fmul2_rn(a, unpack2(word(g, i)));
                z[j][i] = __ffma2_rn(a, u[j][i], unpack2(word(x, i)));
                const float2 e = __fmul2_rn(unpack2(word(dh, i)), unpack2(word(gr, i)));
                zz = __ffma2_rn(z[j][i], z[j][i], zz);
                ez = __ffma2_rn(e, z[j][i], ez);
            }
        }
        const float2 za = row_sum2<true>(make_float2(zz.x + zz.y, ez.x + ez.y), red, red2, sums);
        const float rz = inv_rms(za.x, p.inv_H, p.eps);
        const float k2 = za.y * p.inv_H * rz * rz * rz;
        const size_t off = static_cast<size_t>(t) * H;
        float2 bu = both(0.0f), gt = both(0.0f);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint4 dz = get(rows + 2 * H2, j), dh = get(rows + 3 * H2, j), gp = get(par, j), gr = get(par + H2, j);
            const uint4 g = GK == kGFull ? get(rows + 4 * H2, j) : GK == kGChannel ? get(par + 2 * H2, j) : uint4{};
            uint32_t odx[4], odg[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 h = unpack2(word(dh, i)), gp2 = unpack2(word(gp, i));
                const float2 e = __fmul2_rn(h, unpack2(word(gr, i)));
                float2 D = __ffma2_rn(e, both(rz), unpack2(word(dz, i)));
                D = __ffma2_rn(z[j][i], both(-k2), D);
                a_pre[j][i] = __ffma2_rn(h, __fmul2_rn(z[j][i], both(rz)), a_pre[j][i]);
                odx[i] = pack_bf16(D.x, D.y);
                const float2 q = GK == kGScalar ? both(gs) : __fmul2_rn(unpack2(word(g, i)), both(gs));
                const float2 tu = __fmul2_rn(D, u[j][i]);
                a_post[j][i] = __ffma2_rn(q, tu, a_post[j][i]);
                if (GK == kGScalar) gt = __ffma2_rn(gp2, tu, gt);
                if (GK == kGChannel) a_gate[j][i] = __ffma2_rn(gp2, tu, a_gate[j][i]);
                if (GK == kGFull) {
                    const float2 dg = __fmul2_rn(__fmul2_rn(gp2, both(p.scale)), tu);
                    odg[i] = pack_bf16(dg.x, dg.y);
                }
                z[j][i] = __fmul2_rn(__fmul2_rn(q, gp2), D);  // b
                bu = __ffma2_rn(z[j][i], u[j][i], bu);
            }
            if (j ? in1 : in0) {
                *reinterpret_cast<uint4*>(p.dx + off + (j ? c1 : c0)) = make_uint4(odx[0], odx[1], odx[2], odx[3]);
                if (GK == kGFull && p.d_gate_full)
                    *reinterpret_cast<uint4*>(p.d_gate_full + off + (j ? c1 : c0)) = make_uint4(odg[0], odg[1], odg[2], odg[3]);
            }
        }
        float m = 0.0f;
        if (post || p.d_gate_token) {
            const float2 s = row_sum2<true>(make_float2(bu.x + bu.y, gt.x + gt.y), red, red2, sums);
            m = post ? s.x * p.inv_H : 0.0f;
            if (p.d_gate_token && threadIdx.x == 0) p.d_gate_token[t] = s.y * p.scale;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 v = __fmul2_rn(__ffma2_rn(u[j][i], both(-m), z[j][i]), both(ry));
                o[i] = pack_bf16(v.x, v.y);
            }
            if (j ? in1 : in0) *reinterpret_cast<uint4*>(p.dy + off + (j ? c1 : c0)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
    cp_async_wait<0>();
    float* part = p.part + static_cast<size_t>(blockIdx.x) * 3 * H;
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (j ? in1 : in0)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float* o = part + (j ? c1 : c0) + 2 * i;  // H is a multiple of 8: 8-byte aligned
                *reinterpret_cast<float2*>(o) = a_post[j][i];
                *reinterpret_cast<float2*>(o + H) = a_pre[j][i];
                if (GK == kGChannel) *reinterpret_cast<float2*>(o + 2 * H) = __fmul2_rn(a_gate[j][i], both(p.scale));
            }
}

struct NormSumArgs {
    const float* part;
    float* out[3];  // the wanted ones of d_gamma_post, d_gamma_pre, d_gate
    int arr[3];     // which
    int H, parts;
    const int32_t* d_T;
    int T_max;
};

// Column sums of the partial rows: 32 columns x 32 row groups a CTA, so that the
// (L2-resident) loads of a column are in flight together.
__global__ void __launch_bounds__(1024) norm_sum_kernel(const NormSumArgs p) {
    __shared__ float red[32][33];
    grid_begin();
    if (p.d_T && (*p.d_T < 0 || *p.d_T > p.T_max)) return;
    float* out = p.out[blockIdx.y];
    const int arr = p.arr[blockIdx.y];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < p.H)
#pragma unroll 10
        for (int g = grp; g < p.parts; g += 32)
            s += __ldcg(p.part + (static_cast<size_t>(g) * 3 + arr) * p.H + c);
    red[grp][lane] = s;
    __syncthreads();
    s = warp_sum(red[lane][grp]);  // warp grp: its column's 32 groups
    if (lane == 0 && blockIdx.x * 32 + grp < p.H) out[blockIdx.x * 32 + grp] = s;
}

size_t norm_ws_bytes(int T_max, int H) {
    const size_t parts = T_max < kNormParts ? T_max : kNormParts;
    return (kHeaderBytes + parts * 3 * H * sizeof(float) + 255) / 256 * 256;
}

bool norm_shape_ok(int T_max, int H, std::string* why) {
    if (T_max < 1 || T_max > (1 << 24)) { *why = "T_max must be in [1, 2^24]"; return false; }
    if (H < 1 || H > kNormHMax) { *why = "H must be in [1, 16384]"; return false; }
    return true;
}

// Checks what both directions share.
int norm_check(const void* x, const void* y, const void* gamma_post, const void* gate, int gate_kind,
               float scale, const void* gamma_pre, float eps, int T, const int32_t* d_T, int T_max, int H) {
    std::string why;
    if (!norm_shape_ok(T_max, H, &why)) return api_fail(ET_ERR_UNSUPPORTED, why);
    if (!x) return api_fail(ET_ERR_INVALID, "x must be non-NULL");
    if (gate_kind < kGateNone || gate_kind > kGateFull)
        return api_fail(ET_ERR_INVALID, "gate_kind must be in [0, 3]");
    if ((gate_kind == kGateNone) != (gate == nullptr))
        return api_fail(ET_ERR_INVALID, "gate must be given exactly when gate_kind is not 0");
    if (!y && (gamma_post || gate)) return api_fail(ET_ERR_INVALID, "gamma_post and gate need y");
    if (!(eps > 0.0f) || !std::isfinite(eps)) return api_fail(ET_ERR_INVALID, "eps must be > 0 and finite");
    if (!std::isfinite(scale)) return api_fail(ET_ERR_INVALID, "scale must be finite");
    const void* need2[] = {x, y, gamma_post, gamma_pre};
    for (const void* q : need2)
        if (!api_aligned(q, 2)) return api_fail(ET_ERR_INVALID, "tensors must be aligned to their element size");
    if (!api_aligned(gate, gate_kind == kGateToken ? 4 : 2) || !api_aligned(d_T, 4))
        return api_fail(ET_ERR_INVALID, "tensors must be aligned to their element size");
    if (!d_T && (T < 0 || T > T_max)) return api_fail(ET_ERR_INVALID, "T must be in [0, T_max]");
    return ET_OK;
}

// 16-byte accesses: H a multiple of 8 and every bf16 tensor 16-byte aligned.
bool norm_vec(int H, std::initializer_list<const void*> ps) {
    if (H % 8) return false;
    for (const void* q : ps)
        if (!api_aligned(q, 16)) return false;
    return true;
}

// Threads of a row: 16 columns (two vectors) each, 8 for a row of up to 512.
int norm_threads(int H) {
    const int vecs = (H + 7) / 8;
    return ((vecs > 64 ? (vecs + 1) / 2 : vecs) + 31) / 32 * 32;
}

template <bool VEC>
cudaError_t launch_fwd(const NormArgs& a, int rows, int sms, void* stream) {
    if (a.H <= 256) {
        const int warps = rows < 8 ? rows : 8;
        int grid = (rows + warps - 1) / warps;
        grid = grid < 8 * sms ? grid : 8 * sms;
        return api_launch(norm_fwd_kernel<1, VEC, false>, grid, warps * 32, 0, stream, a);
    }
    const int th = norm_threads(a.H);
    const int most = sms * (1024 / th);
    const int grid = rows < most ? rows : most;
    if (a.H <= 512) return api_launch(norm_fwd_kernel<1, VEC, true>, grid, th, 0, stream, a);
    return api_launch(norm_fwd_kernel<2, VEC, true>, grid, th, 0, stream, a);
}

template <int GK, int MAXT>
cudaError_t launch_bwd_staged(const NormArgs& a, int dev, int sms, int threads, int rows, int* parts, void* stream) {
    static SmemOptIn opt;
    // 2 A rows and the parameters: 12 rows at most, 197 KB at H = 8192
    const int smem = (GK == kGFull ? 12 : GK == kGChannel ? 11 : 10) * a.H * static_cast<int>(sizeof(bf16));
    const cudaError_t e = api_smem_opt_in(opt, dev, norm_bwd_staged_kernel<GK, MAXT>, kSmemLimit - 2048);
    if (e != cudaSuccess) return e;
    const int most = sms * (512 / MAXT);
    *parts = *parts < most ? *parts : most;
    return api_launch(norm_bwd_staged_kernel<GK, MAXT>, *parts, threads, smem, stream, a);
}

// The grid is also the number of partial rows that norm_sum_kernel reads.
template <bool VEC>
cudaError_t launch_bwd(const NormArgs& a, int dev, int sms, int rows, int parts_max, int* parts, void* stream) {
    if (a.H <= 256) {
        const int warps = 8;
        const int need = (rows + warps - 1) / warps;
        *parts = need < parts_max ? need : parts_max;
        return api_launch(norm_bwd_kernel<1, VEC, false, 256>, *parts, warps * 32, warps * 768 * sizeof(float),
                          stream, a);
    }
    const int th = norm_threads(a.H);
    *parts = rows < parts_max ? rows : parts_max;
    if (VEC && a.H > 512 && th <= 512 && a.y && a.gamma_pre && a.d_x_out && a.d_x_hat) {
        if (th <= 256) {
            if (a.gate_kind == kGateFull) return launch_bwd_staged<kGFull, 256>(a, dev, sms, th, rows, parts, stream);
            if (a.gate_kind == kGateChannel) return launch_bwd_staged<kGChannel, 256>(a, dev, sms, th, rows, parts, stream);
            return launch_bwd_staged<kGScalar, 256>(a, dev, sms, th, rows, parts, stream);
        }
        if (a.gate_kind == kGateFull) return launch_bwd_staged<kGFull, 512>(a, dev, sms, th, rows, parts, stream);
        if (a.gate_kind == kGateChannel) return launch_bwd_staged<kGChannel, 512>(a, dev, sms, th, rows, parts, stream);
        return launch_bwd_staged<kGScalar, 512>(a, dev, sms, th, rows, parts, stream);
    }
    if (a.H <= 512) return api_launch(norm_bwd_kernel<1, VEC, true, 512>, *parts, th, 0, stream, a);
    if (th <= 512) return api_launch(norm_bwd_kernel<2, VEC, true, 512>, *parts, th, 0, stream, a);
    return api_launch(norm_bwd_kernel<2, VEC, true, 1024>, *parts, th, 0, stream, a);
}

}  // namespace
}  // namespace et

using namespace et;

extern "C" {

size_t et_block_norm_workspace_bytes(int T_max, int H) {
    if (T_max < 1 || T_max > (1 << 24) || H < 1 || H > kNormHMax) return 0;
    return norm_ws_bytes(T_max, H);
}

int et_block_norm(const void* x, const void* y, const void* gamma_post, const void* gate,
                  int gate_kind, float scale, const void* gamma_pre, float eps, void* x_out,
                  void* x_hat, int T, const int32_t* d_T, int T_max, int H, void* workspace,
                  size_t workspace_bytes, void* stream) {
    return api_entry([&]() -> int {
        int rc = norm_check(x, y, gamma_post, gate, gate_kind, scale, gamma_pre, eps, T, d_T, T_max, H);
        if (rc) return rc;
        if (!x_out && !x_hat) return api_fail(ET_ERR_INVALID, "x_out or x_hat must be given");
        if ((x_hat == nullptr) != (gamma_pre == nullptr))
            return api_fail(ET_ERR_INVALID, "x_hat and gamma_pre go together");
        if (!api_aligned(x_out, 2) || !api_aligned(x_hat, 2))
            return api_fail(ET_ERR_INVALID, "tensors must be aligned to their element size");
        if ((rc = api_check_ws(workspace, workspace_bytes, kHeaderBytes))) return rc;
        if (!d_T && T == 0) return ET_OK;
        int dev = 0, sms = 0;
        if ((rc = api_device(&dev, &sms))) return rc;
        NormArgs a{};
        a.x = static_cast<const bf16*>(x);
        a.y = static_cast<const bf16*>(y);
        a.gamma_post = static_cast<const bf16*>(gamma_post);
        a.gate = gate;
        a.gamma_pre = static_cast<const bf16*>(gamma_pre);
        a.scale = scale;
        a.eps = eps;
        a.inv_H = 1.0f / static_cast<float>(H);
        a.gate_kind = gate_kind;
        a.d_T = d_T;
        a.T_host = T;
        a.T_max = T_max;
        a.H = H;
        a.hdr = static_cast<EtHeader*>(workspace);
        a.x_out = static_cast<bf16*>(x_out);
        a.x_hat = static_cast<bf16*>(x_hat);
        const int rows = d_T ? T_max : T;
        const bool vec = norm_vec(H, {x, y, gamma_post, gate_kind == kGateToken ? nullptr : gate,
                                      gamma_pre, x_out, x_hat});
        const cudaError_t e = vec ? launch_fwd<true>(a, rows, sms, stream) : launch_fwd<false>(a, rows, sms, stream);
        if (e != cudaSuccess) return api_fail_cuda(e, "launch of the block norm kernel");
        return ET_OK;
    });
}

int et_block_norm_bwd(const void* x, const void* y, const void* gamma_post, const void* gate,
                      int gate_kind, float scale, const void* gamma_pre, float eps,
                      const void* d_x_out, const void* d_x_hat, void* dx, void* dy,
                      float* d_gamma_post, float* d_gamma_pre, void* d_gate, int T,
                      const int32_t* d_T, int T_max, int H, void* workspace,
                      size_t workspace_bytes, void* stream) {
    return api_entry([&]() -> int {
        int rc = norm_check(x, y, gamma_post, gate, gate_kind, scale, gamma_pre, eps, T, d_T, T_max, H);
        if (rc) return rc;
        if (!dx) return api_fail(ET_ERR_INVALID, "dx must be non-NULL");
        if (!d_x_out && !d_x_hat) return api_fail(ET_ERR_INVALID, "d_x_out or d_x_hat must be given");
        if (d_x_hat && !gamma_pre) return api_fail(ET_ERR_INVALID, "d_x_hat needs gamma_pre");
        if ((y == nullptr) != (dy == nullptr)) return api_fail(ET_ERR_INVALID, "y and dy go together");
        if ((d_gamma_post && !gamma_post) || (d_gamma_pre && !gamma_pre) || (d_gate && !gate))
            return api_fail(ET_ERR_INVALID, "a parameter's gradient needs the parameter");
        const void* need2[] = {d_x_out, d_x_hat, dx, dy};
        for (const void* q : need2)
            if (!api_aligned(q, 2)) return api_fail(ET_ERR_INVALID, "tensors must be aligned to their element size");
        if (!api_aligned(d_gamma_post, 4) || !api_aligned(d_gamma_pre, 4) ||
            !api_aligned(d_gate, gate_kind == kGateFull ? 2 : 4))
            return api_fail(ET_ERR_INVALID, "tensors must be aligned to their element size");
        if ((rc = api_check_ws(workspace, workspace_bytes, norm_ws_bytes(T_max, H)))) return rc;
        int dev = 0, sms = 0;
        if ((rc = api_device(&dev, &sms))) return rc;
        NormArgs a{};
        a.x = static_cast<const bf16*>(x);
        a.y = static_cast<const bf16*>(y);
        a.gamma_post = static_cast<const bf16*>(gamma_post);
        a.gate = gate;
        a.gamma_pre = static_cast<const bf16*>(gamma_pre);
        a.scale = scale;
        a.eps = eps;
        a.inv_H = 1.0f / static_cast<float>(H);
        a.gate_kind = gate_kind;
        a.d_T = d_T;
        a.T_host = T;
        a.T_max = T_max;
        a.H = H;
        a.hdr = static_cast<EtHeader*>(workspace);
        a.d_x_out = static_cast<const bf16*>(d_x_out);
        a.d_x_hat = static_cast<const bf16*>(d_x_hat);
        a.dx = static_cast<bf16*>(dx);
        a.dy = static_cast<bf16*>(dy);
        a.d_gate_full = gate_kind == kGateFull ? static_cast<bf16*>(d_gate) : nullptr;
        a.d_gate_token = gate_kind == kGateToken ? static_cast<float*>(d_gate) : nullptr;
        a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kHeaderBytes);
        const int parts_max = T_max < kNormParts ? T_max : kNormParts;
        const int rows = d_T ? T_max : T;
        int parts = 0;
        if (rows > 0) {
            const bool vec = norm_vec(H, {x, y, gamma_post, gate_kind == kGateToken ? nullptr : gate, gamma_pre,
                                          d_x_out, d_x_hat, dx, dy, a.d_gate_full});
            const cudaError_t e = vec ? launch_bwd<true>(a, dev, sms, rows, parts_max, &parts, stream)
                                      : launch_bwd<false>(a, dev, sms, rows, parts_max, &parts, stream);
            if (e != cudaSuccess) return api_fail_cuda(e, "launch of the block norm's backward kernel");
        }
        float* d_gate_channel = gate_kind == kGateChannel ? static_cast<float*>(d_gate) : nullptr;
        NormSumArgs s{a.part, {}, {}, H, parts, d_T, T_max};
        float* wanted[3] = {d_gamma_post, d_gamma_pre, d_gate_channel};
        int n = 0;
        for (int i = 0; i < 3; ++i)
            if (wanted[i]) {
                s.out[n] = wanted[i];
                s.arr[n++] = i;
            }
        if (n) {
            const cudaError_t e = api_launch(norm_sum_kernel, dim3((H + 31) / 32, n), 1024, 0, stream, s);
            if (e != cudaSuccess) return api_fail_cuda(e, "launch of the block norm's parameter sums");
        }
        return ET_OK;
    });
}

}  // extern "C"
