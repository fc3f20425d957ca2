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
constexpr int kNormChain = 256;  // most rows that a thread adds up where parameter gradients are wanted

struct NormArgs {
    const bf16* x;           // [T, H]
    const bf16* y;           // [T, H] or null (z = x)
    const bf16* gamma_post;  // [H] or null
    const void* gate;        // bf16 [H], fp32 [T], bf16 [T, H] or null
    const bf16* gamma_pre;   // [H] or null
    float scale, eps, inv_H;
    int gate_kind;
    int row_threads;         // threads of a row
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
    int row0, row_end;       // the rows of this launch
    int part_of;             // which parameter gradients are wanted (bit 0 post, 1 pre, 2 gate)
    float* part;             // [kNormParts][3][H]: d_gamma_post, d_gamma_pre, d_gate per channel
};

// Eight consecutive bf16 of a row, packed.
struct Vec8 {
    uint32_t u[4];
    __device__ __forceinline__ float operator[](int i) const {
        return (i & 1) ? bf_hi(u[i >> 1]) : bf_lo(u[i >> 1]);
    }
};

// The threads of a row, and how its columns fall to them.  A CTA holds one row, or
// several with a group of threads (a multiple of a warp) each.  A thread has
// sixteen columns in two vectors of eight.  VEC (H a multiple of 8, tensors
// 16-byte aligned): eight neighbours, one 16-byte access; else columns a group
// apart, so that neighbouring threads still read neighbouring elements.
enum RowMode { kRowsWarp = 0, kRowsGroup = 1, kRowsOne = 2 };  // a row a warp (eight columns a thread
                                                               // are enough), a group, a CTA
template <int MODE>
struct RowGroup {
    int threads, group;  // kRowsGroup only

    __device__ __forceinline__ explicit RowGroup(int row_threads) {
        if (MODE == kRowsGroup) {
            threads = row_threads;
            group = threadIdx.x / row_threads;
        }
    }
    __device__ __forceinline__ int th() const {  // threads of a row
        return MODE == kRowsWarp ? 32 : MODE == kRowsOne ? static_cast<int>(blockDim.x) : threads;
    }
    __device__ __forceinline__ int groups() const {  // rows of the CTA
        return MODE == kRowsOne ? 1 : MODE == kRowsWarp ? static_cast<int>(blockDim.x >> 5) : static_cast<int>(blockDim.x) / threads;
    }
    __device__ __forceinline__ int id() const {  // this thread's row of the CTA,
        return MODE == kRowsOne ? 0 : MODE == kRowsWarp ? static_cast<int>(threadIdx.x >> 5) : group;
    }
    __device__ __forceinline__ int lane() const {  // and its place in it
        return MODE == kRowsOne ? static_cast<int>(threadIdx.x)
             : MODE == kRowsWarp ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x) - group * threads;
    }
    template <bool VEC>
    __device__ __forceinline__ int col(int j, int i) const {
        return VEC ? (j * th() + lane()) * 8 + i : (j * 8 + i) * th() + lane();
    }
    __device__ __forceinline__ void sync() const {
        if (MODE == kRowsOne) __syncthreads();
        else if (MODE == kRowsWarp) __syncwarp();
        else asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(threads) : "memory");
    }
};

constexpr int kNormCtaThreads = 256;  // of a CTA that holds several rows
__host__ __device__ constexpr int norm_v(int mode) { return mode == kRowsWarp ? 1 : 2; }  // vectors of a thread

// This thread's vector j of a row of H columns; zeros past its end.
template <bool VEC, int MODE>
__device__ __forceinline__ Vec8 load8(const bf16* row, const RowGroup<MODE>& g, int j, int H) {
    Vec8 v{};
    if (VEC) {
        const int c = g.template col<VEC>(j, 0);
        if (c < H) {
            const uint4 q = *reinterpret_cast<const uint4*>(row + c);
            v.u[0] = q.x; v.u[1] = q.y; v.u[2] = q.z; v.u[3] = q.w;
        }
    } else {
        const uint16_t* r = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = g.template col<VEC>(j, i);
            if (c < H) v.u[i >> 1] |= static_cast<uint32_t>(r[c]) << (16 * (i & 1));
        }
    }
    return v;
}

template <bool VEC, int MODE>
__device__ __forceinline__ void store8(bf16* row, const RowGroup<MODE>& g, int j, int H, const float* f) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
    if (VEC) {
        const int c = g.template col<VEC>(j, 0);
        if (c < H) *reinterpret_cast<uint4*>(row + c) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
        uint16_t* r = reinterpret_cast<uint16_t*>(row);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = g.template col<VEC>(j, i);
            if (c < H) r[c] = static_cast<uint16_t>(u[i >> 1] >> (16 * (i & 1)));
        }
    }
}

// One or two sums over the row's threads, the same bits in every one of them.
// Consecutive sums alternate between two slots of `red` (n counts them), so one
// barrier a sum is enough: who has passed the next sum's barrier knows that all
// have read this one.
template <int MODE>
__device__ __forceinline__ float row_sum(float v, float (*red)[32], const RowGroup<MODE>& g, int& n) {
    v = warp_sum(v);
    if (MODE != kRowsWarp) {
        const int slot = n++ & 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int first = g.id() * (g.th() >> 5);
        if (lane == 0) red[slot][warp] = v;
        g.sync();
        v = warp_sum(lane < (g.th() >> 5) ? red[slot][first + lane] : 0.0f);
    }
    return v;
}
template <int MODE>
__device__ __forceinline__ float2 row_sum2(float2 v, float (*red)[32], float (*red2)[32], const RowGroup<MODE>& g, int& n) {
    v.x = warp_sum(v.x);
    v.y = warp_sum(v.y);
    if (MODE != kRowsWarp) {
        const int slot = n++ & 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int first = g.id() * (g.th() >> 5);
        if (lane == 0) { red[slot][warp] = v.x; red2[slot][warp] = v.y; }
        g.sync();
        const bool in = lane < (g.th() >> 5);
        v.x = warp_sum(in ? red[slot][first + lane] : 0.0f);
        v.y = warp_sum(in ? red2[slot][first + lane] : 0.0f);
    }
    return v;
}

// 1 / sqrt(sum / H + eps)
__device__ __forceinline__ float inv_rms(float sum, float inv_H, float eps) { return rsqrtf(sum * inv_H + eps); }

// Bound by HBM: every load of a row goes out before its first sum, and many rows
// are in flight on an SM (T = H = 4096 with a full gate, 168 MB: 26 us, 95 % of
// the measured copy rate).
template <bool VEC, int MODE>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(const NormArgs p) {
    constexpr int V = norm_v(MODE);
    __shared__ float red[2][32];
    int n_sums = 0;
    const RowGroup<MODE> g(p.row_threads);
    grid_begin();
    bool ok;
    const int T = row_count(p.d_T, p.T_host, p.T_max, p.hdr, &ok);
    const int H = p.H;
    for (int t = blockIdx.x * g.groups() + g.id(); t < T; t += gridDim.x * g.groups()) {
        const size_t off = static_cast<size_t>(t) * H;
        float z[V][8];
        Vec8 yv[V], gv[V];
        float ss = 0.0f;
        const bool vec_gate = p.gate_kind == kGateFull || p.gate_kind == kGateChannel;
        const bf16* grow = static_cast<const bf16*>(p.gate) + (p.gate_kind == kGateFull ? off : 0);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const Vec8 xv = load8<VEC>(p.x + off, g, j, H);
            yv[j] = p.y ? load8<VEC>(p.y + off, g, j, H) : Vec8{};
            gv[j] = vec_gate ? load8<VEC>(grow, g, j, H) : Vec8{};
#pragma unroll
            for (int i = 0; i < 8; ++i) z[j][i] = xv[i];
        }
        const float gtok = p.gate_kind == kGateToken ? static_cast<const float*>(p.gate)[t] : 1.0f;
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) ss += yv[j][i] * yv[j][i];
        float ry = 1.0f;
        if (p.y && p.gamma_post) ry = inv_rms(row_sum(ss, red, g, n_sums), p.inv_H, p.eps);
        float zz = 0.0f;
        const float gs = p.scale * gtok;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (p.y) {
                const Vec8 gp = p.gamma_post ? load8<VEC>(p.gamma_post, g, j, H) : Vec8{};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float n = p.gamma_post ? yv[j][i] * ry * gp[i] : yv[j][i];
                    z[j][i] += (vec_gate ? gs * gv[j][i] : gs) * n;  // 0 past H, where y is 0
                }
            }
            if (p.x_out) store8<VEC>(p.x_out + off, g, j, H, z[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) zz += z[j][i] * z[j][i];
        }
        if (p.x_hat) {
            const float rz = inv_rms(row_sum(zz, red, g, n_sums), p.inv_H, p.eps);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const Vec8 gp = load8<VEC>(p.gamma_pre, g, j, H);
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = z[j][i] * rz * gp[i];
                store8<VEC>(p.x_hat + off, g, j, H, o);
            }
        }
    }
}

// The parameter gradients of a CTA: its row groups' sums added up in order and
// stored as this CTA's row of partial sums (those that are wanted).
// get(arr, j, i): this thread's sum.
template <bool VEC, int MODE, class F>
__device__ __forceinline__ void store_part(const NormArgs& p, const RowGroup<MODE>& g, float* smem, F&& get) {
    const int H = p.H;
    float* part = p.part + static_cast<size_t>(blockIdx.x) * 3 * H;
    float* to = MODE == kRowsOne || g.groups() == 1 ? part : smem + static_cast<size_t>(g.id()) * 3 * H;
    if (MODE != kRowsOne) __syncthreads();  // what else lies there has been read
#pragma unroll
    for (int arr = 0; arr < 3; ++arr)
        if (p.part_of >> arr & 1)
#pragma unroll
            for (int j = 0; j < norm_v(MODE); ++j) {
                if (VEC) {
                    const int c = g.template col<VEC>(j, 0);
                    if (c < H) {
                        float4* o = reinterpret_cast<float4*>(to + arr * H + c);
                        o[0] = make_float4(get(arr, j, 0), get(arr, j, 1), get(arr, j, 2), get(arr, j, 3));
                        o[1] = make_float4(get(arr, j, 4), get(arr, j, 5), get(arr, j, 6), get(arr, j, 7));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int c = g.template col<VEC>(j, i);
                        if (c < H) to[arr * H + c] = get(arr, j, i);
                    }
                }
            }
    if (MODE != kRowsOne && g.groups() > 1) {
        __syncthreads();
        for (int o = threadIdx.x; o < 3 * H; o += blockDim.x) {
            float s = 0.0f;
            if (p.part_of >> (o / H) & 1)
                for (int k = 0; k < g.groups(); ++k) s += smem[static_cast<size_t>(k) * 3 * H + o];
            part[o] = s;
        }
    }
}

// The gradient.  A row's statistics are recomputed from x and y (they are read
// anyway).  The parameter gradients are summed over this CTA's rows in
// registers, thread by thread for its own columns, then over its row groups and
// over CTAs (norm_sum_kernel) in a fixed order.  Three sums a row: mean y^2;
// mean z^2 with the second norm's projection; the first norm's projection (with
// a per-token gate's gradient).
//
// This form serves every H, alignment and combination of the optional parts;
// norm_bwd_staged_kernel the usual one.  MAXT: most threads, which bounds the
// registers.  Bound by its loads' latency, which only the other warps of the SM
// hide (T = 1000, H = 16384 with a full gate, 262 MB: 138 us, 1.9 TB/s; such rows
// do not fit shared memory twice).
template <bool VEC, int MODE, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? 2 : 1) norm_bwd_kernel(const NormArgs p) {
    constexpr int V = norm_v(MODE);
    __shared__ float red[2][32], red2[2][32];
    extern __shared__ __align__(16) uint8_t dyn[];  // [groups][3][H] floats
    int n_sums = 0;
    const RowGroup<MODE> g(p.row_threads);
    grid_begin();
    bool ok;
    const int T = min(row_count(p.d_T, p.T_host, p.T_max, p.hdr, &ok), p.row_end);
    if (!ok) return;
    const int H = p.H;
    const bool post = p.y && p.gamma_post;
    const bool full = p.gate_kind == kGateFull;
    float a_post[V][8], a_pre[V][8], a_gate[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) a_post[j][i] = a_pre[j][i] = a_gate[j][i] = 0.0f;
    auto row8 = [&](const bf16* base, size_t off, int j) -> Vec8 {  // zeros where it is not given
        return base ? load8<VEC>(base + off, g, j, H) : Vec8{};
    };

    for (int t = p.row0 + blockIdx.x * g.groups() + g.id(); t < T; t += gridDim.x * g.groups()) {
        const size_t off = static_cast<size_t>(t) * H;
        const float gs = p.scale * (p.gate_kind == kGateToken ? static_cast<const float*>(p.gate)[t] : 1.0f);
        auto gate_of = [&](int j, float* q) {  // scale * gate of vector j
            if (full || p.gate_kind == kGateChannel) {
                const Vec8 v = row8(static_cast<const bf16*>(p.gate), full ? off : 0, j);
#pragma unroll
                for (int i = 0; i < 8; ++i) q[i] = gs * v[i];
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) q[i] = gs;
            }
        };
        Vec8 xv[V], yv[V], dz[V], dh[V];
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            xv[j] = row8(p.x, off, j);
            yv[j] = row8(p.y, off, j);
            dz[j] = row8(p.d_x_out, off, j);
            dh[j] = row8(p.d_x_hat, off, j);
#pragma unroll
            for (int i = 0; i < 8; ++i) ss += yv[j][i] * yv[j][i];
        }
        float ry = 1.0f;
        if (post) ry = inv_rms(row_sum(ss, red, g, n_sums), p.inv_H, p.eps);
        // z, and with it the statistics of the second norm and sum(d_x_hat gamma_pre z)
        float z[V][8];
        float2 za = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < V; ++j) {
#pragma unroll
            for (int i = 0; i < 8; ++i) z[j][i] = xv[j][i];
            if (p.y) {
                float q[8];
                gate_of(j, q);
                const Vec8 gp = post ? row8(p.gamma_post, 0, j) : Vec8{};
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    z[j][i] += q[i] * (post ? yv[j][i] * ry * gp[i] : yv[j][i]);  // 0 past H, where y is 0
            }
            if (p.d_x_hat) {
                const Vec8 gr = row8(p.gamma_pre, 0, j);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    za.x += z[j][i] * z[j][i];
                    za.y += dh[j][i] * gr[i] * z[j][i];
                }
            }
        }
        float rz = 0.0f, k2 = 0.0f;
        if (p.d_x_hat) {
            za = row_sum2(za, red, red2, g, n_sums);
            rz = inv_rms(za.x, p.inv_H, p.eps);
            k2 = za.y * p.inv_H * rz * rz * rz;
        }
        // d z, the parameter gradients, and sum(d n gamma_post y)
        float2 bg = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float d[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = dz[j][i];
            if (p.d_x_hat) {
                const Vec8 gr = row8(p.gamma_pre, 0, j);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    d[i] += rz * (dh[j][i] * gr[i]) - z[j][i] * k2;
                    a_pre[j][i] += dh[j][i] * (z[j][i] * rz);
                }
            }
            store8<VEC>(p.dx + off, g, j, H, d);
            if (p.y) {
                float q[8], dgf[8];
                gate_of(j, q);
                const Vec8 gp = post ? row8(p.gamma_post, 0, j) : Vec8{};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float u = yv[j][i] * ry;  // the normalised value
                    dgf[i] = p.scale * (post ? u * gp[i] : yv[j][i]) * d[i];
                    d[i] *= q[i];  // d n
                    a_post[j][i] += d[i] * u;
                    if (post) {
                        d[i] *= gp[i];
                        bg.x += d[i] * yv[j][i];
                    }
                    a_gate[j][i] += dgf[i];
                    bg.y += dgf[i];
                    z[j][i] = d[i];
                }
                if (p.d_gate_full) store8<VEC>(p.d_gate_full + off, g, j, H, dgf);
            }
        }
        if (p.y) {
            if (post || p.d_gate_token) bg = row_sum2(bg, red, red2, g, n_sums);
            const float k1 = post ? bg.x * p.inv_H * ry * ry * ry : 0.0f;
            if (p.d_gate_token && g.lane() == 0) p.d_gate_token[t] = bg.y;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = post ? ry * z[j][i] - yv[j][i] * k1 : z[j][i];
                store8<VEC>(p.dy + off, g, j, H, o);
            }
        }
    }
    store_part<VEC>(p, g, reinterpret_cast<float*>(dyn),
                    [&](int arr, int j, int i) { return arr == 0 ? a_post[j][i] : arr == 1 ? a_pre[j][i] : a_gate[j][i]; });
}

// The same gradient where y, gamma_pre and both incoming gradients are given and H
// is at most 8192.
//
// Bound by HBM (T = H = 4096 with a full gate, 268 MB: 45 us, 88 % of the measured
// copy rate) if a row's latencies are hidden: the input rows of this CTA's next row are copied to shared memory
// while the current one is worked on, each thread reading back only what it
// copied itself, so that the copies need no barrier; the parameters lie there
// for all rows.  Without VEC (see RowGroup) a row is copied by the 16-byte pieces
// that hold it -- the first of a tensor element by element, the last cut to its
// end, so that nothing outside is read -- and read back by element, with a
// barrier on either side.  Sixteen columns a thread, in pairs (fp32x2 products): the three
// sums and the addresses cost as much as the columns' arithmetic.
//   u = y r_y, a = scale gate gamma_post, z = x + a u, e = d_x_hat gamma_pre,
//   D = d_x_out + r_z e - z r_z^3 mean(e z),  b = a D,
//   dx = D, dy = r_y (b - u mean(b u)).
enum NormGate { kGScalar = 0, kGChannel = 1, kGFull = 2 };

__device__ __forceinline__ float2 unpack2(uint32_t w) { return make_float2(bf_lo(w), bf_hi(w)); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Bytes of a staged row: without VEC it starts anywhere in its first 16-byte piece.
__host__ __device__ constexpr int norm_row_bytes(int H, bool vec) { return vec ? H * 2 : (H * 2 + 29) / 16 * 16; }

template <bool VEC, int GK, int MODE, int MAXT>
__global__ void __launch_bounds__(MAXT, 512 / MAXT) norm_bwd_staged_kernel(const NormArgs p) {
    constexpr int V = norm_v(MODE);
    constexpr int A = GK == kGFull ? 5 : 4;  // staged rows: x, y, d_x_out, d_x_hat (, gate)
    __shared__ float red[2][32], red2[2][32];
    // [groups][2][A] rows; gamma_post, gamma_pre (, gate), each thread's own 16 values
    // together; at the end [groups][3][H] floats
    extern __shared__ __align__(16) uint8_t dyn[];
    int n_sums = 0;
    const RowGroup<MODE> grp(p.row_threads);
    grid_begin();
    bool ok;
    const int T = min(row_count(p.d_T, p.T_host, p.T_max, p.hdr, &ok), p.row_end);
    if (!ok) return;
    const int H = p.H, H2 = H * 2;
    const bool post = p.gamma_post != nullptr;
    const int row_b = norm_row_bytes(H, VEC), par_b = grp.th() * V * 16;  // bytes of a staged row, of a parameter
    const int c0 = grp.template col<true>(0, 0), c1 = grp.template col<true>(1, 0);
    const bool in0 = c0 < H, in1 = V > 1 && c1 < H;  // VEC only
    uint8_t* mine = dyn + static_cast<size_t>(grp.id()) * 2 * A * row_b;
    uint8_t* par = dyn + static_cast<size_t>(grp.groups()) * 2 * A * row_b + grp.lane() * 16;

    auto source = [&](int a) -> const bf16* {
        return a == 0 ? p.x : a == 1 ? p.y : a == 2 ? p.d_x_out : a == 3 ? p.d_x_hat : static_cast<const bf16*>(p.gate);
    };
    auto stage = [&](int t, int buf) {
        if (t < T) {
            const size_t off = static_cast<size_t>(t) * H;
            const uint32_t dst = smem_addr(mine) + buf * A * row_b;
#pragma unroll
            for (int a = 0; a < A; ++a) {
                if (VEC) {
                    if (in0) cp_async16(dst + a * row_b + c0 * 2, source(a) + off + c0);
                    if (in1) cp_async16(dst + a * row_b + c1 * 2, source(a) + off + c1);
                } else {
                    const uint8_t* base = reinterpret_cast<const uint8_t*>(source(a));
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
    const int t0 = p.row0 + blockIdx.x * grp.groups() + grp.id(), step = gridDim.x * grp.groups();
    stage(t0, 0);
    // the parameters, 1 for a missing gamma_post; every thread reads back what it wrote
    // (the groups write the same)
#pragma unroll
    for (int j = 0; j < V; ++j) {
        auto put = [&](int a, const bf16* src) {
            const Vec8 v = src ? load8<VEC>(src, grp, j, H) : Vec8{{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u}};
            *reinterpret_cast<uint4*>(par + a * par_b + j * grp.th() * 16) = make_uint4(v.u[0], v.u[1], v.u[2], v.u[3]);
        };
        put(0, p.gamma_post);
        put(1, p.gamma_pre);
        if (GK == kGChannel) put(2, static_cast<const bf16*>(p.gate));
    }
    float2 a_post[V][4], a_pre[V][4], a_gate[V][4];
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) a_post[j][i] = a_pre[j][i] = a_gate[j][i] = both(0.0f);

    for (int t = t0; t < T; t += step, buf ^= 1) {
        stage(t + step, buf ^ 1);  // this thread has read that buffer's last row
        cp_async_wait<1>();
        if (!VEC) grp.sync();  // the other threads' pieces
        const uint8_t* rows = mine + buf * A * row_b;
        const size_t off = static_cast<size_t>(t) * H;
        auto get = [&](int a, int j) -> uint4 {  // vector j of staged row a; zeros past H
            if (VEC) return (j ? in1 : in0) ? *reinterpret_cast<const uint4*>(rows + a * row_b + (j ? c1 : c0) * 2) : make_uint4(0, 0, 0, 0);
            const uint16_t* r = reinterpret_cast<const uint16_t*>(rows + a * row_b + (reinterpret_cast<uintptr_t>(source(a) + off) & 15));
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int lo = grp.template col<VEC>(j, 2 * i), hi = grp.template col<VEC>(j, 2 * i + 1);
                w[i] = (lo < H ? r[lo] : 0u) | (hi < H ? static_cast<uint32_t>(r[hi]) << 16 : 0u);
            }
            return make_uint4(w[0], w[1], w[2], w[3]);
        };
        auto param = [&](int a, int j) -> uint4 { return *reinterpret_cast<const uint4*>(par + a * par_b + j * grp.th() * 16); };
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
        const float gs = p.scale * (GK == kGScalar && p.gate ? static_cast<const float*>(p.gate)[t] : 1.0f);
        float2 u[V][4], z[V][4];
        float2 ss = both(0.0f);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint4 y = get(1, j);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                u[j][i] = unpack2(word(y, i));
                ss = __ffma2_rn(u[j][i], u[j][i], ss);
            }
        }
        const float ry = post ? inv_rms(row_sum(ss.x + ss.y, red, grp, n_sums), p.inv_H, p.eps) : 1.0f;
        float2 zz = both(0.0f), ez = both(0.0f);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint4 x = get(0, j), dh = get(3, j), gp = param(0, j), gr = param(1, j);
            const uint4 g = GK == kGFull ? get(4, j) : GK == kGChannel ? param(2, j) : uint4{};
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
        const float2 za = row_sum2(make_float2(zz.x + zz.y, ez.x + ez.y), red, red2, grp, n_sums);
        const float rz = inv_rms(za.x, p.inv_H, p.eps);
        const float k2 = za.y * p.inv_H * rz * rz * rz;
        float2 bu = both(0.0f), gt = both(0.0f);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint4 dz = get(2, j), dh = get(3, j), gp = param(0, j), gr = param(1, j);
            const uint4 g = GK == kGFull ? get(4, j) : GK == kGChannel ? param(2, j) : uint4{};
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
            put_row(p.dx, j, odx);
            if (GK == kGFull && p.d_gate_full) put_row(p.d_gate_full, j, odg);
        }
        float m = 0.0f;
        if (post || p.d_gate_token) {
            const float2 s = row_sum2(make_float2(bu.x + bu.y, gt.x + gt.y), red, red2, grp, n_sums);
            m = post ? s.x * p.inv_H : 0.0f;
            if (p.d_gate_token && grp.lane() == 0) p.d_gate_token[t] = s.y * p.scale;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 v = __fmul2_rn(__ffma2_rn(u[j][i], both(-m), z[j][i]), both(ry));
                o[i] = pack_bf16(v.x, v.y);
            }
            put_row(p.dy, j, o);
        }
        if (!VEC) grp.sync();  // this buffer is copied to again
    }
    cp_async_wait<0>();
    store_part<VEC>(p, grp, reinterpret_cast<float*>(dyn), [&](int arr, int j, int i) {
        const float2 v = arr == 0 ? a_post[j][i >> 1] : arr == 1 ? a_pre[j][i >> 1] : a_gate[j][i >> 1];
        return (i & 1 ? v.y : v.x) * (arr == 2 ? p.scale : 1.0f);
    });
}

struct NormSumArgs {
    const float* part;
    float* out[3];  // the wanted ones of d_gamma_post, d_gamma_pre, d_gate
    int arr[3];     // which
    int H, parts;
    const int32_t* d_T;
    int T_max;
    bool add;       // to what an earlier launch of the call has put there
};

// Column sums of the partial rows: 32 columns x 32 row groups a CTA, so that the
// (L2-resident) loads of a column are in flight together.  Two sums of 304 rows of
// 4096: 10 MB, 10.7 to 11.4 us by itself with cold caches.  Half as many rows, from CTAs
// of 512 threads with two rows each, cost more there than they saved here (forward,
// backward and this, T = H = 4096: 83 us, then 93).
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
    if (lane == 0 && blockIdx.x * 32 + grp < p.H) {
        float* o = out + blockIdx.x * 32 + grp;
        *o = p.add ? *o + s : s;
    }
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

// Threads of a row: sixteen columns each.
int norm_threads(int H) { return ((H + 15) / 16 + 31) / 32 * 32; }

// Rows of a CTA: as many as make 256 threads.  With fewer, a small H left most of
// an SM idle (forward and backward, T = 4096, H = 512: 62 us, with eight rows 20).
int norm_groups(int threads, int rows) {
    const int g = threads < kNormCtaThreads ? kNormCtaThreads / threads : 1;
    return g < rows ? g : rows;
}

RowMode norm_mode(int H, int threads) {
    return H <= 256 ? kRowsWarp : 2 * threads <= kNormCtaThreads ? kRowsGroup : kRowsOne;
}

template <bool VEC>
cudaError_t launch_fwd(NormArgs a, int rows, int sms, void* stream) {
    a.row_threads = norm_threads(a.H);
    const RowMode mode = norm_mode(a.H, a.row_threads);
    const int groups = norm_groups(a.row_threads, rows), th = a.row_threads * groups;
    const int need = (rows + groups - 1) / groups, most = sms * (1024 / th);
    const int grid = need < most ? need : most;
    return api_launch(mode == kRowsWarp ? norm_fwd_kernel<VEC, kRowsWarp> : mode == kRowsGroup ? norm_fwd_kernel<VEC, kRowsGroup>
                                                                          : norm_fwd_kernel<VEC, kRowsOne>,
                      grid, th, 0, stream, a);
}

struct NormLaunch {
    int dev, sms, rows, parts_max;
    int* parts;
    void* stream;
};

// The grid is also the number of partial rows that norm_sum_kernel reads: two CTAs
// an SM of up to 256 threads (128 registers each), else one.
template <class K>
cudaError_t launch_bwd_rows(SmemOptIn& opt, K kernel, const NormArgs& a, const NormLaunch& l, int smem_row, int smem_cta) {
    const cudaError_t e = api_smem_opt_in(opt, l.dev, kernel, kSmemLimit - 2048);
    if (e != cudaSuccess) return e;
    const int groups = norm_groups(a.row_threads, l.rows), th = a.row_threads * groups;
    const int need = (l.rows + groups - 1) / groups, most = th <= kNormCtaThreads ? 2 * l.sms : l.sms;
    int n = need < l.parts_max ? need : l.parts_max;
    *l.parts = n = n < most ? n : most;
    // the rows of a CTA, then (at the end) its groups' sums
    const int staged = groups * smem_row + smem_cta, merge = groups > 1 ? groups * 3 * a.H * 4 : 0;
    return api_launch(kernel, n, th, staged > merge ? staged : merge, l.stream, a);
}

template <bool VEC, int GK>
cudaError_t launch_bwd_staged(const NormArgs& a, RowMode mode, const NormLaunch& l) {
    static SmemOptIn opt[4];
    constexpr int A = GK == kGFull ? 5 : 4;
    const int row = 2 * A * norm_row_bytes(a.H, VEC);                        // 197 KB at most,
    const int par = (GK == kGChannel ? 3 : 2) * a.row_threads * norm_v(mode) * 16;  // with these
    if (mode == kRowsWarp) return launch_bwd_rows(opt[0], norm_bwd_staged_kernel<VEC, GK, kRowsWarp, 256>, a, l, row, par);
    if (mode == kRowsGroup) return launch_bwd_rows(opt[1], norm_bwd_staged_kernel<VEC, GK, kRowsGroup, 256>, a, l, row, par);
    if (a.row_threads <= 256) return launch_bwd_rows(opt[2], norm_bwd_staged_kernel<VEC, GK, kRowsOne, 256>, a, l, row, par);
    return launch_bwd_rows(opt[3], norm_bwd_staged_kernel<VEC, GK, kRowsOne, 512>, a, l, row, par);
}

template <bool VEC>
cudaError_t launch_bwd(NormArgs a, const NormLaunch& l) {
    a.row_threads = norm_threads(a.H);
    const RowMode mode = norm_mode(a.H, a.row_threads);
    if (a.row_threads <= 512 && a.y && a.gamma_pre && a.d_x_out && a.d_x_hat) {
        if (a.gate_kind == kGateFull) return launch_bwd_staged<VEC, kGFull>(a, mode, l);
        if (a.gate_kind == kGateChannel) return launch_bwd_staged<VEC, kGChannel>(a, mode, l);
        return launch_bwd_staged<VEC, kGScalar>(a, mode, l);
    }
    static SmemOptIn opt[5];
    if (mode == kRowsWarp) return launch_bwd_rows(opt[0], norm_bwd_kernel<VEC, kRowsWarp, 256>, a, l, 0, 0);
    if (mode == kRowsGroup) return launch_bwd_rows(opt[1], norm_bwd_kernel<VEC, kRowsGroup, 256>, a, l, 0, 0);
    if (a.row_threads <= 256) return launch_bwd_rows(opt[2], norm_bwd_kernel<VEC, kRowsOne, 256>, a, l, 0, 0);
    if (a.row_threads <= 512) return launch_bwd_rows(opt[3], norm_bwd_kernel<VEC, kRowsOne, 512>, a, l, 0, 0);
    return launch_bwd_rows(opt[4], norm_bwd_kernel<VEC, kRowsOne, 1024>, a, l, 0, 0);
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
        a.part_of = (d_gamma_post ? 1 : 0) | (d_gamma_pre ? 2 : 0) | (gate_kind == kGateChannel && d_gate ? 4 : 0);
        const int parts_max = T_max < kNormParts ? T_max : kNormParts;
        const int rows = d_T ? T_max : T;
        const bool vec = norm_vec(H, {x, y, gamma_post, gate_kind == kGateToken ? nullptr : gate, gamma_pre,
                                      d_x_out, d_x_hat, dx, dy, a.d_gate_full});
        NormSumArgs s{a.part, {}, {}, H, 0, d_T, T_max, false};
        float* wanted[3] = {d_gamma_post, d_gamma_pre, gate_kind == kGateChannel ? static_cast<float*>(d_gate) : nullptr};
        int n = 0;
        for (int i = 0; i < 3; ++i)
            if (wanted[i]) {
                s.out[n] = wanted[i];
                s.arr[n++] = i;
            }
        // Parameter gradients: launches of as many rows as leave no thread with more than
        // kNormChain to add up, each adding its sums to the ones before.  One chain for all
        // rows would lose up to 2^-24 of the sum with each (500000 equal rows of H = 2056:
        // off by 400 x 2^-24).  A launch takes 0.5 ms or more then, its sums 0.01.
        const int groups = norm_groups(norm_threads(H), rows);
        const int ctas = norm_threads(H) * groups <= kNormCtaThreads ? kNormParts : kNormParts / 2;
        const int most = n ? kNormChain * ctas * groups : rows;
        for (int row0 = 0; row0 < rows || row0 == 0; row0 += most) {
            a.row0 = row0;
            a.row_end = rows - row0 < most ? rows : row0 + most;
            s.add = row0 > 0;
            if (rows > 0) {
                const NormLaunch l{dev, sms, a.row_end - row0, parts_max, &s.parts, stream};
                const cudaError_t e = vec ? launch_bwd<true>(a, l) : launch_bwd<false>(a, l);
                if (e != cudaSuccess) return api_fail_cuda(e, "launch of the block norm's backward kernel");
            }
            if (n) {
                const cudaError_t e = api_launch(norm_sum_kernel, dim3((H + 31) / 32, n), 1024, 0, stream, s);
                if (e != cudaSuccess) return api_fail_cuda(e, "launch of the block norm's parameter sums");
            }
            if (rows == 0) break;
        }
        return ET_OK;
    });
}

}  // extern "C"
