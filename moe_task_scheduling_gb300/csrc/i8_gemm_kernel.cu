// i8_gemm_kernel.cu -- Y = (s_x s_w^T) * (x_q w_q^T) on the tensor cores.
//
// GB300's integer tensor rate is far below its 16-bit rate, but every int8 value is
// an fp16 value and a product of two of them is exact in fp32: the products run as
// tcgen05 kind::f16 with fp32 sums, exact while those stay within 2^24.  The tokens
// are written as fp16 once a call (i8_expand_kernel; they are few or the product is
// long).  The weights, which are the traffic of a small batch, stay int8 up to the SM:
// converter warps turn each 128 x 128 block into fp16 in TMEM, where the MMA takes its
// A operand from, so that shared memory carries a weight once, as one byte.
//
// Roles (608 threads):
//   warp 0        weights: TMA, int8 blocks of 128 channels x 128 k
//   warp 1        one thread issues tcgen05.mma, D[channel, token] += W X^T
//   warps 2..9    converters: shared memory -> registers -> fp16 -> TMEM; a thread has
//                 half a row
//   warps 10..17  epilogue: TMEM -> scales -> bf16, or a part's sums to the workspace; four
//                 take the even 16-token chunks, four the odd ones
//   warp 18       tokens: TMA, fp16 blocks of tn tokens x 128 k
// With CG = 2 a pair of CTAs takes 256 channels: each loads and converts its own 128,
// loads half the tokens, and the pair's MMA reads both halves, which halves the
// traffic of the tokens into shared memory.
//
// Work: tiles of 128 CG channels x tn tokens.  With many tiles a CTA takes whole ones in
// turn; with few (share) the k-blocks of all tiles are one list, cut into even ranges,
// and a tile that several CTAs have a part of is summed in the order of k by the one
// that stores its part last: the same bits on every run.  Every wait is bounded.
#include <cuda_fp16.h>

#include "et_device.cuh"
#include "i8_gemm.h"
#include "ops_device.cuh"

namespace et {
namespace {

constexpr int kI8Threads = 608;
constexpr int kConvWarp0 = 2, kConvWarps = 8, kEpiWarpI8 = 10, kEpiWarps = 8, kTokenWarp = 18;
constexpr int kAStages = 4;          // TMEM blocks of converted weights, 64 columns each
constexpr int kACol = 256;           // the accumulators are columns 0 .. 255
constexpr int kWBytes = 128 * kI8KBlock;
constexpr int kEpiBar = 1;           // named barrier of the epilogue warps

struct I8Ctl {
    uint64_t full_w[kI8MaxStages], empty_w[kI8MaxStages];
    uint64_t full_x[kI8MaxStages], empty_x[kI8MaxStages];
    uint64_t full_a[kAStages], empty_a[kAStages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int32_t go[2];                   // the epilogue's: the accumulator is complete (0: an abort),
    int32_t last;                    // this part was the tile's last
    alignas(16) float sx[2][kI8TokensMax];
};

// ---------------------------------------------------------------- PTX that et_device.cuh has for one CTA

template <int CG>
__device__ __forceinline__ uint32_t leader_addr(const void* p) {  // of this variable in the pair's first CTA
    uint32_t a = smem_u32(p);
    if (CG == 2) asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
    return a;
}

// (Without .cluster scope, which would make every arrival wait for this SM's stores and
// every wait drop its L1: what the barriers order is in TMEM and in the async proxy.)
template <int CG>
__device__ __forceinline__ void arrive_leader(uint64_t* bar) {
    if (CG == 1) mbar_arrive(bar);
    else asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(leader_addr<2>(bar)) : "memory");
}

// mbar_wait (bounded) that polls for longer before it sleeps.
__device__ __forceinline__ bool wait(const WaitCtx& c, uint64_t* bar, uint32_t parity, int where) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if (it > 1024) __nanosleep(64);
        if ((it & 63u) == 0) {
            if (aborted(c)) return false;
            if (globaltimer_ns() - t0 > c.timeout_ns) {
                raise_error(c, ET_ERR_TIMEOUT, where);
                return false;
            }
        }
    }
}

template <int CG>
__device__ __forceinline__ void tma_tokens(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
    if (CG == 1)
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
                     "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
                     : "memory");
    else  // the barrier may be the pair's other CTA's
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
                     "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
                     : "memory");
}

template <int CG>
__device__ __forceinline__ void mma_f16(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    if (CG == 1)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
                     : "memory");
}

// Arrive on `bar` (of both CTAs of a pair) once every MMA issued so far is done.
template <int CG>
__device__ __forceinline__ void commit(uint64_t* bar) {
    if (CG == 1)
        tc_commit(bar);
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
                     "h"(static_cast<uint16_t>(3))
                     : "memory");
}

// True in one lane of a converged warp, the same every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

template <int CG>
__device__ __forceinline__ void tmem_take(uint32_t* slot) {
    if (CG == 1) {
        tmem_alloc(slot, 512);
        tmem_relinquish();
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t taddr) {
    if (CG == 1) tmem_dealloc(taddr, 512);
    else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(taddr) : "memory");
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// 32 registers to 32 columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
        "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Four int8 of a word as two pairs of fp16, exact: with the sign bits turned over a byte is
// x + 128, 0x6400 | b is 1024 + b in fp16, and 1152 less is x.
__device__ __forceinline__ void int8_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
    w ^= 0x80808080u;
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off), y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
}

// A thread's values of up to 16 tokens, a row of `to` each.  The whole sixteen go out
// without a branch between them.
template <class V>
__device__ __forceinline__ void store16(V* to, size_t row, const V (&v)[16], int left) {
    if (left >= 16) {
#pragma unroll
        for (int c = 0; c < 16; ++c) to[c * row] = v[c];
    } else {
#pragma unroll
        for (int c = 0; c < 16; ++c)
            if (c < left) to[c * row] = v[c];
    }
}

// ---------------------------------------------------------------- work

// The rows of this pass.  A device count out of range is recorded and taken as none.
__device__ __forceinline__ int pass_rows(const I8Rows& r, EtHeader* hdr) {
    if (!r.d_M) return r.count;
    const int M = *reinterpret_cast<const volatile int32_t*>(r.d_M);
    if (M < 0 || M > r.call_max) {
        if (threadIdx.x == 0 && blockIdx.x == 0) record_status(hdr, ET_ERR_BOUNDS, kWhereBoundsT);
        return 0;
    }
    return max(0, min(r.count, M - r.first));
}

// A CTA's (pair's) next piece: k-blocks [kb0, kb1) of a tile.
struct Piece {
    int tile, kb0, kb1;
};

struct Work {
    long long total, at, end;  // share: of the list of all tiles' k-blocks
    int grid;                  // CTAs that have some of it (the device's M may leave less than one each)
    int tile, tiles, step;
    int kblocks, share;

    // The list's first k-block of CTA b.
    __device__ __forceinline__ long long first(int b) const { return total * b / grid; }
    // The CTA that has k-block x of the list.
    __device__ __forceinline__ int owner(long long x) const { return static_cast<int>(((x + 1) * grid - 1) / total); }
    __device__ __forceinline__ Work(const I8TcArgs& p, int tiles_, int b) : tiles(tiles_), kblocks(p.kblocks), share(p.share) {
        total = static_cast<long long>(tiles) * kblocks;
        grid = total < p.grid ? static_cast<int>(total) : p.grid;
        at = b < grid ? first(b) : 0;
        end = b < grid ? first(b + 1) : 0;
        tile = b;
        step = p.grid;
    }
    __device__ __forceinline__ bool next(Piece& w) {
        if (share) {
            if (at >= end) return false;
            w.tile = static_cast<int>(at / kblocks);
            w.kb0 = static_cast<int>(at - static_cast<long long>(w.tile) * kblocks);
            const long long n = end - at;
            w.kb1 = n < kblocks - w.kb0 ? w.kb0 + static_cast<int>(n) : kblocks;
            at += w.kb1 - w.kb0;
            return true;
        }
        if (tile >= tiles) return false;
        w = {tile, 0, kblocks};
        tile += step;
        return true;
    }
};

template <int CG>
__global__ void __launch_bounds__(kI8Threads, 1)
i8_tc_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ I8TcArgs p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int xrows = p.tn / CG, xbytes = xrows * 256;  // a stage of tokens: two boxes of 64 k
    uint8_t* ring_w = base;
    uint8_t* ring_x = base + p.stages_w * kWBytes;
    I8Ctl* ctl = reinterpret_cast<I8Ctl*>(ring_x + p.stages_x * xbytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0;
    const int cta = blockIdx.x / CG;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kI8MaxStages; ++i) {
            mbar_init(&ctl->full_w[i], 1);
            mbar_init(&ctl->empty_w[i], kConvWarps);
            mbar_init(&ctl->full_x[i], 1);
            mbar_init(&ctl->empty_x[i], 1);
        }
        for (int i = 0; i < kAStages; ++i) {
            mbar_init(&ctl->full_a[i], kConvWarps * CG);
            mbar_init(&ctl->empty_a[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->acc_full[i], 1);
            mbar_init(&ctl->acc_empty[i], kEpiWarps * CG);
        }
        mbar_init(&ctl->drain, 1);
        fence_mbar_init();
        tma_prefetch_map(&tm_w);
        tma_prefetch_map(&tm_x);
    }
    if (warp == 1) tmem_take<CG>(&ctl->tmem_base);
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();
    tc_fence_after();
    grid_release();

    const WaitCtx wc{p.hdr, p.timeout_ns};
    const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem_base, 0);
    if (p.rows.d_M) grid_wait();
    const int M = pass_rows(p.rows, p.hdr);
    const int mt = ceil_div(M, p.tn), tiles = mt * p.nt;  // tile = n tile * mt + m tile
    const int slots = p.tn > 128 ? 1 : 2;                 // accumulators
    uint32_t posted_w = 0, posted_x = 0;
    Work work(p, tiles, cta);
    Piece w;

    if (warp == 0) {
        if (lane == 0) {
            // May start before what comes before this kernel ends: that is the call's own
            // first kernel, which lets this one start only when all before it has ended.
            const uint64_t pol = policy_evict_first();
            bool ok = true;
            while (ok && work.next(w)) {
                const int n0 = (w.tile / mt) * 128 * CG + static_cast<int>(rank) * 128;
                for (int kb = w.kb0; kb < w.kb1; ++kb) {
                    const uint32_t s = posted_w % p.stages_w;
                    if (!(ok = wait(wc, &ctl->empty_w[s], ((posted_w / p.stages_w) & 1u) ^ 1u, kWhereEmpty))) break;
                    mbar_arrive_expect_tx(&ctl->full_w[s], kWBytes);
                    tma_load_2d(ring_w + s * kWBytes, &tm_w, &ctl->full_w[s], kb * kI8KBlock, n0, pol);
                    ++posted_w;
                }
            }
            if (!ok)  // unwinding: let the copies land
                for (uint32_t i = posted_w > static_cast<uint32_t>(p.stages_w) ? posted_w - p.stages_w : 0; i < posted_w; ++i)
                    mbar_drain(&ctl->full_w[i % p.stages_w], (i / p.stages_w) & 1u, 1000000ull);
        }
        __syncwarp();
    } else if (warp == kTokenWarp) {
        if (lane == 0) {
            grid_wait();
            fence_proxy_async_global();  // the first kernel's stores, read by TMA
            bool ok = true;
            while (ok && work.next(w)) {
                const int m0 = (w.tile % mt) * p.tn + static_cast<int>(rank) * xrows;
                for (int kb = w.kb0; kb < w.kb1; ++kb) {
                    const uint32_t s = posted_x % p.stages_x;
                    if (!(ok = wait(wc, &ctl->empty_x[s], ((posted_x / p.stages_x) & 1u) ^ 1u, kWhereEmpty))) break;
                    if (rank == 0) mbar_arrive_expect_tx(&ctl->full_x[s], xbytes * CG);
                    const uint32_t bar = leader_addr<CG>(&ctl->full_x[s]), dst = smem_u32(ring_x + s * xbytes);
                    tma_tokens<CG>(dst, &tm_x, bar, kb * kI8KBlock, m0);
                    tma_tokens<CG>(dst + xrows * 128, &tm_x, bar, kb * kI8KBlock + 64, m0);
                    ++posted_x;
                }
            }
            if (!ok && rank == 0)
                for (uint32_t i = posted_x > static_cast<uint32_t>(p.stages_x) ? posted_x - p.stages_x : 0; i < posted_x; ++i)
                    mbar_drain(&ctl->full_x[i % p.stages_x], (i / p.stages_x) & 1u, 1000000ull);
        }
        __syncwarp();
    } else if (warp == 1) {
        // The whole warp walks the work and one elected lane issues: descriptors and addresses
        // are then uniform, which an MMA takes 37 cycles to issue with; from a branch on the
        // lane it took 100, more than a tile of few tokens computes for.
        if (rank == 0) {
            // D fp32, A and B fp16, both K-major
            const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(p.tn >> 3) << 17) | (static_cast<uint32_t>(128 * CG >> 4) << 24);
            uint32_t acc = 0, kx = 0, px = 0, ka = 0, pa = 0;  // ring places and their phases
            bool ok = true;
            while (ok && work.next(w)) {
                const uint32_t slot = slots == 1 ? 0 : acc & 1, turn = slots == 1 ? acc : acc >> 1;
                ok = wait(wc, &ctl->acc_empty[slot], (turn & 1u) ^ 1u, kWhereAcc);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                const uint32_t d = tmem + slot * 128;
                for (int kb = w.kb0; kb < w.kb1; ++kb) {
                    ok = wait(wc, &ctl->full_x[kx], px, kWhereFull) && wait(wc, &ctl->full_a[ka], pa, kWhereFull);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    tc_fence_after();
                    const uint64_t b0 = sdesc_sw128(smem_u32(ring_x + kx * xbytes)), b1 = b0 + (xrows * 128 >> 4);
                    const uint32_t a = tmem + kACol + ka * 64;
                    if (elect_one()) {
                        mma_f16<CG>(d, a, b0, idesc, kb > w.kb0 ? 1u : 0u);
#pragma unroll
                        for (int k = 1; k < kI8KBlock / 16; ++k)  // 16 k are 32 bytes of a row of 64 k
                            mma_f16<CG>(d, a + k * 8, (k < 4 ? b0 : b1) + (k & 3) * 2, idesc, 1u);
                        commit<CG>(&ctl->empty_x[kx]);
                        commit<CG>(&ctl->empty_a[ka]);
                    }
                    __syncwarp();
                    if (++kx == static_cast<uint32_t>(p.stages_x)) { kx = 0; px ^= 1u; }
                    if (++ka == kAStages) { ka = 0; pa ^= 1u; }
                }
                if (!ok) break;
                if (elect_one()) commit<CG>(&ctl->acc_full[slot]);
                __syncwarp();
                ++acc;
            }
            if (elect_one()) commit<CG>(&ctl->drain);  // every arrival above has come when this one has
        }
        __syncwarp();
    } else if (warp < kEpiWarpI8) {
        const int q = warp & 3, half = (warp - kConvWarp0) >> 2, r = q * 32 + lane;
        const uint32_t row = static_cast<uint32_t>(r) * 128, x7 = r & 7;
        const uint32_t a0 = tmem + kACol + half * 32 + (static_cast<uint32_t>(q * 32) << 16);
        uint32_t it = 0;
        bool ok = true;
        while (ok && work.next(w)) {
            for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
                const uint32_t sw = it % p.stages_w, sa = it % kAStages;
                ok = wait(wc, &ctl->full_w[sw], (it / p.stages_w) & 1u, kWhereFull);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                const uint32_t src = smem_u32(ring_w + sw * kWBytes) + row;
                uint4 v[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = lds_v4(src + (((half * 4 + c) ^ x7) << 4));
                uint32_t h[32];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    int8_to_half(v[c].x, h[c * 8 + 0], h[c * 8 + 1]);
                    int8_to_half(v[c].y, h[c * 8 + 2], h[c * 8 + 3]);
                    int8_to_half(v[c].z, h[c * 8 + 4], h[c * 8 + 5]);
                    int8_to_half(v[c].w, h[c * 8 + 6], h[c * 8 + 7]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->empty_w[sw]);
                ok = wait(wc, &ctl->empty_a[sa], ((it / kAStages) & 1u) ^ 1u, kWhereEmpty);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                tc_fence_after();
                tmem_st32(a0 + sa * 64, h);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_leader<CG>(&ctl->full_a[sa]);
            }
        }
    } else {
        const int q = warp & 3, odd = (warp - kEpiWarpI8) >> 2, et = threadIdx.x - kEpiWarpI8 * 32, row = q * 32 + lane;
        constexpr int kChannels = 128 * CG;
        grid_wait();
        uint32_t acc = 0;
        bool ok = true;
        while (ok && work.next(w)) {
            const uint32_t slot = acc % slots;
            const int m0 = (w.tile % mt) * p.tn, n = (w.tile / mt) * kChannels + static_cast<int>(rank) * 128 + row;
            const int rows = min(p.tn, M - m0);
            float* sx = ctl->sx[acc & 1];
            for (int m = et; m < rows; m += kEpiWarps * 32) sx[m] = p.sx[m0 + m];
            const float sw = n < p.N ? p.sw[n] : 0.0f;
            // one thread waits for all four warps: a named barrier is not bounded, so they must
            // never part
            if (et == 0) ctl->go[acc & 1] = wait(wc, &ctl->acc_full[slot], (acc / slots) & 1u, kWhereAcc);
            named_bar_sync(kEpiBar, kEpiWarps * 32);
            if (!(ok = ctl->go[acc & 1] != 0)) break;
            tc_fence_after();
            const bool part = w.kb1 - w.kb0 != p.kblocks;
            // a part that begins its tile, or the CTA's range: one of each at most
            float* mine = p.part + ((static_cast<size_t>(cta) * 2 + (w.kb0 == 0)) * p.tn) * kChannels + rank * 128 + row;
            bf16* y = p.y + static_cast<size_t>(m0) * p.N + n;
            const uint32_t d = tmem + slot * 128 + (static_cast<uint32_t>(q * 32) << 16);
            for (int c0 = odd * 16; c0 < rows; c0 += 32) {
                float v[16];
                tmem_ld16(d + c0, v);
                tmem_ld_wait();
                const int left = rows - c0;
                if (part) {
                    store16(mine + static_cast<size_t>(c0) * kChannels, kChannels, v, left);
                } else if (n < p.N) {
                    bf16 o[16];
#pragma unroll
                    for (int c = 0; c < 16; c += 4) {
                        const float4 f = *reinterpret_cast<const float4*>(sx + c0 + c);
                        o[c] = __float2bfloat16_rn(v[c] * (f.x * sw));
                        o[c + 1] = __float2bfloat16_rn(v[c + 1] * (f.y * sw));
                        o[c + 2] = __float2bfloat16_rn(v[c + 2] * (f.z * sw));
                        o[c + 3] = __float2bfloat16_rn(v[c + 3] * (f.w * sw));
                    }
                    store16(y + static_cast<size_t>(c0) * p.N, p.N, o, left);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_leader<CG>(&ctl->acc_empty[slot]);
            ++acc;
            if (part) {
                const long long t0 = static_cast<long long>(w.tile) * p.kblocks;
                const int b0 = work.owner(t0), b1 = work.owner(t0 + p.kblocks - 1);
                // both CTAs of a pair count their own half of the channels
                int* count = p.tile_count + w.tile * CG + rank;
                named_bar_sync(kEpiBar, kEpiWarps * 32);
                if (et == 0) {
                    __threadfence();
                    ctl->last = atom_acq_rel_add(count, 1) == b1 - b0;
                }
                named_bar_sync(kEpiBar, kEpiWarps * 32);
                if (ctl->last) {
                    __threadfence();
                    const float* from = p.part + rank * 128 + row;
                    for (int c0 = odd * 8; c0 < rows; c0 += 16) {
                        float s[8];
#pragma unroll
                        for (int c = 0; c < 8; ++c) s[c] = 0.0f;
                        for (int b = b0; b <= b1; b += 4) {  // in the order of k, four parts' loads in flight
                            float v[4][8];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int begins = work.first(b + i) <= t0;
                                const float* f = from + ((static_cast<size_t>(b + i) * 2 + begins) * p.tn + c0) * kChannels;
#pragma unroll
                                for (int c = 0; c < 8; ++c) v[i][c] = b + i <= b1 ? __ldcg(f + c * kChannels) : 0.0f;
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i)
#pragma unroll
                                for (int c = 0; c < 8; ++c) s[c] += v[i][c];
                        }
                        if (n < p.N)
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                if (c0 + c < rows) y[static_cast<size_t>(c0 + c) * p.N] = __float2bfloat16_rn(s[c] * (sx[c0 + c] * sw));
                    }
                }
                named_bar_sync(kEpiBar, kEpiWarps * 32);  // `last` is written again
            }
        }
    }

    __syncthreads();
    // the pair's commits have arrived here, and no CTA goes while the other may still reach into it
    if (threadIdx.x == 32 && (CG == 2 || rank == 0)) (void)mbar_drain(&ctl->drain, 0, 2000000ull);
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();
    tc_fence_after();
    if (warp == 1) tmem_free<CG>(tmem);
}

__global__ void __launch_bounds__(256) i8_expand_kernel(const I8ExpandArgs p) {
    // In this order: the product's kernel may start when every CTA has come past the second,
    // so all that came before this call is complete by then.
    grid_wait();
    grid_release();
    const int at = blockIdx.x * blockDim.x + threadIdx.x, step = gridDim.x * blockDim.x;
    for (int i = at; i < p.tiles; i += step) p.tile_count[i] = 0;
    if (at == 0) p.hdr->abort = 0;
    const int M = pass_rows(p.rows, p.hdr);
    const long long n = static_cast<long long>(M) * p.K / 16;
    const uint4* x = reinterpret_cast<const uint4*>(p.x);
    uint4* out = static_cast<uint4*>(p.x16);
    for (long long i = at; i < n; i += step) {
        const uint4 v = x[i];
        uint4 a, b;
        int8_to_half(v.x, a.x, a.y);
        int8_to_half(v.y, a.z, a.w);
        int8_to_half(v.z, b.x, b.y);
        int8_to_half(v.w, b.z, b.w);
        out[2 * i] = a;
        out[2 * i + 1] = b;
    }
}

constexpr int kCtlBytes = (static_cast<int>(sizeof(I8Ctl)) + 127) / 128 * 128;

}  // namespace

// Weights first: a few 16 KB blocks more in flight matter to a small batch, whose
// tokens need little; never less than two stages of either.
int i8_tc_stages(bool pair, int tn, int* w, int* x) {
    const int xbytes = tn / (pair ? 2 : 1) * 256, room = kSmemLimit - 1024 - kCtlBytes;
    *x = xbytes > 32768 ? 2 : xbytes > 16384 ? 4 : xbytes > 8192 ? 5 : 8;
    *w = (room - *x * xbytes) / kWBytes;
    if (*w > kI8MaxStages) *w = kI8MaxStages;
    return 1024 + kCtlBytes + *w * kWBytes + *x * xbytes;
}

cudaError_t launch_i8_tc(const I8TcArgs& a, const CUtensorMap* map_w, const CUtensorMap* map_x, bool pair, int dev, void* stream) {
    static bool done[2][64] = {};
    int w, x;
    const int smem = i8_tc_stages(pair, a.tn, &w, &x);
    auto kernel = pair ? i8_tc_kernel<2> : i8_tc_kernel<1>;
    if (!__atomic_load_n(&done[pair][dev], __ATOMIC_ACQUIRE)) {
        const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
        if (e != cudaSuccess) return e;
        __atomic_store_n(&done[pair][dev], true, __ATOMIC_RELEASE);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.grid * (pair ? 2 : 1));
    cfg.blockDim = dim3(kI8Threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = pair ? 2 : 1;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, *map_w, *map_x, a);
}

cudaError_t launch_i8_expand(const I8ExpandArgs& a, int sms, void* stream) {
    cudaLaunchConfig_t cfg{};
    const long long n = (static_cast<long long>(a.rows.count) * a.K / 16 + 255) / 256;
    cfg.gridDim = dim3(static_cast<unsigned>(n < 1 ? 1 : n < 8ll * sms ? n : 8ll * sms));
    cfg.blockDim = dim3(256);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, i8_expand_kernel, a);
}

}  // namespace et
