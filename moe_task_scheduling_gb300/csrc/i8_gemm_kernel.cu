// i8_gemm_kernel.cu -- Y = (s_x s_w^T) * (x_q w_q^T) on the tensor cores.
//
// GB300's integer tensor rate is far below its 16-bit rate, but every int8 value is
// an fp16 value and a product of two of them is exact in fp32: the products run as
// tcgen05 kind::f16 with fp32 sums, exact while those stay within 2^24.  The weights,
// which are the traffic of a small batch, stay int8 up to the SM: converter warps turn
// each block of 128 channels x 128 k into fp16 in TMEM, where the MMA takes its A operand
// from, so that shared memory carries a weight once, as one byte.
//
// Roles (608 threads):
//   warp 0        weights: TMA, int8 blocks of 128 channels x 128 k
//   warp 1        one elected thread issues tcgen05.mma, D[channel, token] += W X^T
//   warps 2..9    converters: shared memory -> registers -> fp16 -> TMEM, a thread a row;
//                 four warps take the even blocks, four the odd ones
//   warps 10..17  tokens of one CTA's tile: int8 from memory -> fp16 in shared memory;
//                 and the epilogue: TMEM -> scales -> bf16
//   warp 18       tokens of a pair: TMA, fp16 blocks
// A pair of CTAs (CG = 2) takes 256 channels: each loads and converts its own 128 and
// loads half the tokens, and the pair's MMA reads both halves, which halves the traffic of
// the tokens into shared memory.  Its tokens come as fp16, written once a call by
// i8_expand_kernel: with a batch that long they are read by many pairs.
//
// Work: tiles of 128 CG channels x tn tokens, whole ones in turn.  Where tiles are few a
// cluster of `split` CTAs or pairs takes one, each its share of k; their sums meet in shared
// memory over the cluster and are added in the order of k: the same bits on every run.
// Every wait is bounded.
//
// What bounds it: few tokens the weights' conversion, 560 cycles a block of 16 KB where HBM
// brings one in 700, on those SMs that have a tile (M = 32, 14336 x 4096: 15.6 us, 112 of 152
// SMs, 3.8 TB/s with 6 us before and after); many tokens the tensor cores (M = 4096, 14336 x
// 4096: 260 us, 1.85 PFLOP/s, 96 % of a bf16 library product's burst; at 2048 x 4096 x 4096 the
// tensor pipe is busy for 75 % of the kernel, the rest is the last tiles' epilogue and the
// pipeline's start).
#include "et_api.h"
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
constexpr int kEpiThreads = kEpiWarps * 32;

struct I8Ctl {
    uint64_t full_w[kI8MaxStages], empty_w[kI8MaxStages];
    uint64_t full_x[kI8MaxStages], empty_x[kI8MaxStages];
    uint64_t full_a[kAStages], empty_a[kAStages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t drain;
    uint32_t posted_w, posted_x[2];  // stages that copies were posted for: weights; tokens by either CTA of a pair
    int32_t gave_up;                 // a wait of this CTA ran out
    uint32_t tmem_base;
    int32_t go[2];                   // the epilogue's: the accumulator is complete (0: an abort)
    alignas(16) float sx[2][kI8TokensMax];
};

// ---------------------------------------------------------------- PTX that et_device.cuh has for one CTA

__device__ __forceinline__ uint32_t leader_addr(const void* p, uint32_t cta) {  // of this variable in the pair's first CTA
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(cta & ~1u));
    return a;
}

// (Without .cluster scope, which would make every arrival wait for this SM's stores and
// every wait drop its L1: what the barriers order is in TMEM and in the async proxy.)
template <int CG>
__device__ __forceinline__ void arrive_leader(uint64_t* bar, uint32_t cta) {
    if (CG == 1) mbar_arrive(bar);
    else asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(leader_addr(bar, cta)) : "memory");
}

struct I8Wait {
    EtHeader* hdr;
    uint64_t timeout_ns;
    int32_t* gave_up;
};

// mbar_wait (bounded) that polls for longer before it sleeps, and whose time alone ends it:
// every role of a CTA whose wait ran out sees its own run out too, and no flag in memory has
// to be taken back when the kernel ends (0.5 us of a small product).
__device__ __forceinline__ bool wait(const I8Wait& c, uint64_t* bar, uint32_t parity, int where) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if (it > 1024) __nanosleep(64);
        if ((it & 63u) == 0 && globaltimer_ns() - t0 > c.timeout_ns) {
            record_status(c.hdr, ET_ERR_TIMEOUT, where);
            *c.gave_up = 1;
            return false;
        }
    }
}

// A pair's tokens: `bar` is the first CTA's, which counts both CTAs' copies.
__device__ __forceinline__ void tma_tokens(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
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
__device__ __forceinline__ void commit(uint64_t* bar, uint32_t cta) {
    if (CG == 1)
        tc_commit(bar);
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
                     "h"(static_cast<uint16_t>(3u << (cta & ~1u)))
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
__device__ __forceinline__ void sts_v4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

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

// A CTA's (pair's) pieces: k-blocks [kb0, kb1) of a tile.
struct Work {
    int tile, kb0, kb1;
    int at, tiles, step;

    __device__ __forceinline__ Work(const I8TcArgs& p, int tiles_, int cta) : tiles(tiles_) {
        const int part = cta % p.split;
        at = cta / p.split;
        step = p.split > 1 ? tiles_ : p.grid;  // a cluster has one tile
        kb0 = p.kblocks * part / p.split;
        kb1 = p.kblocks * (part + 1) / p.split;
    }
    __device__ __forceinline__ bool next() {
        if (at >= tiles) return false;
        tile = at;
        at += step;
        return true;
    }
};

// The tokens of a tile's k-blocks, by the 256 threads of the epilogue: int8 from memory (a
// row of 128 bytes by eight neighbouring threads), as fp16 into the swizzled blocks of 64 k
// that the MMA reads.  C: 16-byte chunks of a thread in a block; AHEAD: blocks that are on
// their way from L2 in registers, which takes longer than the MMAs of a block of few tokens.
template <int C, int AHEAD>
__device__ __forceinline__ bool load_tokens(const I8TcArgs& p, I8Ctl* ctl, uint8_t* ring, const I8Wait& wc, int m0, int rows,
                                            int kb0, int kb1, int et, int lane, uint32_t& s, uint32_t& phase) {
    const int chunk = et & 7, row0 = et >> 3, xbytes = p.tn * 256;
    const int8_t* x = p.x + static_cast<size_t>(m0) * p.K + chunk * 16;
    uint4 v[AHEAD][C];
    auto fetch = [&](uint4 (&to)[C], int kb) {
        const int k = kb * kI8KBlock;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int r = row0 + i * (kEpiThreads / 8);
            to[i] = make_uint4(0, 0, 0, 0);
            if (kb < kb1 && r < rows && k + chunk * 16 < p.K) to[i] = *reinterpret_cast<const uint4*>(x + static_cast<size_t>(r) * p.K + k);
        }
    };
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) fetch(v[j], kb0 + j);
    for (int kb = kb0; kb < kb1; kb += AHEAD) {
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            if (kb + j >= kb1) break;
            const bool ok = wait(wc, &ctl->empty_x[s], phase ^ 1u, kWhereEmpty);
            if (!__all_sync(0xffffffffu, ok)) return false;
            const uint32_t dst = smem_u32(ring + s * xbytes) + (chunk >> 2) * p.tn * 128;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int r = row0 + i * (kEpiThreads / 8);
                if (r < p.tn) {
                    uint32_t h[8];
                    int8_to_half(v[j][i].x, h[0], h[1]);
                    int8_to_half(v[j][i].y, h[2], h[3]);
                    int8_to_half(v[j][i].z, h[4], h[5]);
                    int8_to_half(v[j][i].w, h[6], h[7]);
                    const uint32_t at = dst + r * 128, c = (chunk & 3) * 2;
                    sts_v4(at + ((c ^ (r & 7)) << 4), h[0], h[1], h[2], h[3]);
                    sts_v4(at + (((c + 1) ^ (r & 7)) << 4), h[4], h[5], h[6], h[7]);
                }
            }
            fetch(v[j], kb + j + AHEAD);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->full_x[s]);
            if (++s == static_cast<uint32_t>(p.stages_x)) { s = 0; phase ^= 1u; }
        }
    }
    return true;
}

template <int CG>
__global__ void __launch_bounds__(kI8Threads, 1)
i8_tc_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ I8TcArgs p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int xrows = p.tn / CG, xbytes = xrows * 256;  // a stage of tokens: two blocks of 64 k
    uint8_t* ring_w = base;
    uint8_t* ring_x = base + p.stages_w * kWBytes;
    I8Ctl* ctl = reinterpret_cast<I8Ctl*>(ring_x + p.stages_x * xbytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t crank = cluster_rank(), rank = CG == 2 ? crank & 1u : 0;  // in the cluster, in the pair
    if (threadIdx.x == 0) {
        for (int i = 0; i < kI8MaxStages; ++i) {
            mbar_init(&ctl->full_w[i], 1);
            mbar_init(&ctl->empty_w[i], kConvWarps / 2);
            mbar_init(&ctl->full_x[i], CG == 1 ? kEpiWarps : 1);
            mbar_init(&ctl->empty_x[i], 1);
        }
        for (int i = 0; i < kAStages; ++i) {
            mbar_init(&ctl->full_a[i], kConvWarps / 2 * CG);
            mbar_init(&ctl->empty_a[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->acc_full[i], 1);
            mbar_init(&ctl->acc_empty[i], kEpiWarps * CG);
        }
        mbar_init(&ctl->drain, 1);
        ctl->gave_up = 0;
        fence_mbar_init();
        tma_prefetch_map(&tm_w);
        if (CG == 2) tma_prefetch_map(&tm_x);
    }
    if (warp == 1) tmem_take<CG>(&ctl->tmem_base);
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();
    tc_fence_after();
    grid_release();

    const I8Wait wc{p.hdr, p.timeout_ns, &ctl->gave_up};
    const uint32_t tmem = __shfl_sync(0xffffffffu, ctl->tmem_base, 0);
    if (p.rows.d_M) grid_wait();
    const int M = pass_rows(p.rows, p.hdr);
    const int mt = ceil_div(M, p.tn), tiles = mt * p.nt;  // tile = n tile * mt + m tile
    const int slots = p.tn > 128 ? 1 : 2;                 // accumulators
    Work w(p, tiles, blockIdx.x / CG);
    // Nothing else is read before what comes before this kernel has ended (for a pair that is
    // the call's own first kernel, which has waited for the rest): an early start shows this
    // kernel nothing of that, the wait does.  The first blocks of weights may be on their way
    // to L2 by then.  Every role waits, so that the limit of its own waits runs in this
    // kernel's time and not in an earlier one's, however long that goes on.
    if (threadIdx.x == 0) {
        Work f = w;
        if (f.next())
            for (int kb = f.kb0; kb < f.kb1 && kb < f.kb0 + p.stages_w; ++kb)
                tma_prefetch_l2(&tm_w, kb * kI8KBlock, (f.tile / mt) * 128 * CG + static_cast<int>(rank) * 128);
    }
    grid_wait();

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol = policy_evict_first();
            fence_proxy_async_global();  // weights that a kernel wrote, read by TMA
            uint32_t s = 0, phase = 0, posted = 0;
            bool ok = static_cast<int>(blockIdx.x) != p.fault_cta;
            while (ok && w.next()) {
                const int n0 = (w.tile / mt) * 128 * CG + static_cast<int>(rank) * 128;
                for (int kb = w.kb0; kb < w.kb1; ++kb) {
                    if (!(ok = wait(wc, &ctl->empty_w[s], phase ^ 1u, kWhereEmpty))) break;
                    mbar_arrive_expect_tx(&ctl->full_w[s], kWBytes);
                    tma_load_2d(ring_w + s * kWBytes, &tm_w, &ctl->full_w[s], kb * kI8KBlock, n0, pol);
                    ++posted;
                    if (++s == static_cast<uint32_t>(p.stages_w)) { s = 0; phase ^= 1u; }
                }
            }
            ctl->posted_w = posted;
        }
        __syncwarp();
    } else if (warp == kTokenWarp) {
        if (CG == 2 && lane == 0) {
            fence_proxy_async_global();  // the first kernel's stores, read by TMA
            uint32_t s = 0, phase = 0, posted = 0;
            bool ok = true;
            while (ok && w.next()) {
                const int m0 = (w.tile % mt) * p.tn + static_cast<int>(rank) * xrows;
                for (int kb = w.kb0; kb < w.kb1; ++kb) {
                    if (!(ok = wait(wc, &ctl->empty_x[s], phase ^ 1u, kWhereEmpty))) break;
                    if (rank == 0) mbar_arrive_expect_tx(&ctl->full_x[s], xbytes * CG);
                    const uint32_t bar = leader_addr(&ctl->full_x[s], crank), dst = smem_u32(ring_x + s * xbytes);
                    tma_tokens(dst, &tm_x, bar, kb * kI8KBlock, m0);
                    tma_tokens(dst + xrows * 128, &tm_x, bar, kb * kI8KBlock + 64, m0);
                    ++posted;
                    if (++s == static_cast<uint32_t>(p.stages_x)) { s = 0; phase ^= 1u; }
                }
            }
            ctl->posted_x[rank] = posted;
            uint32_t other;
            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(other) : "r"(smem_u32(&ctl->posted_x[rank])), "r"(crank ^ 1u));
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(other), "r"(posted) : "memory");
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
            while (ok && w.next()) {
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
                        commit<CG>(&ctl->empty_x[kx], crank);
                        commit<CG>(&ctl->empty_a[ka], crank);
                    }
                    __syncwarp();
                    if (++kx == static_cast<uint32_t>(p.stages_x)) { kx = 0; px ^= 1u; }
                    if (++ka == kAStages) { ka = 0; pa ^= 1u; }
                }
                if (!ok) break;
                if (elect_one()) commit<CG>(&ctl->acc_full[slot], crank);
                __syncwarp();
                ++acc;
            }
            if (elect_one()) commit<CG>(&ctl->drain, crank);  // every arrival above has come when this one has
        }
        __syncwarp();
    } else if (warp < kEpiWarpI8) {
        const int q = warp & 3, group = (warp - kConvWarp0) >> 2, r = q * 32 + lane;
        const uint32_t row = static_cast<uint32_t>(r) * 128, x7 = r & 7;
        const uint32_t a0 = tmem + kACol + (static_cast<uint32_t>(q * 32) << 16);
        uint32_t it = 0, s = 0, phase = 0;
        bool ok = true;
        while (ok && w.next()) {
            for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
                if ((it & 1u) == static_cast<uint32_t>(group)) {
                    const uint32_t sa = it % kAStages;
                    ok = wait(wc, &ctl->full_w[s], phase, kWhereFull);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    const uint32_t src = smem_u32(ring_w + s * kWBytes) + row;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
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
                        if (!half) {
                            ok = wait(wc, &ctl->empty_a[sa], ((it / kAStages) & 1u) ^ 1u, kWhereEmpty);
                            if (!(ok = __all_sync(0xffffffffu, ok))) break;
                            tc_fence_after();
                        }
                        tmem_st32(a0 + sa * 64 + half * 32, h);
                    }
                    if (!ok) break;
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    // Both only now.  An arrival on empty_w right after the loads came before them: they
                    // queue behind the first store to TMEM, and the next block was in their place.
                    if (lane == 0) {
                        mbar_arrive(&ctl->empty_w[s]);
                        arrive_leader<CG>(&ctl->full_a[sa], crank);
                    }
                }
                if (++s == static_cast<uint32_t>(p.stages_w)) { s = 0; phase ^= 1u; }
            }
        }
    } else {
        const int q = warp & 3, odd = (warp - kEpiWarpI8) >> 2, et = threadIdx.x - kEpiWarpI8 * 32, row = q * 32 + lane;
        uint32_t acc = 0, s = 0, phase = 0;
        bool ok = true;
        while (ok && w.next()) {
            const uint32_t slot = slots == 1 ? 0 : acc & 1, turn = slots == 1 ? acc : acc >> 1;
            const int m0 = (w.tile % mt) * p.tn, n = (w.tile / mt) * 128 * CG + static_cast<int>(rank) * 128 + row;
            const int rows = min(p.tn, M - m0);
            float* sx = ctl->sx[acc & 1];
            for (int m = et; m < rows; m += kEpiThreads) sx[m] = p.sx[m0 + m];
            const float sw = n < p.N ? p.sw[n] : 0.0f;
            if (CG == 1) {
                if (p.tn <= 32) ok = load_tokens<1, 6>(p, ctl, ring_x, wc, m0, rows, w.kb0, w.kb1, et, lane, s, phase);
                else if (p.tn <= 64) ok = load_tokens<2, 4>(p, ctl, ring_x, wc, m0, rows, w.kb0, w.kb1, et, lane, s, phase);
                else if (p.tn <= 128) ok = load_tokens<4, 2>(p, ctl, ring_x, wc, m0, rows, w.kb0, w.kb1, et, lane, s, phase);
                else ok = load_tokens<8, 1>(p, ctl, ring_x, wc, m0, rows, w.kb0, w.kb1, et, lane, s, phase);
            }
            // One thread waits for all eight warps: a named barrier is not bounded, so they must
            // never part.
            if (et == 0) ctl->go[acc & 1] = wait(wc, &ctl->acc_full[slot], turn & 1u, kWhereAcc);
            named_bar_sync(kEpiBar, kEpiThreads);
            if (!(ok = ctl->go[acc & 1] != 0)) break;
            tc_fence_after();
            ++acc;
            if (p.split > 1) break;  // the cluster's sums come first
            bf16* y = p.y + static_cast<size_t>(m0) * p.N + n;
            const uint32_t d = tmem + slot * 128 + (static_cast<uint32_t>(q * 32) << 16);
            for (int c0 = odd * 16; c0 < rows; c0 += 32) {
                float v[16];
                tmem_ld16(d + c0, v);
                tmem_ld_wait();
                if (n < p.N) {
                    bf16 o[16];
#pragma unroll
                    for (int c = 0; c < 16; c += 4) {
                        const float4 f = *reinterpret_cast<const float4*>(sx + c0 + c);
                        o[c] = __float2bfloat16_rn(v[c] * (f.x * sw));
                        o[c + 1] = __float2bfloat16_rn(v[c + 1] * (f.y * sw));
                        o[c + 2] = __float2bfloat16_rn(v[c + 2] * (f.z * sw));
                        o[c + 3] = __float2bfloat16_rn(v[c + 3] * (f.w * sw));
                    }
                    store16(y + static_cast<size_t>(c0) * p.N, p.N, o, rows - c0);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_leader<CG>(&ctl->acc_empty[slot], crank);
        }
    }

    __syncthreads();
    if (ctl->gave_up && threadIdx.x == 0) {
        // Every copy has landed before this CTA goes, whichever role gave up.  (Where none did, all
        // of them were used.  The tokens' barriers count both CTAs' copies.)
        auto landed = [](uint64_t* full, uint32_t posted, uint32_t stages) {
            for (uint32_t i = posted > stages ? posted - stages : 0; i < posted; ++i)
                (void)mbar_drain(&full[i % stages], (i / stages) & 1u, 1000000ull);
        };
        landed(ctl->full_w, ctl->posted_w, p.stages_w);
        if (CG == 2 && rank == 0) landed(ctl->full_x, ctl->posted_x[0], p.stages_x);
    }
    // the commits have arrived here, and no CTA goes while the pair's other may reach into it
    if (threadIdx.x == 32) (void)mbar_drain(&ctl->drain, 0, 2000000ull);
    tc_fence_before();
    __syncthreads();
    if (CG == 2) {
        cluster_sync();
        const uint32_t armed = ctl->posted_x[0], posted = ctl->posted_x[1];
        if (posted > armed) {
            // A wait ran out in between: copies of the pair's second CTA that the first one never
            // armed its barriers for.  It does so now, and both stay until they have landed.
            if (rank == 0 && threadIdx.x == 0)
                for (uint32_t i = armed; i < posted; ++i) {
                    uint64_t* bar = &ctl->full_x[i % p.stages_x];
                    mbar_arrive_expect_tx(bar, xbytes);
                    mbar_drain(bar, (i / p.stages_x) & 1u, 1000000ull);
                }
            __syncthreads();
            if (p.split == 1) cluster_sync();
        }
    }
    tc_fence_after();
    if (p.split > 1) {
        // Part r of the cluster sums tokens [r tn / split, (r + 1) tn / split) of the tile; what
        // the others have of them comes into its rings, which nothing uses any more.
        if (CG == 1) cluster_sync();
        const int tile = blockIdx.x / (CG * p.split), mine = crank / CG, each = p.tn / p.split;
        const bool have = tile < tiles;
        if (have && warp < 16) {
            const uint32_t row = (warp & 3) * 32 + lane;
            const uint32_t to = smem_u32(base) + (static_cast<uint32_t>(mine) * each * 128 + row) * 4;
            for (int c0 = (warp >> 2) * 16; c0 < p.tn; c0 += 64) {
                float v[16];
                tmem_ld16(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + c0, v);
                tmem_ld_wait();
                int at = c0 / each, c = c0 - at * each;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    uint32_t dst;
                    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(dst) : "r"(to + c * 512), "r"(at * CG + rank));
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst), "f"(v[i]) : "memory");
                    if (++c == each) { c = 0; ++at; }
                }
            }
        }
        tc_fence_before();
        cluster_sync();
        tc_fence_after();
        if (have) {
            const int m0 = (tile % mt) * p.tn, n0 = (tile / mt) * 128 * CG + static_cast<int>(rank) * 128, rows = min(p.tn, M - m0);
            const float* part = reinterpret_cast<const float*>(base);
            for (int o = threadIdx.x; o < each * 128; o += kI8Threads) {
                const int c = mine * each + o / 128, n = n0 + o % 128;
                if (c >= rows || n >= p.N) continue;
                float sum = 0.0f;
#pragma unroll 4
                for (int b = 0; b < p.split; ++b) sum += part[b * each * 128 + o];  // in the order of k
                p.y[static_cast<size_t>(m0 + c) * p.N + n] = __float2bfloat16_rn(sum * (ctl->sx[0][c] * p.sw[n]));
            }
        }
    }
    if (warp == 1) tmem_free<CG>(tmem);
}

__global__ void __launch_bounds__(256) i8_expand_kernel(const I8ExpandArgs p) {
    grid_begin();
    const int at = blockIdx.x * blockDim.x + threadIdx.x, step = gridDim.x * blockDim.x;
    const long long n = static_cast<long long>(pass_rows(p.rows, p.hdr)) * p.K / 16;
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
// tokens need little; never less than two stages of either.  An even number of them, so that
// a stage is always the same converters': who sees only every other use of a barrier could
// take a phase that has not come for the one before it.
int i8_tc_stages(bool pair, int tn, int blocks, int* w, int* x) {
    const int xbytes = tn / (pair ? 2 : 1) * 256, room = kSmemLimit - 1024 - kCtlBytes;
    *x = xbytes > 32768 ? 2 : xbytes > 16384 ? 4 : xbytes > 8192 ? 5 : 8;
    *w = (room - *x * xbytes) / kWBytes;
    if (*w > kI8MaxStages) *w = kI8MaxStages;
    *w &= ~1;
    if (*x > blocks) *x = blocks > 2 ? blocks : 2;
    while (*w > 2 && *w - 2 >= blocks && (*w - 2) * kWBytes + *x * xbytes >= tn * 512) *w -= 2;  // (a cluster's sums)
    return 1024 + kCtlBytes + *w * kWBytes + *x * xbytes;
}

cudaError_t launch_i8_tc(const I8TcArgs& a, const CUtensorMap* map_w, const CUtensorMap* map_x, bool pair, int dev, void* stream) {
    static SmemOptIn opt[2];
    int w, x;
    const int smem = i8_tc_stages(pair, a.tn, a.blocks, &w, &x);
    auto kernel = pair ? i8_tc_kernel<2> : i8_tc_kernel<1>;
    const cudaError_t e = api_smem_opt_in(opt[pair], dev, kernel, kSmemLimit);
    if (e != cudaSuccess) return e;
    const int cluster = a.split * (pair ? 2 : 1);
    return api_launch_cluster(kernel, a.grid * cluster, kI8Threads, cluster, true, smem, stream, *map_w, *map_x, a);
}

cudaError_t launch_i8_expand(const I8ExpandArgs& a, int sms, void* stream) {
    const long long n = (static_cast<long long>(a.rows.count) * a.K / 16 + 255) / 256;
    return api_launch(i8_expand_kernel, static_cast<unsigned>(n < 1 ? 1 : n < 8ll * sms ? n : 8ll * sms), 256, 0, stream, a);
}

}  // namespace et
