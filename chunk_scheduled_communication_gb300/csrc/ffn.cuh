// ffn.cuh -- what the gated feed-forward kernels share: a persistent GEMM on CTA
// pairs whose tiles name their operands (operators: include/syn_ffn.h).
//
// A pair of CTAs (a cluster of two) multiplies 256 rows by NT columns: the even
// CTA issues 256 x NT x 16 tcgen05.mma (cta_group::2), which read rows 0-127 of A
// and the first half of B's columns from its shared memory, the others from its
// peer's, and leave each CTA's 128 rows in that CTA's TMEM, in one of two
// accumulators of NT columns.
//
// CTA layout (320 threads, one CTA an SM):
//   warp 0      producer: TMA boxes of 64 x 64 elements into a ring of S stages
//               (two for the 128 rows of A, NT/128 for the NT/2 columns of B)
//   warp 1      TMEM, and in the even CTA the products
//   warps 2-9   epilogue: a thread a row, two warps to a row.  At NT 256 each has boxes
//               of its own, at 128 half of each box (and barriers between them)
//
// An operand's inner dimension (of the product) may be the contiguous one of its
// matrix ("K-major": boxes of 64 rows, the tile's, by 64 columns) or the other
// ("MN-major": 64 rows of the inner dimension by 64 of the tile's columns); both
// fill a box of 64 128-byte rows, 128-byte swizzle, and the instruction descriptor
// says which it is.
//
// What bounds it, measured on one GB300: at 256 x 256 tiles the tensor pipe, 512 cycles a
// k-block of 64 (8192 tokens, 4096 -> 14336: 959-990 us in short runs, 1.99 PFLOP/s, and
// 1030-1150 in long ones, 1.70, under the power cap), once the products' warp needs less than
// that for its wait, its products and its commit: one diverged lane took 630 cycles for
// them, converged warps 620, an elected lane 500, two k-blocks a stage 320.  With few
// tokens the weights' bytes bound it (8 tokens: 40-43 us, 35 of them HBM's).  Where a tile
// has few k-blocks its end does, 1.8 us (SiLU) to 2.3 (GELU) at 256 x 256: 19456 tokens,
// 128 -> 1280 21.3 us, ten tiles a pair.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"
#include "syn.h"
#include "window.cuh"

namespace syn {
namespace ffn {

constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kTileM = 256, kBK = 64;
constexpr uint32_t kBox = 64 * 128;  // bytes of a box
constexpr int kEpiSlots = 2, kEpiSlot = 32 * 128;  // of two epilogue warps: boxes of 32 rows of 128 bytes

// AR: rows of A that a stage has room for, 128, or where the call has no more (in
// the even CTA), 64 or 16: the products read 128 rows all the same, of whatever
// lies behind them in shared memory, into rows that are not stored.
// KS: k-blocks of a stage.
template <int NT_, int AR, int KS_> struct Lay {
    static constexpr int NT = NT_, KS = KS_;
    static constexpr int B_BOXES = NT / 128;
    static constexpr int A_BLOCK = AR * 128, B_BLOCK = B_BOXES * (int)kBox;
    static constexpr int A_BYTES = KS * A_BLOCK, B_BYTES = KS * B_BLOCK;
    static constexpr uint32_t STAGE = A_BYTES + B_BYTES;
    static constexpr int kRoom = (226 - 1) * 1024 - kEpiWarps / 2 * kEpiSlots * kEpiSlot - 512;  // (1 KB to align, barriers)
    static constexpr int S = kRoom / (int)STAGE;
    static constexpr int OFF_B = S * A_BYTES;
    static constexpr int OFF_EPI = OFF_B + S * B_BYTES;
    static constexpr int OFF_BAR = OFF_EPI + kEpiWarps / 2 * kEpiSlots * kEpiSlot;
    static constexpr int FULL = 0, EMPTY = S, TFULL = 2 * S, TEMPTY = TFULL + 2, DRAIN = TEMPTY + 2, PEER = DRAIN + 1;
    // TMEM address, abort, the odd CTA's k-blocks, its bytes in each stage, an answer for each quarter
    static constexpr int OFF_MISC = OFF_BAR + 8 * (PEER + 1), OFF_LAST = OFF_MISC + 12 + 4 * S;
    static constexpr int BYTES = OFF_LAST + 16 + 1024;  // (room to align to 1024)
    static_assert(BYTES <= 227 * 1024, "shared memory of a CTA");
    static_assert(S * B_BYTES >= 128 * 128, "what a product reads past the last stage of A");
};

struct Common {
    int32_t *err;  // {code, site, CTA, info}
    uint64_t timeout_ns;
};

// Boxes of 64 rows (or columns) from `at` on that meet a matrix of `end`, `most` at
// most.  Those past it are not brought: what they hold gives only results that are
// not stored, and zeros would cost the SM's bandwidth (a call of 8 tokens 94 us
// with them).
__device__ __forceinline__ int boxes_in(int at, int end, int most) { return window::clampi((end - at + 63) / 64, 0, most); }

// One operand of a tile: k-block kb (counted anew from the second matrix on) has its
// box i of n at column x + i * bx + kb * kx, row y + i * by + kb * ky
struct Operand {
    const CUtensorMap *m0, *m1;
    int x, y, bx, by, kx, ky, n;
    __device__ __forceinline__ void k_major(const CUtensorMap *a, const CUtensorMap *b, int row, int boxes) {
        m0 = a;
        m1 = b;
        x = 0;
        y = row;
        bx = 0;
        by = 64;
        kx = 64;
        ky = 0;
        n = boxes;
    }
    __device__ __forceinline__ void mn_major(const CUtensorMap *a, int col, int boxes) {
        m0 = m1 = a;
        x = col;
        y = 0;
        bx = 64;
        by = 0;
        kx = 0;
        ky = 64;
        n = boxes;
    }
};

struct Tile {
    Operand a, b;
    int k0, k1, half;      // stages [k0, k1); those before `half` are of the first pair of matrices
    uint32_t a_box, bytes; // of a box of A, of a k-block (both CTAs')
    bool a_mn, b_mn;
};

struct Cta {
    uint8_t *sm;
    uint32_t base, bar, tmem, rank;
    int unit, n_units, warp, lane;  // unit: the pair
    int quarter, half;              // an epilogue warp's 32 rows (the TMEM lanes it may read), and its half of their boxes
    volatile int *abort;
};

// Row-major walk in bands of `band` row tiles, columns outermost in a band, so
// that the tiles under way share rows and columns in L2
__device__ __forceinline__ void raster(int t, int tiles_m, int tiles_n, int band, int &m, int &n) {
    const int per = band * tiles_n, b = t / per, first = b * band, rows = min(band, tiles_m - first), r = t - b * per;
    n = r / rows;
    m = first + r - n * rows;
}

// ------------------------------------------------------------------ bounded waits
// Waits are made by whole, converged warps, single-thread instructions by an elected
// lane of theirs.
//
// A few polls without looking at the clock, each suspended for up to kSuspendNs (4 us on
// this GPU, whatever is asked: 80 us in all): a warp that polls without it takes the others'
// barrier operations time.  (The ring's barriers are completed by copies and products
// alone, which the barrier itself orders before the products and copies behind it: no
// acquire at cluster scope.)
constexpr uint32_t kSuspendNs = 20000;
__device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
        "mov.u32 n, 0;\n\t"
        "POLL_%=:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "@p bra DONE_%=;\n\t"
        "add.u32 n, n, 1;\n\t"
        "setp.lt.u32 q, n, 20;\n\t"
        "@q bra POLL_%=;\n\t"
        "DONE_%=:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(kSuspendNs)
        : "memory");
    return ok != 0;
}
// The rest of a wait: bounded; false after a wait of the CTA or of the grid ran out
__device__ __forceinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile int *abort, const Common &p) {
    const uint64_t t0 = ptx::globaltimer();
    while (!poll(bar, parity)) {
        if (*abort) return false;
        const bool late = ptx::globaltimer() - t0 > p.timeout_ns;
        if (late && atomicCAS(p.err, 0, SYN_ERR_TIMEOUT) == 0) {
            p.err[1] = window::WHERE_PIPE;
            p.err[2] = (int)blockIdx.x;
            p.err[3] = (int)bar;
        }
        if (late || *reinterpret_cast<volatile int32_t *>(p.err) != 0) {
            *abort = 1;
            return false;
        }
    }
    return true;
}
// A warp's wait; the same answer in all its lanes
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int *abort, const Common &p) {
    bool ok = poll(bar, parity);
    if (!ok) ok = wait_long(bar, parity, abort, p);
    return __all_sync(0xffffffffu, ok);
}
// On the way out: ignores the abort flag, with a limit of its own from `since` on (0: now)
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity, const Common &p, uint64_t since = 0) {
    if (!poll(bar, parity)) {
        const uint64_t t0 = since != 0 ? since : ptx::globaltimer(), limit = p.timeout_ns > window::kDrainNs ? p.timeout_ns : window::kDrainNs;
        while (!poll(bar, parity))
            if (ptx::globaltimer() - t0 > limit) {
                atomicCAS(p.err, 0, SYN_ERR_TIMEOUT);
                break;
            }
    }
    __syncwarp();
}

// One lane of a converged warp, the same every time
__device__ __forceinline__ bool elect() {
    uint32_t on;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(on));
    return on != 0;
}
// arrive on the barrier of both CTAs when the thread's products so far have completed
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"((uint16_t)3)
                 : "memory");
}

// ------------------------------------------------------------------ set-up and end of a CTA
template <class L> __device__ __forceinline__ Cta set_up(uint8_t *raw) {
    Cta c;
    c.sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    c.base = ptx::smem_u32(c.sm);
    c.bar = c.base + L::OFF_BAR;
    c.rank = ptx::cluster_ctarank();
    c.unit = (int)blockIdx.x / 2;
    c.n_units = (int)gridDim.x / 2;
    c.warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);
    c.lane = (int)threadIdx.x & 31;
    c.quarter = c.warp & 3;
    c.half = (c.warp - 2) >> 2;
    uint32_t *slot = reinterpret_cast<uint32_t *>(c.sm + L::OFF_MISC);
    c.abort = reinterpret_cast<volatile int *>(slot + 1);
    if (threadIdx.x == 0) {
        *c.abort = 0;
        for (int s = 0; s < L::S; ++s) {
            ptx::mbar_init(c.bar + 8 * (L::FULL + s), 1);
            ptx::mbar_init(c.bar + 8 * (L::EMPTY + s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(c.bar + 8 * (L::TFULL + a), 1);
            ptx::mbar_init(c.bar + 8 * (L::TEMPTY + a), 2 * kEpiWarps);  // an epilogue warp each, of both CTAs
        }
        ptx::mbar_init(c.bar + 8 * L::DRAIN, 1);
        ptx::mbar_init(c.bar + 8 * L::PEER, 1);
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    if (c.warp == 1) {
        ptx::tmem_alloc_pair(ptx::smem_u32(slot), 2 * L::NT);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();  // both CTAs' barriers exist before any remote arrive
    ptx::tc_fence_after();
    c.tmem = *slot;
    return c;
}

// A map's 128 bytes on their way to the TMA unit (from the kernel's own arguments:
// nothing that an earlier kernel wrote)
__device__ __forceinline__ void fetch_map(const CUtensorMap &m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&m)) : "memory");
}

// ------------------------------------------------------------------ producer and products (a warp each)
template <class L, class Walk> __device__ __forceinline__ uint32_t produce(const Cta &c, const Walk &walk, const Common &p) {
    volatile uint32_t *count = reinterpret_cast<volatile uint32_t *>(c.sm + L::OFF_MISC + 8), *bytes = count + 1;
    const uint32_t full0 = ptx::mapa(c.bar + 8 * L::FULL, 0);  // the even CTA's
    uint32_t it = 0, s = 0, ph = 0;
    bool ok = true;
    Tile t;
    for (int i = 0; ok && walk.tile(c, i, t); ++i) {
        const uint32_t mine = L::KS * ((uint32_t)t.a.n * t.a_box + (uint32_t)t.b.n * kBox);
        const int past = L::KS * (t.k0 < t.half ? t.k0 : t.k0 - t.half);  // k-blocks of the first matrix read by other parts
        int ax = t.a.x + past * t.a.kx, ay = t.a.y + past * t.a.ky, bx = t.b.x + past * t.b.kx, by = t.b.y + past * t.b.ky;
        const CUtensorMap *am = t.k0 < t.half ? t.a.m0 : t.a.m1, *bm = t.k0 < t.half ? t.b.m0 : t.b.m1;
        for (int kb = t.k0; kb < t.k1; ++kb, ++it) {
            // until the pair's products have read the stage (its first use is free)
            if (!wait(c.bar + 8 * (L::EMPTY + s), ph ^ 1u, c.abort, p)) {
                ok = false;
                break;
            }
            if (kb == t.half && kb > t.k0) {
                am = t.a.m1;
                bm = t.b.m1;
                ax = t.a.x;
                ay = t.a.y;
                bx = t.b.x;
                by = t.b.y;
            }
            const uint32_t a = c.base + s * L::A_BYTES, b = c.base + L::OFF_B + s * L::B_BYTES, full = full0 + 8 * s;
            if (elect()) {
                if (c.rank == 0) ptx::mbar_arrive_expect_tx(c.bar + 8 * (L::FULL + s), L::KS * t.bytes);
                else bytes[s] = mine;
#pragma unroll
                for (int k = 0; k < L::KS; ++k) {
                    const uint32_t ak = a + k * L::A_BLOCK, bk = b + k * L::B_BLOCK;
                    const int axk = ax + k * t.a.kx, ayk = ay + k * t.a.ky, bxk = bx + k * t.b.kx, byk = by + k * t.b.ky;
                    if (t.a.n > 0) ptx::tma_load_2d_pair(ak, am, full, axk, ayk);
                    if (L::A_BLOCK > (int)kBox && t.a.n > 1) ptx::tma_load_2d_pair(ak + kBox, am, full, axk + t.a.bx, ayk + t.a.by);
                    if (t.b.n > 0) ptx::tma_load_2d_pair(bk, bm, full, bxk, byk);
                    if (L::B_BOXES > 1 && t.b.n > 1) ptx::tma_load_2d_pair(bk + kBox, bm, full, bxk + t.b.bx, byk + t.b.by);
                }
            }
            __syncwarp();
            ax += L::KS * t.a.kx;
            ay += L::KS * t.a.ky;
            bx += L::KS * t.b.kx;
            by += L::KS * t.b.ky;
            if (++s == (uint32_t)L::S) {
                s = 0;
                ph ^= 1u;
            }
        }
    }
    // the odd one reports how many k-blocks and bytes it issued
    __syncwarp();
    if (c.rank != 0 && c.lane == 0) {
        const uint32_t to = ptx::mapa(c.base + L::OFF_MISC + 8, 0);
        ptx::st_shared_cluster_u32(to, it);
        for (uint32_t k = 0; k < (uint32_t)L::S && k < it; ++k) ptx::st_shared_cluster_u32(to + 4 + 4 * k, bytes[k]);
        ptx::mbar_arrive_remote(ptx::mapa(c.bar + 8 * L::PEER, 0));
    }
    __syncwarp();
    return it;
}

// After a wait of the even CTA that ran out: what either CTA loads into its stages must
// have landed before the pair leaves (else the products have waited for all of it).  Both
// producers wake on the same commit, so one can be a use of a stage ahead of the other:
// the even one arms the phases that only the odd one loads into (one that only the even
// one loads into ends with the limit, which counts once for all stages).
template <class L> __device__ __forceinline__ void land(const Cta &c, uint32_t it, const Common &p) {
    volatile uint32_t *count = reinterpret_cast<volatile uint32_t *>(c.sm + L::OFF_MISC + 8), *bytes = count + 1;
    const uint64_t since = ptx::globaltimer();
    drain(c.bar + 8 * L::PEER, 0, p, since);
    (void)ptx::mbar_try_wait_cluster(c.bar + 8 * L::PEER, 0);  // (complete: acquires what the odd CTA wrote)
    const uint32_t other = *count, most = max(it, other);
    for (uint32_t k = 0; k < (uint32_t)L::S; ++k) {
        const uint32_t mine = it > k ? (it - 1u - k) / L::S + 1u : 0u, theirs = other > k ? (other - 1u - k) / L::S + 1u : 0u;
        if (theirs > mine && c.lane == 0) ptx::mbar_arrive_expect_tx(c.bar + 8 * (L::FULL + k), bytes[k]);
    }
    __syncwarp();
    for (uint32_t k = 0; k < (uint32_t)L::S; ++k)
        if (most > k) drain(c.bar + 8 * (L::FULL + k), (((most - 1u - k) / L::S)) & 1u, p, since);
}

// issued: the producer's k-blocks (warp 0)
template <class L> __device__ __forceinline__ void tear_down(const Cta &c, uint32_t issued, const Common &p) {
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (c.warp == 0 && c.rank == 0 && *c.abort != 0) land<L>(c, issued, p);
    __syncwarp();
    ptx::cluster_sync();  // no remote arrive or copy may target a CTA that has left
    ptx::tc_fence_after();
    if (c.warp == 1) ptx::tmem_dealloc_pair(c.tmem, 2 * L::NT);
}

template <class L, class Walk> __device__ __forceinline__ void multiply(const Cta &c, const Walk &walk, bool bf16, const Common &p) {
    if (c.rank != 0) return;
    uint32_t n = 0, s = 0, ph = 0;
    bool ok = true;
    Tile t;
    for (int i = 0; ok && walk.tile(c, i, t); ++i, ++n) {
        const uint32_t acc = n & 1u, d = c.tmem + acc * L::NT;
        if (!wait(c.bar + 8 * (L::TEMPTY + acc), ((n >> 1) & 1u) ^ 1u, c.abort, p)) break;
        ptx::tc_fence_after();
        const uint32_t idesc = ptx::idesc_16bit_f32(bf16, kTileM, L::NT, t.b_mn) | (t.a_mn ? 1u << 15 : 0u);
        // a slice of 16 of the inner dimension: 32 bytes on inside the swizzled rows, or 16 rows on
        const int a_step = t.a_mn ? 2048 : 32, b_step = t.b_mn ? 2048 : 32;
        const uint32_t a0 = window::desc_lo(c.base, t.a_mn ? kBox : 16u), b0 = window::desc_lo(c.base + L::OFF_B, t.b_mn ? kBox : 16u);
        for (int kb = t.k0; kb < t.k1; ++kb) {
            if (!wait(c.bar + 8 * (L::FULL + s), ph, c.abort, p)) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            const uint32_t a = a0 + s * (L::A_BYTES >> 4), b = b0 + s * (L::B_BYTES >> 4);
            if (elect()) {
#pragma unroll
                for (int k = 0; k < L::KS * (kBK / 16); ++k)
                    ptx::umma_bf16_pair(d, window::desc_at(a, k / 4 * L::A_BLOCK + k % 4 * a_step),
                                        window::desc_at(b, k / 4 * L::B_BLOCK + k % 4 * b_step), idesc, kb > t.k0 || k > 0 ? 1u : 0u);
                // the stage is free in both CTAs once these have completed
                commit(c.bar + 8 * (L::EMPTY + s));
            }
            __syncwarp();
            if (++s == (uint32_t)L::S) {
                s = 0;
                ph ^= 1u;
            }
        }
        if (ok && elect()) commit(c.bar + 8 * (L::TFULL + acc));
        __syncwarp();
    }
    // every product must have ended before TMEM is freed
    if (elect()) ptx::umma_commit_pair(c.bar + 8 * L::DRAIN);
    __syncwarp();
    drain(c.bar + 8 * L::DRAIN, 0, p);
}

// ------------------------------------------------------------------ epilogue
// The accumulator of tile number n is complete; false after a wait that ran out.
// TOGETHER: the same answer for both warps of a quarter, which go on to barriers of theirs.
template <class L, bool TOGETHER> __device__ __forceinline__ bool accumulated(const Cta &c, uint32_t n, const Common &p) {
    uint32_t ok = wait(c.bar + 8 * (L::TFULL + (n & 1u)), (n >> 1) & 1u, c.abort, p) ? 1u : 0u;
    if (TOGETHER)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %0, 0;\n\tbar.red.and.pred q, %1, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
            : "+r"(ok)
            : "r"(1 + c.quarter)
            : "memory");
    if (ok == 0) return false;
    ptx::tc_fence_after();
    return true;
}
// The warp's loads from TMEM are complete: v and w are there from here on
template <int N> __device__ __forceinline__ void loaded(uint32_t (&v)[N], uint32_t (&w)[N]) {
    ptx::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(v[i]), "+r"(w[i]));
}
// N fp32 values as pairs of 16-bit ones
template <int N> __device__ __forceinline__ void pack(bool bf16, const uint32_t (&f)[N], uint32_t *out) {
    if (bf16)
#pragma unroll
        for (int i = 0; i < N / 2; ++i) out[i] = window::pack16<true>(__uint_as_float(f[2 * i]), __uint_as_float(f[2 * i + 1]));
    else
#pragma unroll
        for (int i = 0; i < N / 2; ++i) out[i] = window::pack16<false>(__uint_as_float(f[2 * i]), __uint_as_float(f[2 * i + 1]));
}
// This warp has read the accumulator of tile number n.  The odd CTA's arrive orders
// nothing but what tcgen05 has read: with a release at cluster scope it waited for the
// warp's other memory operations, 300 of its 1600 ns a tile, and both CTAs for it.
template <class L> __device__ __forceinline__ void release(const Cta &c, uint32_t n) {
    ptx::tc_fence_before();
    __syncwarp();
    if (c.lane != 0) return;
    const uint32_t bar = c.bar + 8 * (L::TEMPTY + (n & 1u));
    if (c.rank == 0) ptx::mbar_arrive(bar);
    else asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(ptx::mapa(bar, 0)) : "memory");
}

// Barrier of the two warps of a quarter
__device__ __forceinline__ void meet(const Cta &c) { asm volatile("bar.sync %0, 64;" ::"r"(1 + c.quarter) : "memory"); }

// Tiles whose inner dimension is cut into parts (there are fewer tiles than pairs).
// The epilogue warps leave the sums of a part in the plan's workspace, four columns of
// their 32 rows at a time; the quarter that arrives last at its rows of the tile adds
// the parts in their order.
struct Parts {
    float *sums;        // [part item][CTA][quarter][columns / 4][32 rows][4]
    uint32_t *arrived;  // [tile][CTA][quarter], zero between calls
};
template <class L> __device__ __forceinline__ float4 *strip_of(const Parts &p, int item, const Cta &c) {
    return reinterpret_cast<float4 *>(p.sums) + ((int64_t)(item * 2 + (int)c.rank) * 4 + c.quarter) * (L::NT * 8);
}
// 32 columns of the thread's row of a part, from TMEM to the strip
__device__ __forceinline__ void leave(float4 *strip, int col, uint32_t acc, int lane) {
    uint32_t v[32];
    ptx::tmem_ld_32x32b_x32(acc + col, v);
    ptx::tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 8; ++k)
        __stcg(strip + (col / 4 + k) * 32 + lane, make_float4(__uint_as_float(v[4 * k]), __uint_as_float(v[4 * k + 1]),
                                                             __uint_as_float(v[4 * k + 2]), __uint_as_float(v[4 * k + 3])));
}
// All parts have arrived at this quarter of a tile (the same in both warps)
template <class L> __device__ __forceinline__ bool last_of(const Parts &p, int tile, int parts, const Cta &c) {
    volatile uint32_t *answer = reinterpret_cast<volatile uint32_t *>(c.sm + L::OFF_LAST) + c.quarter;
    __threadfence();
    meet(c);
    if (c.half == 0 && c.lane == 0) {
        uint32_t *n = p.arrived + (tile * 2 + (int)c.rank) * 4 + c.quarter;
        const uint32_t last = ptx::atom_add_acq_rel_gpu(n, 1u) == (uint32_t)parts - 1u;
        if (last) *n = 0u;  // for the next call
        __threadfence();
        *answer = last;
    }
    meet(c);
    return *answer != 0;
}
// W x 32 columns of the thread's row from columns col, col + next, the sum of parts
// that lie `apart` vectors from each other; a part's loads, and those of the next, are
// under way together
template <int W> __device__ __forceinline__ void join(const float4 *first, int64_t apart, int parts, int col, int next, int lane, float (&f)[W][32]) {
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
        for (int k = 0; k < 32; ++k) f[w][k] = 0.f;
#pragma unroll 2
    for (int i = 0; i < parts; ++i) {
        float4 v[W][8];
#pragma unroll
        for (int w = 0; w < W; ++w)
#pragma unroll
            for (int k = 0; k < 8; ++k) v[w][k] = __ldcg(first + i * apart + ((col + w * next) / 4 + k) * 32 + lane);
#pragma unroll
        for (int w = 0; w < W; ++w)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                f[w][4 * k] += v[w][k].x;
                f[w][4 * k + 1] += v[w][k].y;
                f[w][4 * k + 2] += v[w][k].z;
                f[w][4 * k + 3] += v[w][k].w;
            }
    }
}

// Results through a quarter's two slots (128-byte rows, 128-byte swizzle) to boxes of 32
// rows of a matrix; rows and columns past its end are not written.  (A gradient of 128
// tokens writes 235 MB of dW in 49 us, 4.8 TB/s.)
struct Stores {
    uint32_t slots, n;  // the quarter's slots; 16-bit boxes stored so far
    // 64 columns rounded to 16 bits, 32 a warp (NT 128).  `wide`: among boxes of fp32, whose
    // slots are a warp's own
    __device__ __forceinline__ void box(const Cta &c, const CUtensorMap *m, bool bf16, const float (&f)[32], int col, int row, bool wide = false) {
        const uint32_t slot = slots + (wide ? 0u : (n++ & 1u) * kEpiSlot);
        if (c.half == 0 && c.lane == 0) {  // the slot's last store has read it
            if (wide) ptx::bulk_wait_read<0>();
            else ptx::bulk_wait_read<1>();
        }
        meet(c);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float *e = f + 8 * k;
            const uint32_t at = slot + (uint32_t)(c.lane * 128) + ((uint32_t)((4 * c.half + k) ^ (c.lane & 7)) << 4);
            if (bf16)
                ptx::st_shared_u4(at, window::pack16<true>(e[0], e[1]), window::pack16<true>(e[2], e[3]), window::pack16<true>(e[4], e[5]),
                                  window::pack16<true>(e[6], e[7]));
            else
                ptx::st_shared_u4(at, window::pack16<false>(e[0], e[1]), window::pack16<false>(e[2], e[3]), window::pack16<false>(e[4], e[5]),
                                  window::pack16<false>(e[6], e[7]));
        }
        ptx::fence_proxy_async_smem();
        meet(c);
        if (c.half == 0 && c.lane == 0) {
            ptx::tma_store_2d(m, slot, col, row);
            ptx::bulk_commit();
        }
    }
    __device__ __forceinline__ void wide(const Cta &c, const CUtensorMap *m, const float (&f)[32], int col, int row) {
        uint32_t v[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(f[k]);
        wide(c, m, v, col, row);
    }
    // 64 columns of 16 bits, all a warp's own, from pairs (NT 256)
    __device__ __forceinline__ void own(const Cta &c, const CUtensorMap *m, const uint32_t (&v)[32], int col, int row) {
        const uint32_t slot = slots + (uint32_t)c.half * kEpiSlot;
        if (c.lane == 0) ptx::bulk_wait_read<0>();
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k)
            ptx::st_shared_u4(slot + (uint32_t)(c.lane * 128) + ((uint32_t)(k ^ (c.lane & 7)) << 4), v[4 * k], v[4 * k + 1], v[4 * k + 2],
                              v[4 * k + 3]);
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (c.lane == 0) {
            ptx::tma_store_2d(m, slot, col, row);
            ptx::bulk_commit();
        }
    }
    // a warp's 32 columns in fp32
    __device__ __forceinline__ void wide(const Cta &c, const CUtensorMap *m, const uint32_t (&f)[32], int col, int row) {
        const uint32_t slot = slots + (uint32_t)c.half * kEpiSlot;
        if (c.lane == 0) ptx::bulk_wait_read<0>();
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k)
            ptx::st_shared_u4(slot + (uint32_t)(c.lane * 128) + ((uint32_t)(k ^ (c.lane & 7)) << 4), f[4 * k], f[4 * k + 1], f[4 * k + 2],
                              f[4 * k + 3]);
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (c.lane == 0) {
            ptx::tma_store_2d(m, slot, col, row);
            ptx::bulk_commit();
        }
    }
};
template <class L> __device__ __forceinline__ Stores stores_of(const Cta &c) {
    return {c.base + L::OFF_EPI + (uint32_t)(c.quarter * kEpiSlots * kEpiSlot), 0u};
}

// ------------------------------------------------------------------ launches
struct FwdMaps {
    CUtensorMap x, wg, wu, h, g, u;
};
struct FwdParams {
    Common c;
    int32_t m, k, f;          // tokens, columns of X, columns of H
    int32_t tiles_m, tiles_n, band;
    int32_t x_rows;           // rows of a box of X: 64, fewer where there are fewer tokens
    int32_t keep, bf16;       // keep: G and U are wanted (2: in fp32)
    int32_t split;            // parts of a tile's inner dimension
    Parts parts;
};
struct BwdMaps {
    CUtensorMap x, wg, wu, dg, du, dx, dwg, dwu;
};
struct BwdParams {
    Common c;
    int32_t m, k, f;
    int32_t dx_m, dx_n;                 // tiles of dX (0: not wanted)
    int32_t dw_m, dw_n;                 // of dWg and dWu together
    int32_t dw_first;                   // the longer of the two kinds is dealt out first
    int32_t items1, split;              // parts of that kind's tiles, in all and of a tile
    int32_t tiles2;                     // tiles of the other kind
    int32_t even, rest;                 // rounds of these in which all pairs take part; pairs that take no part later
    int32_t band, bf16;
    Parts parts;
};
struct ActParams {
    const void *dh, *g, *u;
    void *dg, *du;
    int64_t dh_row, g_row, u_row, dg_row, du_row;
    uint32_t n, per_row, magic, shift;  // vectors of 8 elements, in all and of a row
};

cudaError_t fwd_prepare(int act);
cudaError_t bwd_prepare();
cudaError_t fwd_launch(int act, int nt, int pairs, const FwdParams &p, const FwdMaps &m, cudaStream_t st);
cudaError_t bwd_launch(int pairs, const BwdParams &p, const BwdMaps &m, cudaStream_t st);
cudaError_t act_grad_launch(int act, bool bf16, bool wide, const ActParams &p, cudaStream_t st);  // wide: G and U in fp32

}  // namespace ffn
}  // namespace syn
