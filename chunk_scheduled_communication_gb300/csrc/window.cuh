// window.cuh -- what the windowed-attention kernels share: their work items,
// launch parameters, bounded waits and the descriptors of their tiles
// (operators: include/syn_window.h).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"
#include "syn.h"

namespace syn {
namespace window {

constexpr int kNoWindow = 0x3fffffff;  // "no window": above every position

// Forward work item: two 128-row query tiles that read the same key blocks --
// the same rows of two heads of a group, or consecutive rows of one head.
// Key blocks of fwd_block(d) keys: of the sinks [0, s_end), then of [w_lo, k_end)
// (keys relative to the sequence).
struct alignas(16) FwdItem {
    int32_t q_row[2], head[2], n_rows[2], pos0[2];  // n_rows 0: no second tile
    int32_t kv_row0, hk, s_end, w_lo, k_end, n_blk, pad[2];
};

// Gradient work item: 128 stationary rows, and what streams past them.
//   dK, dV: stationary keys j0 .. of kv head hk; query blocks [b0, b1) of 64
//           rows of the sequence for each head of [h0, h1)
//   dQ:     stationary query rows of head h0; key blocks of the sinks
//           [0, s_end), then of [w_lo, k_end)
struct alignas(16) BwdItem {
    int32_t row0;             // first stationary row (global)
    int32_t n_rows;           // valid stationary rows
    int32_t pos0;             // position of the first stationary row (dK, dV: its key index)
    int32_t hk, h0, h1;
    int32_t stream0;          // global row of the sequence's first streaming row
    int32_t stream_len;       // the sequence's streaming rows
    int32_t off;              // k_len - q_len
    int32_t b0, b1;           // dK, dV: query blocks
    int32_t s_end, w_lo, k_end;  // dQ
    int32_t pad_row0;         // first row of the sequence in the padded statistics
    int32_t part;             // dK, dV: slot of the partial sums, -1: write the gradients
};

// dK, dV tile whose sum is in several parts: slots [part0, part0 + n_parts)
struct alignas(16) SumItem {
    int32_t row0, n_rows, hk, part0, n_parts, pad[3];
};

// Rows of a [rows, heads, d] tensor that a kernel stores to
struct Out {
    void *p;
    int64_t token, head;
};

struct Common {
    int32_t window, sinks, H_q, G;
    float scale, scale_log2;
    uint64_t timeout_ns;
    int32_t *err;  // {code, site, CTA, info}
};

constexpr int WHERE_PIPE = 3;

// Waits, arrivals and tensor-core instructions are made by whole, converged
// warps, single-thread ones predicated: a diverged lane pays three times as
// much for a barrier that is already complete (186 cycles against 58) and twice
// for one that another warp arrives at (284 against 132).
//
// Up to a thousand polls without looking at the clock.
__device__ __forceinline__ bool poll_bar(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
        "mov.u32 n, 0;\n\t"
        "POLL_%=:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra DONE_%=;\n\t"
        "add.u32 n, n, 1;\n\t"
        "setp.lt.u32 q, n, 1000;\n\t"
        "@q bra POLL_%=;\n\t"
        "DONE_%=:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

constexpr uint64_t kDrainNs = 1000000000;  // limit of the waits on the way out, at least

// The rest of a wait: bounded.  A wait that runs out records SYN_ERR_TIMEOUT and
// sets `abort`, after which no wait lasts; the warp goes on, with wrong results
// but within its buffers, to the end of its loop.  The producer stops (a barrier
// whose copies are still under way is not armed again) and waits for what it has
// issued, as the issuers do; these waits have a limit of their own, so that a short
// one of the caller's does not end a CTA before its copies and products.
__device__ __forceinline__ void wait_long(uint32_t bar, uint32_t parity, volatile int *abort, const Common &p) {
    const uint64_t t0 = ptx::globaltimer(), limit = abort != nullptr || p.timeout_ns > kDrainNs ? p.timeout_ns : kDrainNs;
    while (!poll_bar(bar, parity)) {
        if (abort != nullptr && *abort != 0) return;
        const bool late = ptx::globaltimer() - t0 > limit;
        if (late && atomicCAS(p.err, 0, SYN_ERR_TIMEOUT) == 0) {
            p.err[1] = WHERE_PIPE;
            p.err[2] = (int)blockIdx.x;
            p.err[3] = (int)bar;
        }
        if (late || *reinterpret_cast<volatile int32_t *>(p.err) != 0) {
            if (abort == nullptr) {
                if (late) return;
                continue;
            }
            *abort = 1;
            return;
        }
    }
}

// Bounded wait of a warp on a shared-memory barrier phase.
__device__ __forceinline__ void wait_bar(uint32_t bar, uint32_t parity, volatile int *abort, const Common &p) {
    if (!poll_bar(bar, parity)) wait_long(bar, parity, abort, p);
    __syncwarp();
}

// Whether a wait of the CTA ran out (one read of a converged warp: the same for
// all its lanes)
__device__ __forceinline__ bool aborted(volatile int *abort) { return *abort != 0; }

// Wait used while draining on the way out: ignores the abort flag.
__device__ __forceinline__ void drain_bar(uint32_t bar, uint32_t parity, const Common &p) {
    wait_long(bar, parity, nullptr, p);
    __syncwarp();
}

// One lane's arrival, MMA or commit (`on`: this lane's)
__device__ __forceinline__ void arrive_if(uint32_t on, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %0, 0;\n\t"
        "@p mbarrier.arrive.shared::cta.b64 _, [%1];\n\t}" ::"r"(on), "r"(bar) : "memory");
}
__device__ __forceinline__ void umma_if(uint32_t on, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem), "l"(adesc), "l"(bdesc),
        "r"(idesc), "r"(accumulate), "r"(on) : "memory");
}
__device__ __forceinline__ void umma_ts_if(uint32_t on, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc),
        "r"(idesc), "r"(accumulate), "r"(on) : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t on, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %0, 0;\n\t"
        "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t}" ::"r"(on), "r"(bar) : "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Packed fp32 pairs (one instruction for two lanes of work) and a three-input max
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unf2(uint64_t r, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Bits [0, n) of a 32-bit word whose first bit is number `at`
__device__ __forceinline__ uint32_t bits_below(int n, int at) {
    const int m = n - at;
    return m <= 0 ? 0u : m >= 32 ? 0xffffffffu : (1u << m) - 1u;
}
// v where bit `bit` of the mask is set, else `other`: a select (a condition in C
// became a branch for each element, each of them diverging)
template <int BIT> __device__ __forceinline__ uint32_t keep_if(uint32_t mask, uint32_t v, uint32_t other) {
    uint32_t r;
    asm("{\n\t.reg .pred p;\n\t.reg .b32 t;\n\t"
        "and.b32 t, %1, %4;\n\t"
        "setp.ne.u32 p, t, 0;\n\t"
        "selp.b32 %0, %2, %3, p;\n\t}"
        : "=r"(r)
        : "r"(mask), "r"(v), "r"(other), "n"(1u << BIT));
    return r;
}
// v[K ..]: `other` where the mask's bit is not set
template <int K, int N> struct MaskRow {
    static __device__ __forceinline__ void apply(uint32_t (&v)[N], const uint32_t (&mask)[(N + 31) / 32], uint32_t other) {
        v[K] = keep_if<K % 32>(mask[K / 32], v[K], other);
        if constexpr (K + 1 < N) MaskRow<K + 1, N>::apply(v, mask, other);
    }
};

// Two fp32 values rounded to the 16-bit type, the lower in the low half
template <bool BF16> __device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if (BF16) {
        __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&v);
    }
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
}

// A tile of 128 (or 64) rows x D 16-bit elements lies in shared memory as D/64
// boxes of 64 columns, 128 bytes a row, 128-byte swizzle, `box` bytes apart.
// K-major operand (columns are the product's inner dimension): 16-element
// slice kk lies in box kk/4, 32 bytes a slice inside the swizzled row; 8-row
// atoms 1024 bytes apart.
__device__ __forceinline__ uint64_t kmajor_desc(uint32_t tile, uint32_t box, int kk) {
    return ptx::sdesc(tile + (uint32_t)(kk >> 2) * box + (uint32_t)(kk & 3) * 32u, 16, 1024, ptx::kSwizzle128B);
}
// MN-major B operand (rows are the inner dimension, columns N): slice kk is
// rows 16kk .. 16kk+15 (2048 bytes on), the boxes `box` apart.
__device__ __forceinline__ uint64_t mnmajor_desc(uint32_t tile, uint32_t box, int kk) {
    return ptx::sdesc(tile + (uint32_t)kk * 2048u, box, 1024, ptx::kSwizzle128B);
}

// The same descriptors from their two words: the upper is the same for all (8-row
// atoms 1024 bytes apart, version 1, 128-byte swizzle), the lower holds address
// and box distance, and a later slice of the tile only adds to the address.
__device__ __forceinline__ uint32_t desc_lo(uint32_t tile, uint32_t lbo_bytes) {
    return ((tile & 0x3FFFFu) >> 4) | ((lbo_bytes >> 4) << 16);
}
__device__ __forceinline__ uint64_t desc_at(uint32_t lo, int bytes) {
    constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (ptx::kSwizzle128B << 29);
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo + (uint32_t)(bytes >> 4)), "r"(hi));
    return d;
}

// Zero rows [r0, r1) of a tile of D columns (one warp, generic proxy); the
// caller fences to the async proxy.
template <int D> __device__ __forceinline__ void zero_rows(uint8_t *tile, int box, int r0, int r1, int lane) {
    for (int b = 0; b < D / 64; ++b) {
        uint4 *p = reinterpret_cast<uint4 *>(tile + b * box + r0 * 128);
        for (int i = lane; i < (r1 - r0) * 8; i += 32) p[i] = make_uint4(0, 0, 0, 0);
    }
}

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return min(max(v, lo), hi); }

// 32 accumulator columns of this thread's row to 16-bit (dst) or fp32 (part)
template <bool BF16>
__device__ __forceinline__ void store_cols(uint32_t taddr, uint16_t *dst, float *part, float scale) {
    uint32_t v[32];
    ptx::tmem_ld_32x32b_x32(taddr, v);
    ptx::tmem_ld_wait();
    if (dst != nullptr) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint4 o;
            o.x = pack16<BF16>(__uint_as_float(v[8 * k + 0]) * scale, __uint_as_float(v[8 * k + 1]) * scale);
            o.y = pack16<BF16>(__uint_as_float(v[8 * k + 2]) * scale, __uint_as_float(v[8 * k + 3]) * scale);
            o.z = pack16<BF16>(__uint_as_float(v[8 * k + 4]) * scale, __uint_as_float(v[8 * k + 5]) * scale);
            o.w = pack16<BF16>(__uint_as_float(v[8 * k + 6]) * scale, __uint_as_float(v[8 * k + 7]) * scale);
            reinterpret_cast<uint4 *>(dst)[k] = o;
        }
    } else if (part != nullptr) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            reinterpret_cast<uint4 *>(part)[k] = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
    }
}

// ------------------------------------------------------------------ launches
struct FwdMaps {
    CUtensorMap q, k, k16, v, v16;  // boxes of a tile, and of 16 rows for narrow key blocks
};
struct FwdParams {
    Common c;
    const FwdItem *items;
    const int32_t *begin;   // [grid + 1] items of each CTA
    const FwdItem *empty;   // tiles none of whose rows see a key
    int32_t n_empty;
    Out o;
    float *lse;
};

struct BwdMaps {
    CUtensorMap x, y;       // stationary rows (128-row boxes): K, V or Q, dO
    CUtensorMap u, w;       // streaming rows (boxes of a block): Q, dO or K, V
};
struct BwdParams {
    Common c;
    const BwdItem *items;
    const int32_t *begin;   // [grid + 1]
    const float *nlse2;     // [H_q][pad_rows]: -lse * log2(e) (-inf: no gradient)
    float *ndelta;          // [H_q][pad_rows]: -rowsum(dO * O); the dQ kernel makes some of them exact
    int64_t pad_rows;
    Out dx, dy;             // dK, dV or dQ
    float *part;            // [parts][2][128][d]
};
struct PrepTile {           // 64 query rows of a sequence, for the statistics
    int32_t row0, n_rows, pad_row0, pad;
};
struct PrepParams {
    const PrepTile *tiles;
    const void *o, *d_o;
    int64_t o_token, o_head, do_token, do_head;
    const float *lse;
    float *nlse2, *ndelta;
    int64_t pad_rows;
    int32_t H_q, d;
};
struct SumParams {
    const SumItem *items;
    const float *part;
    Out dk, dv;
    float scale;
    int32_t d;
};

int fwd_block(int d);  // keys of a key block
cudaError_t fwd_prepare(int d, bool bf16);
cudaError_t dkv_prepare(int d, bool bf16);
cudaError_t dq_prepare(int d, bool bf16);
cudaError_t fwd_launch(int d, bool bf16, int grid, const FwdParams &p, const FwdMaps &m, cudaStream_t st);
cudaError_t bwd_prep_launch(bool bf16, int n_tiles, const PrepParams &p, cudaStream_t st);
cudaError_t dkv_launch(int d, bool bf16, int grid, const BwdParams &p, const BwdMaps &m, cudaStream_t st);
cudaError_t dq_launch(int d, bool bf16, int grid, const BwdParams &p, const BwdMaps &m, cudaStream_t st);
cudaError_t bwd_sum_launch(bool bf16, int n_items, const SumParams &p, cudaStream_t st);

// Launch a kernel whose blocks may start, as far as ptx::grid_wait, while the
// stream's kernel before it ends: its launch, its barriers, TMEM and work list
// cost less (calls in a graph on one GB300, without and with it: a rotation of 8
// tokens 2.7, 2.4 us; norm and rotation of 4 3.5, 3.0; a decode of 3 sequences
// 10.5, 10.1; the five launches of a ragged training step 97.8, 96.1).  The kernel
// before may be of another kind that lets its successor start at its own
// beginning, so every thread of these waits.  None of these lets the next one start
// before its own blocks end: that took the SMs' places out of the order the
// work is dealt in (gradient at 16384 tokens 1980 -> 2015 us, decode 10.3 -> 11.2).
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, const A &...a) {
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a...);
}

}  // namespace window
}  // namespace syn
