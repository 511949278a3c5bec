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

// Gradient work item of either kernel: 128 stationary rows and the 64-row
// blocks that stream past them.
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

__device__ __forceinline__ void raise(const Common &p, int code, int where, int info) {
    if (atomicCAS(p.err, 0, code) == 0) {
        p.err[1] = where;
        p.err[2] = (int)blockIdx.x;
        p.err[3] = info;
    }
}

// Bounded wait on a shared-memory barrier phase; false on abort or timeout.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort, const Common &p) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer();
    for (uint32_t n = 1;; ++n) {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        if ((n & 63u) == 0u) {
            if (*reinterpret_cast<volatile int32_t *>(p.err) != 0) {
                *abort = 1;
                return false;
            }
            if (ptx::globaltimer() - t0 > p.timeout_ns) {
                raise(p, SYN_ERR_TIMEOUT, WHERE_PIPE, (int)bar);
                *abort = 1;
                return false;
            }
        }
    }
}

// Wait used while draining on the way out: ignores the abort flag.
__device__ __forceinline__ void drain_bar(uint32_t bar, uint32_t parity, const Common &p) {
    const uint64_t t0 = ptx::globaltimer();
    for (uint32_t n = 0;; ++n) {
        if (ptx::mbar_try_wait(bar, parity)) return;
        if ((n & 63u) == 63u && ptx::globaltimer() - t0 > p.timeout_ns) {
            raise(p, SYN_ERR_TIMEOUT, WHERE_PIPE, (int)bar);
            return;
        }
    }
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

// Zero rows [r0, r1) of a tile of D columns (one warp, generic proxy); the
// caller fences to the async proxy.
template <int D> __device__ __forceinline__ void zero_rows(uint8_t *tile, int box, int r0, int r1, int lane) {
    for (int b = 0; b < D / 64; ++b) {
        uint4 *p = reinterpret_cast<uint4 *>(tile + b * box + r0 * 128);
        for (int i = lane; i < (r1 - r0) * 8; i += 32) p[i] = make_uint4(0, 0, 0, 0);
    }
}

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return min(max(v, lo), hi); }

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
    CUtensorMap u, w;       // streaming rows (64-row boxes): Q, dO or K, V
};
struct BwdParams {
    Common c;
    const BwdItem *items;
    const int32_t *begin;   // [grid + 1]
    const float *nlse2, *ndelta;  // [H_q][pad_rows]: -lse * log2(e) (-inf: no gradient), -rowsum(dO * O)
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
int fwd_smem(int d);
int bwd_smem(int d);
cudaError_t fwd_prepare(int d, bool bf16);
cudaError_t bwd_prepare(int d, bool bf16);
cudaError_t fwd_launch(int d, bool bf16, int grid, const FwdParams &p, const FwdMaps &m, cudaStream_t st);
cudaError_t bwd_prep_launch(bool bf16, int n_tiles, const PrepParams &p, cudaStream_t st);
cudaError_t bwd_launch(int d, bool bf16, bool keys, int grid, const BwdParams &p, const BwdMaps &m, cudaStream_t st);
cudaError_t bwd_sum_launch(bool bf16, int n_items, const SumParams &p, cudaStream_t st);

}  // namespace window
}  // namespace syn
