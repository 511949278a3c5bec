// decode.cu -- windowed attention of one query token per sequence over a paged
// cache, and its C ABI (include/syn_window.h).
//
// Every visible key and value row meets its group's query heads only and is read
// once for each 16 of them, so HBM bounds a full batch and latency a small one
// (groups above 16 heads read their rows several times).  A CTA takes
// one sequence, one kv head, up to 16 of its query heads and one of `splits`
// ranges of the visible keys (the sinks and the window as one index space), 64
// keys a tile.  Each of 128 threads resolves the page of one K or V row of a
// tile ahead and brings the row into a ring with one bulk copy (rows 16 bytes
// apart from their length, so that ldmatrix meets no bank twice); each of four
// warps takes 16 of a tile's keys with a running maximum and sum of its own
// (mma.sync 16 x 8 x 16: a group's few rows could not fill a tcgen05 tile, and
// the tensor pipe is far from the bound).  The warps join through shared
// memory, the ranges through a workspace in the CTA that arrives last, in the
// ranges' order.
//
// Measured on one GB300 (bf16, 32/8 heads of 128): 128 sequences at window 4096,
// 2.15 GB of visible rows, 348 us, 6.2 TB/s, 0.91 of the measured copy rate
// (two stages and three CTAs an SM; three and two 419 us, six and one 802 us; the
// rows of the join that no query head has written too 358 us); three sequences
// at window 1024 9.8 to 10.2 us, a chain of dependent loads (length, page, row; the
// query and the second tile's page beside it: 1 us less) and the join through
// memory (one through the shared memory of a cluster's CTAs: no change).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <string>

#include "host_util.h"
#include "ptx.cuh"
#include "syn_window.h"
#include "window.cuh"

namespace syn {
namespace window {

constexpr int kDecThreads = 128;
constexpr int kTileKeys = 64;
constexpr int kRowsM = 16;         // query heads of a CTA
constexpr int kDecStages = 2;
constexpr int kDecCtas = 3;        // resident on an SM
constexpr int kMaxSplits = 128;
constexpr int kWaves = 6;          // CTAs wanted per resident slot
constexpr int kMinTiles = 1;       // whole tiles wanted for a range

struct DecParams {
    const void *q, *k, *v;
    int64_t q_seq, q_head, o_seq, o_head;
    int64_t k_page, k_token, k_head, v_page, v_token, v_head;
    const int32_t *table, *lens;
    int64_t table_stride, n_pages;
    int32_t cap;                    // keys a sequence's table can name
    int32_t page_size, page_shift;  // page_shift: log2(page_size), -1: not a power of two
    int32_t window, sinks, H_q, H_kv, G, hgroups, splits;
    float scale_log2;
    uint64_t timeout_ns;
    void *o;
    float *lse;
    float *part;        // [slot][split][16 * (D + 2)]: O, m, l
    uint32_t *arrived;  // [slot]
    int32_t *err;
};

namespace {

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D> struct DecLay {
    static constexpr int kRow = D * 2 + 16;
    static constexpr int kTile = kTileKeys * kRow;
    static constexpr int RING = 0;                                    // [stage][K, V]
    static constexpr int VALID = RING + kDecStages * 2 * kTile;       // [stage][64] key can be read
    static constexpr int MERGE = VALID + kDecStages * kTileKeys * 4;  // [4][16] m, [4][16] l
    static constexpr int BAR = MERGE + 2 * 4 * kRowsM * 4;            // a stage's rows landed
    static constexpr int BYTES = BAR + 8 * kDecStages;
    static_assert(BAR >= 2 * kMaxSplits * kRowsM * 4, "the join's factors take the ring's memory");
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kDecThreads, kDecCtas) window_decode_kernel(const __grid_constant__ DecParams p) {
    using L = DecLay<D>;
    extern __shared__ __align__(16) uint8_t sm[];
    const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
    const int g = lane >> 2, t4 = lane & 3;
    // CTA: split fastest, so that a sequence's ranges run together
    const int split = (int)blockIdx.x % p.splits;
    int slot = (int)blockIdx.x / p.splits;
    const int slot_id = slot;
    const int hg = slot % p.hgroups;
    slot /= p.hgroups;
    const int hk = slot % p.H_kv, s = slot / p.H_kv;
    const int h0 = hk * p.G + hg * kRowsM, rows = min(kRowsM, p.G - hg * kRowsM);

    ptx::grid_wait();
    int len = p.lens[s];  // (used after the query's loads are under way)
    uint32_t qf[D / 16][4];
    {
        const uint16_t *q = static_cast<const uint16_t *>(p.q) + (int64_t)s * p.q_seq;
        const uint16_t *ra = q + (int64_t)(h0 + g) * p.q_head, *rb = q + (int64_t)(h0 + g + 8) * p.q_head;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const int c = kk * 16 + t4 * 2;
            qf[kk][0] = g < rows ? *reinterpret_cast<const uint32_t *>(ra + c) : 0u;
            qf[kk][1] = g + 8 < rows ? *reinterpret_cast<const uint32_t *>(rb + c) : 0u;
            qf[kk][2] = g < rows ? *reinterpret_cast<const uint32_t *>(ra + c + 8) : 0u;
            qf[kk][3] = g + 8 < rows ? *reinterpret_cast<const uint32_t *>(rb + c + 8) : 0u;
        }
    }

    const uint32_t sbase = ptx::smem_u32(sm);
    int *valid = reinterpret_cast<int *>(sm + L::VALID);
    auto bar = [&](int st) { return sbase + (uint32_t)(L::BAR + 8 * st); };
    if (threadIdx.x == 0) {
        for (int st = 0; st < kDecStages; ++st) ptx::mbar_init(bar(st), kDecThreads);
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    if (len < 0 || len > p.cap) {
        if (threadIdx.x == 0) atomicCAS(p.err, 0, SYN_ERR_BOUNDS);
        len = max(len, 0);
    }
    // visible keys as indexes 0 .. n_vis - 1: the sinks below w_lo, then [w_lo, len),
    // both without the keys past the table (so that no length makes a CTA walk them)
    const int w_lo = max(len - p.window, 0), s_end = min(min(p.sinks, w_lo), p.cap);
    const int n_vis = s_end + max(min(len, p.cap) - w_lo, 0);
    const int tiles = (n_vis + kTileKeys - 1) / kTileKeys, per = (tiles + p.splits - 1) / p.splits;
    const int t0 = min(split * per, tiles), t1 = min(t0 + per, tiles);

    // thread: row `r` of a tile's keys (threads 0-63) or values (64-127)
    const int r = (int)threadIdx.x & 63;
    const bool is_v = threadIdx.x >= 64;
    const uint16_t *cache = static_cast<const uint16_t *>(is_v ? p.v : p.k) + hk * (is_v ? p.v_head : p.k_head);
    const int64_t page_stride = is_v ? p.v_page : p.k_page, token_stride = is_v ? p.v_token : p.k_token;
    const int32_t *table = p.table != nullptr ? p.table + (int64_t)s * p.table_stride : nullptr;
    // the row's key in a tile, -1 past the last visible one
    auto key_of = [&](int tile) {
        const int i = tile * kTileKeys + r;
        return i >= n_vis ? -1 : i < s_end ? i : w_lo + (i - s_end);
    };
    auto page_of = [&](int j) { return p.page_shift >= 0 ? j >> p.page_shift : j / p.page_size; };
    // the page that holds a key, -1 where there is none (a table's entry may be any number)
    auto lookup = [&](int tile) -> int {
        const int j = tile < t1 ? key_of(tile) : -1;
        if (j < 0) return -1;
        return table != nullptr ? table[page_of(j)] : s;
    };
    auto load = [&](int tile, int st, int page) {
        uint8_t *dst = sm + L::RING + (st * 2 + (is_v ? 1 : 0)) * L::kTile + r * L::kRow;
        bool real = page >= 0 && page < p.n_pages;
        if (!real && key_of(tile) >= 0) atomicCAS(p.err, 0, SYN_ERR_BOUNDS);
        if (!is_v) valid[st * kTileKeys + r] = real;
        if (real) {
            const int j = key_of(tile), at = j - page_of(j) * p.page_size;
            ptx::mbar_arrive_expect_tx(bar(st), D * 2);
            ptx::bulk_g2s(ptx::smem_u32(dst), cache + page * page_stride + at * token_stride, D * 2, bar(st));
        } else {
#pragma unroll
            for (int c = 0; c < D / 8; ++c) reinterpret_cast<uint4 *>(dst)[c] = make_uint4(0, 0, 0, 0);
            ptx::mbar_arrive(bar(st));
        }
    };
    // the rows of the stage landed; left by a warp's lanes together.  A wait past
    // the limit is reported and goes on for kDrainNs, so that no copy is under way
    // when its memory is used for something else; one past that too is given up.
    auto landed = [&](int st, uint32_t parity) {
        bool ok = poll_bar(bar(st), parity);
        if (!ok) {
            const uint64_t begin = ptx::globaltimer();
            uint64_t limit = p.timeout_ns;
            while (!(ok = poll_bar(bar(st), parity))) {
                if (ptx::globaltimer() - begin <= limit) continue;
                if (limit != p.timeout_ns) break;
                atomicCAS(p.err, 0, SYN_ERR_TIMEOUT);
                limit += kDrainNs;
            }
        }
        __syncwarp();
        return ok;
    };
    int page = lookup(t0), ahead = lookup(t0 + 1);
    __syncthreads();  // the barriers are initialised

    float o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[n][x] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // rows g and g + 8

    static_assert(kDecStages == 2, "one tile ahead");
    if (t0 < t1) load(t0, 0, page);
    page = ahead;
    bool lost = false;  // a wait was given up: nothing more is loaded or waited for
    for (int t = t0; t < t1; ++t) {
        const int st = (t - t0) % kDecStages;
        if (t > t0) __syncthreads();  // the stage read last is free
        if (t + kDecStages - 1 < t1 && !lost) load(t + kDecStages - 1, (t - t0 + kDecStages - 1) % kDecStages, page);
        page = lookup(t + kDecStages);
        if (!lost) lost = !landed(st, (uint32_t)((t - t0) / kDecStages) & 1u);
        const uint32_t kd = sbase + (uint32_t)(L::RING + st * 2 * L::kTile), vd = kd + L::kTile;
        float sc[2][4] = {};
        {
            const int row = warp * 16 + (lane >> 4) * 8 + (lane & 7);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t b[4];
                const int c = 2 * kk + ((lane >> 3) & 1);
                ldsm(b, kd + (uint32_t)(row * L::kRow + c * 16));
                mma<BF16>(sc[0], qf[kk], b[0], b[1]);
                mma<BF16>(sc[1], qf[kk], b[2], b[3]);
            }
        }
        // keys that do not exist or cannot be read
        const int *ok = valid + st * kTileKeys + warp * 16 + t4 * 2;
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                sc[n][x] = ok[n * 8 + (x & 1)] ? sc[n][x] * p.scale_log2 : -INFINITY;
                mx[x >> 1] = fmaxf(mx[x >> 1], sc[n][x]);
            }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
            mx[r] = fmaxf(mx[r], m[r]);
            const float alpha = mx[r] == -INFINITY ? 1.f : ex2(m[r] - mx[r]);
            m[r] = mx[r];
            l[r] *= alpha;
            if (alpha != 1.f) {
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    o[n][2 * r] *= alpha;
                    o[n][2 * r + 1] *= alpha;
                }
            }
        }
        const float base[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
        uint32_t pf[4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            float e[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) e[x] = ex2(sc[n][x] - base[x >> 1]);
            l[0] += e[0] + e[1];
            l[1] += e[2] + e[3];
            pf[2 * n] = pack16<BF16>(e[0], e[1]);
            pf[2 * n + 1] = pack16<BF16>(e[2], e[3]);
        }
        {
            const int row = warp * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
            for (int nn = 0; nn < D / 16; ++nn) {
                uint32_t b[4];
                const int c = 2 * nn + (lane >> 4);
                ldsm_t(b, vd + (uint32_t)(row * L::kRow + c * 16));
                mma<BF16>(o[2 * nn], pf, b[0], b[1]);
                mma<BF16>(o[2 * nn + 1], pf, b[2], b[3]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
    __syncthreads();
    // join the warps: O of each scaled to the common maximum, in the ring's memory
    float *mm = reinterpret_cast<float *>(sm + L::MERGE), *ll = mm + 4 * kRowsM;
    float *os = reinterpret_cast<float *>(sm);  // [4][16][D]
    if (t4 == 0) {
        mm[warp * kRowsM + g] = m[0];
        mm[warp * kRowsM + g + 8] = m[1];
        ll[warp * kRowsM + g] = l[0];
        ll[warp * kRowsM + g + 8] = l[1];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = g + 8 * r;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) top = fmaxf(top, mm[w * kRowsM + row]);
        const float f = m[r] == -INFINITY ? 1.f : ex2(m[r] - top);  // (no key: O is 0, or NaN from NaN scores)
        if (row >= rows) continue;  // (a row that no query head has)
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
            *reinterpret_cast<float2 *>(os + (warp * kRowsM + row) * D + n * 8 + t4 * 2) =
                make_float2(o[n][2 * r] * f, o[n][2 * r + 1] * f);
    }
    __syncthreads();
    // thread: two columns of every (128 / (D / 2))th row
    constexpr int kCols = D / 2, kRowsAt = kDecThreads / kCols;
    const int col = ((int)threadIdx.x % kCols) * 2;
    constexpr int kPart = kRowsM * (D + 2);
    float *part = p.part + ((int64_t)slot_id * p.splits) * kPart;
    auto write = [&](int row, float2 v, float top, float sum) {
        const bool none = sum == 0.f;
        const float inv = none ? 0.f : 1.f / sum;
        uint16_t *dst = static_cast<uint16_t *>(p.o) + (int64_t)s * p.o_seq + (int64_t)(h0 + row) * p.o_head + col;
        *reinterpret_cast<uint32_t *>(dst) = none ? 0u : pack16<BF16>(v.x * inv, v.y * inv);
        if (p.lse != nullptr && col == 0)
            p.lse[(int64_t)s * p.H_q + h0 + row] = none ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
    };
    for (int row = (int)threadIdx.x / kCols; row < rows; row += kRowsAt) {
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) top = fmaxf(top, mm[w * kRowsM + row]);
        float2 v = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float mw = mm[w * kRowsM + row];
            sum += ll[w * kRowsM + row] * (mw == -INFINITY ? 1.f : ex2(mw - top));
            const float2 x = *reinterpret_cast<const float2 *>(os + (w * kRowsM + row) * D + col);
            v.x += x.x;
            v.y += x.y;
        }
        if (p.splits == 1) {
            write(row, v, top, sum);
        } else {
            float *dst = part + (int64_t)split * kPart;
            *reinterpret_cast<float2 *>(dst + row * D + col) = v;
            if (col == 0) {
                dst[kRowsM * D + row] = top;
                dst[kRowsM * D + kRowsM + row] = sum;
            }
        }
    }
    if (p.splits == 1) return;
    // the range that arrives last joins all of them, in their order
    __shared__ uint32_t last;
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();  // (the block's partial results, seen through the barrier)
        last = ptx::atom_add_acq_rel_gpu(p.arrived + slot_id, 1u) == (uint32_t)p.splits - 1u;
        if (last) p.arrived[slot_id] = 0u;  // for the next call
        __threadfence();
    }
    __syncthreads();
    if (!last) return;
    // each range's factor exp2(m - top) and the sums, all loads at once
    float *fm = reinterpret_cast<float *>(sm), *fl = fm + kMaxSplits * kRowsM;  // [split][16]
    for (int i = (int)threadIdx.x; i < p.splits * kRowsM; i += kDecThreads) {
        const float *src = part + (int64_t)(i / kRowsM) * kPart + kRowsM * D + i % kRowsM;
        fm[i] = __ldcg(src);
        fl[i] = __ldcg(src + kRowsM);
    }
    __syncthreads();
    for (int row = (int)threadIdx.x / kCols; row < rows; row += kRowsAt) {
        float top = -INFINITY, sum = 0.f;
        for (int x = 0; x < p.splits; ++x) top = fmaxf(top, fm[x * kRowsM + row]);
        float2 v = make_float2(0.f, 0.f);
#pragma unroll 8
        for (int x = 0; x < p.splits; ++x) {
            const float mw = fm[x * kRowsM + row];
            const float f = mw == -INFINITY ? 1.f : ex2(mw - top);
            sum += fl[x * kRowsM + row] * f;
            const float2 y = __ldcg(reinterpret_cast<const float2 *>(part + (int64_t)x * kPart + row * D + col));
            v.x = fmaf(y.x, f, v.x);
            v.y = fmaf(y.y, f, v.y);
        }
        write(row, v, top, sum);
    }
}

template <int D, bool BF16> cudaError_t dec_prepare() {
    return cudaFuncSetAttribute(window_decode_kernel<D, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, DecLay<D>::BYTES);
}
template <int D, bool BF16> cudaError_t dec_launch(int grid, const DecParams &p, cudaStream_t st) {
    return launch_early(window_decode_kernel<D, BF16>, grid, kDecThreads, DecLay<D>::BYTES, st, p);
}

}  // namespace
}  // namespace window
}  // namespace syn

using namespace syn;
using namespace syn::window;

struct syn_decode_plan_s {
    syn_decode_cfg_t cfg;
    int device = 0, num_sms = 0, hgroups = 1;
    int slots = 0;  // resident CTAs the splitting aims at
    bool bf16 = true;
    float *d_part = nullptr;
    uint32_t *d_arrived = nullptr;
    int32_t *d_err = nullptr;
};

namespace {

#define DEC_CK(call)                                                                                  \
    do {                                                                                              \
        cudaError_t e__ = (call);                                                                     \
        if (e__ != cudaSuccess) return host_fail(SYN_ERR_CUDA, std::string(#call) + ": " + cudaGetErrorString(e__)); \
    } while (0)

bool al16(const void *x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; }

// (a stride of an axis with one entry is never used)
int check_cache(const char *name, const syn_window_cache_t *c, int64_t pages, int page_size, int heads) {
    if (c == nullptr || (pages > 0 && c->p == nullptr)) return host_fail(SYN_ERR_INVALID, std::string(name) + ": null operand");
    if (!al16(c->p)) return host_fail(SYN_ERR_INVALID, std::string(name) + ": operand not 16-byte aligned");
    if ((pages > 1 && c->page % 8 != 0) || (page_size > 1 && c->token % 8 != 0) || (heads > 1 && c->head % 8 != 0))
        return host_fail(SYN_ERR_INVALID, std::string(name) + ": strides must be multiples of 8 elements");
    return SYN_OK;
}

int check_query(const char *name, const syn_window_rows_t *r, int rows, int heads) {
    if (r == nullptr || r->p == nullptr) return host_fail(SYN_ERR_INVALID, std::string(name) + ": null operand");
    if (!al16(r->p) || (rows > 1 && r->token % 8 != 0) || (heads > 1 && r->head % 8 != 0))
        return host_fail(SYN_ERR_INVALID, std::string(name) + ": not 16-byte aligned, or strides not multiples of 8 elements");
    return SYN_OK;
}

}  // namespace

extern "C" {

int syn_decode_cfg_default(syn_decode_cfg_t *c) {
    if (c == nullptr) return host_fail(SYN_ERR_INVALID, "null cfg");
    std::memset(c, 0, sizeof(*c));
    c->dtype = SYN_DTYPE_BF16;
    c->max_seqs = 1;
    c->H_q = c->H_kv = 1;
    c->d = 128;
    c->page_size = 64;
    return SYN_OK;
}

int syn_decode_plan_create(syn_decode_plan_t *out, const syn_decode_cfg_t *cfg) {
    if (out == nullptr || cfg == nullptr) return host_fail(SYN_ERR_INVALID, "null argument");
    *out = nullptr;
    syn_decode_cfg_t c = *cfg;
    if (c.dtype == SYN_DTYPE_F32) return host_fail(SYN_ERR_UNSUPPORTED, "attention takes bf16 or fp16");
    if (c.dtype != SYN_DTYPE_BF16 && c.dtype != SYN_DTYPE_F16) return host_fail(SYN_ERR_INVALID, "unknown dtype");
    if (c.max_seqs < 1) return host_fail(SYN_ERR_INVALID, "max_seqs must be positive");
    if (c.max_seqs > 65536) return host_fail(SYN_ERR_UNSUPPORTED, "max_seqs > 65536");
    if (c.H_q < 1 || c.H_kv < 1 || c.H_q % c.H_kv != 0) return host_fail(SYN_ERR_INVALID, "need H_q % H_kv == 0");
    if (c.H_q > 1024) return host_fail(SYN_ERR_UNSUPPORTED, "H_q > 1024");
    if (c.d != 64 && c.d != 128) return host_fail(SYN_ERR_UNSUPPORTED, "head dimension must be 64 or 128");
    if (c.window < 0 || c.sinks < 0) return host_fail(SYN_ERR_INVALID, "window and sinks must not be negative");
    if (c.page_size < 1) return host_fail(SYN_ERR_INVALID, "page_size must be positive");
    if (!(c.scale >= 0.f) || !std::isfinite(c.scale)) return host_fail(SYN_ERR_INVALID, "bad scale");
    if (c.window == 0 || c.window > kNoWindow) c.window = kNoWindow;
    c.sinks = std::min(c.sinks, kNoWindow);
    if (c.scale == 0.f) c.scale = 1.f / std::sqrt((float)c.d);
    syn_decode_plan_s *pl = new syn_decode_plan_s();
    pl->cfg = c;
    pl->bf16 = c.dtype == SYN_DTYPE_BF16;
    pl->hgroups = (c.H_q / c.H_kv + kRowsM - 1) / kRowsM;
    cudaError_t e = cudaGetDevice(&pl->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&pl->num_sms, cudaDevAttrMultiProcessorCount, pl->device);
    if (e == cudaSuccess)
        e = c.d == 64 ? (pl->bf16 ? dec_prepare<64, true>() : dec_prepare<64, false>())
                      : (pl->bf16 ? dec_prepare<128, true>() : dec_prepare<128, false>());
    pl->slots = pl->num_sms * kDecCtas;
    // at most slots * kWaves + (one a slot) partial results
    const size_t n = (size_t)c.max_seqs * c.H_kv * pl->hgroups, parts = n + (size_t)pl->slots * kWaves;
    if (e == cudaSuccess) e = cudaMalloc(&pl->d_part, parts * kRowsM * (size_t)(c.d + 2) * sizeof(float));
    if (e == cudaSuccess) e = cudaMalloc(&pl->d_arrived, n * sizeof(uint32_t));
    if (e == cudaSuccess) e = cudaMemset(pl->d_arrived, 0, n * sizeof(uint32_t));
    if (e == cudaSuccess) e = cudaMalloc(&pl->d_err, sizeof(int32_t));
    if (e == cudaSuccess) e = cudaMemset(pl->d_err, 0, sizeof(int32_t));
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) {
        syn_decode_plan_destroy(pl);
        return host_fail(SYN_ERR_CUDA, std::string("decode plan: ") + cudaGetErrorString(e));
    }
    *out = pl;
    return SYN_OK;
}

int syn_decode_plan_destroy(syn_decode_plan_t pl) {
    if (pl == nullptr) return SYN_OK;
    cudaFree(pl->d_part);
    cudaFree(pl->d_arrived);
    cudaFree(pl->d_err);
    delete pl;
    return SYN_OK;
}

int syn_window_decode(syn_decode_plan_t pl, const syn_window_rows_t *q, const syn_window_cache_t *k,
                      const syn_window_cache_t *v, const int32_t *page_table, int64_t table_stride, int64_t n_pages,
                      const int32_t *seq_lens, int n_seqs, const syn_window_rows_t *O, float *lse, void *stream) {
    if (pl == nullptr) return host_fail(SYN_ERR_INVALID, "null plan");
    const syn_decode_cfg_t &c = pl->cfg;
    if (n_seqs < 0 || n_seqs > c.max_seqs) return host_fail(SYN_ERR_INVALID, "n_seqs must be in [0, max_seqs]");
    if (n_seqs == 0) return SYN_OK;
    int rc;
    if ((rc = check_query("q", q, n_seqs, c.H_q)) != SYN_OK || (rc = check_query("O", O, n_seqs, c.H_q)) != SYN_OK ||
        (rc = check_cache("k", k, n_pages, c.page_size, c.H_kv)) != SYN_OK ||
        (rc = check_cache("v", v, n_pages, c.page_size, c.H_kv)) != SYN_OK)
        return rc;
    if ((n_seqs > 1 && O->token < c.d) || (c.H_q > 1 && O->head < c.d)) return host_fail(SYN_ERR_INVALID, "O: output rows overlap");
    if (seq_lens == nullptr) return host_fail(SYN_ERR_INVALID, "null seq_lens");
    if (n_pages < 0 || n_pages >= (int64_t)1 << 31) return host_fail(SYN_ERR_INVALID, "n_pages must be in [0, 2^31)");
    if (page_table != nullptr && table_stride < 0) return host_fail(SYN_ERR_INVALID, "negative table_stride");
    if (page_table == nullptr && n_pages < n_seqs) return host_fail(SYN_ERR_INVALID, "without a page table every sequence needs a page");
    if ((reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return host_fail(SYN_ERR_INVALID, "lse: not aligned");
    DecParams p;
    std::memset(&p, 0, sizeof(p));
    p.q = q->p;
    p.q_seq = q->token;
    p.q_head = q->head;
    p.o = O->p;
    p.o_seq = O->token;
    p.o_head = O->head;
    p.k = k->p;
    p.k_page = k->page;
    p.k_token = k->token;
    p.k_head = k->head;
    p.v = v->p;
    p.v_page = v->page;
    p.v_token = v->token;
    p.v_head = v->head;
    p.table = page_table;
    p.table_stride = table_stride;
    p.n_pages = n_pages;
    // (no more than the indexes of a tile that starts below it reach in 32 bits)
    const int64_t pages = page_table != nullptr ? std::min<int64_t>(table_stride, (int64_t)1 << 31) : 1;
    p.cap = (int32_t)std::min<int64_t>(pages * c.page_size, 0x7fffffff - kTileKeys);
    p.lens = seq_lens;
    p.page_size = c.page_size;
    p.window = (int32_t)c.window;
    p.sinks = c.sinks;
    p.H_q = c.H_q;
    p.H_kv = c.H_kv;
    p.G = c.H_q / c.H_kv;
    p.hgroups = pl->hgroups;
    p.scale_log2 = c.scale * 1.4426950408889634f;
    p.lse = lse;
    p.part = pl->d_part;
    p.arrived = pl->d_arrived;
    p.err = pl->d_err;
    p.timeout_ns = host_timeout_ns();
    p.page_shift = -1;
    for (int b = 0; b < 31; ++b)
        if (c.page_size == 1 << b) p.page_shift = b;
    // Ranges: enough CTAs for kWaves rounds of the resident ones, but no more of
    // them than whole tiles that the longest sequence the table allows has.  The
    // count is rounded down and a range's tiles up, so 17 tiles (window 1024 and a
    // few sinks) make 16 ranges of two, of which nine have any.
    const int64_t n = (int64_t)n_seqs * c.H_kv * pl->hgroups;
    const int64_t longest = std::min<int64_t>(p.cap, c.window + (int64_t)c.sinks);
    const int64_t most = std::min<int64_t>(kMaxSplits, std::max<int64_t>(1, longest / (kTileKeys * kMinTiles)));
    p.splits = (int32_t)std::min<int64_t>(most, ((int64_t)pl->slots * kWaves + n - 1) / n);
    const int grid = (int)(n * p.splits);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (c.d == 64) DEC_CK((pl->bf16 ? dec_launch<64, true>(grid, p, st) : dec_launch<64, false>(grid, p, st)));
    else DEC_CK((pl->bf16 ? dec_launch<128, true>(grid, p, st) : dec_launch<128, false>(grid, p, st)));
    return SYN_OK;
}

int syn_decode_sync_status(syn_decode_plan_t pl, void *stream) {
    if (pl == nullptr) return host_fail(SYN_ERR_INVALID, "null plan");
    DEC_CK(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)));
    int32_t e = 0;
    DEC_CK(cudaMemcpy(&e, pl->d_err, sizeof(e), cudaMemcpyDeviceToHost));
    if (e == 0) return SYN_OK;
    DEC_CK(cudaMemset(pl->d_err, 0, sizeof(e)));
    DEC_CK(cudaDeviceSynchronize());  // (cleared before a later call, of whatever stream, can report)
    return host_fail(e, e == SYN_ERR_TIMEOUT ? "decode: rows of the cache did not arrive within the time limit"
                                             : "decode: a length, table entry or page out of range; those keys were left out");
}

}  // extern "C"
