// window_dkv.cu -- gradients of K and V of the windowed attention
// (include/syn_window.h), the statistics they and window_dq.cu read, and the
// joining of partial sums.
//
//   P = exp(scale S - lse),  dP = dO V^T,  dS = P * (dP - rowsum(dO * O))
//   dV = P^T dO,  dK = scale dS^T Q
//
// No sum needs atomics, so the bits do not depend on timing: a CTA keeps 128
// keys and streams query blocks of 64 rows past them, all heads of the group,
// so that shared heads sum in the accumulator; dQ has a kernel of its own, which
// computes the scores again (seven products where five are needed; writing the
// score gradients out instead would move T * W elements a head each way).  With
// X, Y the stationary tiles (K, V) and U, W the streaming ones (Q, dO), a block
// does
//
//   S = X U^T, dP = Y W^T   128 x 64 each, into TMEM
//   P, dS                   by warpgroup g & 1: one key a thread
//   dV += P W, dK += dS U   P and dS read from TMEM as 16-bit operands
//
//   warp 0        TMA producer: an item's X and Y, each block's U and W (ring)
//   warps 1, 2    issue S = X U^T and dP = Y W^T
//   warps 3, 4    issue dK += dS U and dV += P W
//   warp 5        zeroes streaming rows past the sequence's end
//   warps 8-11, 12-15  the two warpgroups
//
// TMEM (512 columns): three places of 64 for S, over which the block's P and dS
// (32 each) stay until their sums are made; one place for dP, free again as
// soon as the warpgroup has loaded it; the sums at 256 and 384.  So three blocks
// are under way at a time.
//
// Measured on one GB300 (bf16, 16384 tokens, 32/8 heads of 128, window 2048, 4
// sinks): 866 us, tensor pipe 59 % active.  It is bound by the round trip of dP's
// one place -- product, commit, load, arrival -- beside products of 64 columns,
// which cost the pipe 48 to 58 cycles where 32 would be the peak's pace.  Blocks
// of 128 queries, S and dP with P and dS over them, had less to overlap (1115
// us); S and dP issued by one warp, dP first, 1290 us.
#include "window.cuh"

namespace syn {
namespace window {

namespace {

constexpr int kBX = 128, kBU = 64;
constexpr int kBoxX = kBX * 128, kBoxU = kBU * 128;
constexpr int kThreads = 512;
constexpr int kStages = 4;

enum {
    B_XF = 0,                  // the item's X, Y landed
    B_XE = 1,                  // X, Y read by the item's last S, dP (a commit of each issuer)
    B_UF = 2,                  // stage landed
    B_UE = B_UF + kStages,     // stage consumed (a commit of each sum's issuer)
    B_ZR = B_UE + kStages,     // a block with rows past the end landed (asked by both S, dP issuers)
    B_UZ = B_ZR + 1,           // its rows past the end zeroed
    B_SF = B_UZ + 1,           // S and dP of block g written (6, g % 6; a commit of each issuer)
    B_TL = B_SF + 6,           // dP of block g loaded into registers
    B_PF = B_TL + 1,           // P, dS of block g written (3, g % 3)
    B_DN = B_PF + 3,           // sums updated by block g (3, g % 3; a commit of each sum's issuer)
    B_AF = B_DN + 3,           // an item's sums complete (a commit of each sum's issuer)
    B_OE = B_AF + 1,           // the item's sums read out
    B_DRAIN = B_OE + 1,        // every MMA of an issuer completed (4)
    N_BAR = B_DRAIN + 4
};

template <int D> struct Lay {
    static constexpr int kTileX = kBX * D * 2, kTileU = kBU * D * 2;
    static constexpr int kStage = 2 * kTileU;
    static constexpr int X = 0, Y = kTileX;
    static constexpr int RING = 2 * kTileX;
    static constexpr int STAT = RING + kStages * kStage;  // [stage][2][64] -lse2, -delta
    static constexpr int BAR = STAT + kStages * 512;
    static constexpr int MISC = BAR + 8 * N_BAR;
    static constexpr int BYTES = MISC + 16 + 1024;
};

// One streaming block of an item
struct Blk {
    int h, start, valid;  // head; first row (of the sequence); rows that exist (64: all)
    bool first, last;
};

struct Walk {
    int i, end, b, h, n;
    const BwdItem *it;
    __device__ __forceinline__ void load(const BwdParams &p) {
        if (i >= end) return;
        it = p.items + i;
        b = 0;
        h = it->h0;
        n = it->b1 - it->b0;
    }
    __device__ __forceinline__ void init(const BwdParams &p) {
        i = p.begin[blockIdx.x];
        end = p.begin[blockIdx.x + 1];
        it = p.items;
        load(p);
    }
    __device__ __forceinline__ bool next(const BwdParams &p, Blk &k) {
        if (i < end && h == it->h1) {
            ++i;
            load(p);
        }
        if (i >= end) return false;
        k.h = h;
        k.first = b == 0 && h == it->h0;
        k.start = (it->b0 + b) * kBU;
        k.valid = min(kBU, it->stream_len - k.start);
        if (++b == n) {
            b = 0;
            ++h;
        }
        k.last = h == it->h1;
        return true;
    }
};

// The first eight warps keep 72 of the 128 registers launched, the two
// warpgroups take 184: 256 * 72 + 256 * 184 = 65,536.
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 72;"); }
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 184;"); }

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) window_dkv_kernel(const __grid_constant__ BwdParams p,
                                                                 const __grid_constant__ BwdMaps m) {
    using L = Lay<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = ptx::smem_u32(sm);
    const uint32_t bar0 = sbase + L::BAR;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L::MISC);
    volatile int *abort = reinterpret_cast<volatile int *>(sm + L::MISC + 4);
    const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
    auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    const Common &c = p.c;

    if (threadIdx.x == 0) {
        *abort = 0;
        for (int i = 0; i < N_BAR; ++i) {
            const bool four = i == B_TL || (i >= B_PF && i < B_PF + 3), eight = i == B_OE;
            const bool products = i == B_XE || i == B_ZR || (i >= B_SF && i < B_SF + 6);
            const bool sums = (i >= B_DN && i < B_DN + 3) || i == B_AF || (i >= B_UE && i < B_UE + kStages);
            ptx::mbar_init(bar(i), four ? 4 : eight ? 8 : products || sums ? 2 : 1);
        }
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
        ptx::tmem_relinquish();
    }
    ptx::grid_wait();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const uint32_t one = lane == 0 ? 1u : 0u;
    if (warp < 8) {
        regs_dec();
        Walk wk;
        wk.init(p);
        Blk b = {};
        if (warp == 0) {
            // ================= TMA producer =================
            uint32_t g = 0, ic = 0;
            for (; wk.next(p, b); ++g) {
                if (b.first) {
                    wait_bar(bar(B_XE), (ic & 1u) ^ 1u, abort, c);
                    if (aborted(abort)) break;
                    if (lane == 0) {
                        ptx::mbar_arrive_expect_tx(bar(B_XF), 2 * L::kTileX);
                        for (int x = 0; x < D / 64; ++x) {
                            ptx::tma_load_3d(sbase + L::X + (uint32_t)(x * kBoxX), &m.x, bar(B_XF), x * 64, wk.it->hk, wk.it->row0);
                            ptx::tma_load_3d(sbase + L::Y + (uint32_t)(x * kBoxX), &m.y, bar(B_XF), x * 64, wk.it->hk, wk.it->row0);
                        }
                    }
                    ++ic;
                }
                const int s = (int)(g % kStages);
                wait_bar(bar(B_UE + s), ((g / kStages) & 1u) ^ 1u, abort, c);
                if (aborted(abort)) break;
                if (lane == 0) {
                    const uint32_t u = sbase + (uint32_t)(L::RING + s * L::kStage);
                    const int row = wk.it->stream0 + b.start;
                    ptx::mbar_arrive_expect_tx(bar(B_UF + s), L::kStage + 512);
                    for (int x = 0; x < D / 64; ++x) {
                        ptx::tma_load_3d(u + (uint32_t)(x * kBoxU), &m.u, bar(B_UF + s), x * 64, b.h, row);
                        ptx::tma_load_3d(u + (uint32_t)(L::kTileU + x * kBoxU), &m.w, bar(B_UF + s), x * 64, b.h, row);
                    }
                    // the block's statistics: 64 rows, aligned in the padded layout
                    const int64_t o = (int64_t)b.h * p.pad_rows + wk.it->pad_row0 + b.start;
                    ptx::bulk_g2s(sbase + (uint32_t)(L::STAT + s * 512), p.nlse2 + o, 256, bar(B_UF + s));
                    ptx::bulk_g2s(sbase + (uint32_t)(L::STAT + s * 512 + 256), p.ndelta + o, 256, bar(B_UF + s));
                }
                __syncwarp();
            }
            // every load issued must land before the CTA exits
            if (ic > 0) drain_bar(bar(B_XF), (ic - 1u) & 1u, c);
            for (uint32_t s = 0; s < kStages; ++s)
                if (g > s) drain_bar(bar(B_UF + (int)s), ((g - 1u - s) / kStages) & 1u, c);
        } else if (warp == 5) {
            // ================= streaming rows past the end =================
            // (asked by the issuers, which follow every block: this warp sees only
            // some, and a phase of the stage's own barrier could pass it by)
            uint32_t nz = 0;
            for (uint32_t g = 0; wk.next(p, b); ++g) {
                if (b.valid >= kBU) continue;
                const int s = (int)(g % kStages);
                wait_bar(bar(B_ZR), nz++ & 1u, abort, c);
                zero_rows<D>(sm + L::RING + s * L::kStage, kBoxU, b.valid, kBU, lane);
                zero_rows<D>(sm + L::RING + s * L::kStage + L::kTileU, kBoxU, b.valid, kBU, lane);
                ptx::fence_proxy_async_smem();
                __syncwarp();
                arrive_if(one, bar(B_UZ));
            }
        } else if (warp <= 2) {
            // ================= S = X U^T (warp 1), dP = Y W^T (warp 2) =================
            const bool is_dp = warp == 2;
            constexpr uint32_t id_s = ptx::idesc_16bit_f32(BF16, 128, kBU, false);
            const uint32_t x_d = desc_lo(sbase + (is_dp ? L::Y : L::X), 16);
            const uint32_t u_d = desc_lo(sbase + L::RING + (is_dp ? L::kTileU : 0), 16);
            uint32_t g = 0, ic = 0, nz = 0;
            for (; wk.next(p, b); ++g) {
                const int s = (int)(g % kStages);
                if (b.first) wait_bar(bar(B_XF), ic++ & 1u, abort, c);
                wait_bar(bar(B_UF + s), (g / kStages) & 1u, abort, c);
                if (b.valid < kBU) {
                    arrive_if(one, bar(B_ZR));
                    wait_bar(bar(B_UZ), nz++ & 1u, abort, c);
                }
                // S: the sums of block g - 3 have read P and dS; dP: block g - 1's is loaded
                if (is_dp) {
                    if (g > 0) wait_bar(bar(B_TL), (g - 1u) & 1u, abort, c);
                } else if (g > 2) {
                    wait_bar(bar(B_DN + (int)(g % 3u)), (g / 3u - 1u) & 1u, abort, c);
                }
                ptx::tc_fence_after();
                const uint32_t u = u_d + (uint32_t)(s * L::kStage >> 4), dst = tmem + (is_dp ? 192u : (g % 3u) * 64u);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    umma_if(one, dst, desc_at(x_d, (kk >> 2) * kBoxX + (kk & 3) * 32), desc_at(u, (kk >> 2) * kBoxU + (kk & 3) * 32),
                            id_s, kk != 0 ? 1u : 0u);
                commit_if(one, bar(B_SF + (int)(g % 6u)));
                if (b.last) commit_if(one, bar(B_XE));
            }
            // every MMA issued must complete before TMEM is released
            commit_if(one, bar(B_DRAIN + warp - 1));
            drain_bar(bar(B_DRAIN + warp - 1), 0, c);
        } else if (warp <= 4) {
            // ================= dX += dS U (warp 3), dY += P W (warp 4) =================
            const bool is_y = warp == 4;
            constexpr uint32_t id_a = ptx::idesc_16bit_f32(BF16, 128, D, true);
            const uint32_t u_d = desc_lo(sbase + L::RING + (is_y ? L::kTileU : 0), kBoxU);
            uint32_t g = 0, item = 0;
            for (; wk.next(p, b); ++g) {
                const int s = (int)(g % kStages);
                if (b.first && item > 0) wait_bar(bar(B_OE), (item - 1u) & 1u, abort, c);  // the sums have been read out
                const uint32_t u = u_d + (uint32_t)(s * L::kStage >> 4);
                const uint32_t src = tmem + (g % 3u) * 64u + (is_y ? 0u : 32u);  // P, dS
                const uint32_t dst = tmem + (is_y ? 384u : 256u);
                wait_bar(bar(B_UF + s), (g / kStages) & 1u, abort, c);
                wait_bar(bar(B_PF + (int)(g % 3u)), (g / 3u) & 1u, abort, c);
                ptx::tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < kBU / 16; ++kk)
                    umma_ts_if(one, dst, src + (uint32_t)(kk * 8), desc_at(u, kk * 2048), id_a, (kk != 0 || !b.first) ? 1u : 0u);
                commit_if(one, bar(B_DN + (int)(g % 3u)));
                commit_if(one, bar(B_UE + s));
                if (b.last) {
                    commit_if(one, bar(B_AF));
                    ++item;
                }
            }
            commit_if(one, bar(B_DRAIN + warp - 1));
            drain_bar(bar(B_DRAIN + warp - 1), 0, c);
        }
    } else {
        regs_inc();
        // ================= P and dS of the warpgroup's blocks; the items' outputs =================
        const int wg = (warp - 8) >> 2;
        const int qd = warp & 3;
        const int row = qd * 32 + lane;
        const uint32_t tl = tmem + ((uint32_t)(qd * 32) << 16);
        const uint64_t scale2 = f2(c.scale_log2, c.scale_log2);
        Walk wk;
        wk.init(p);
        Blk b = {};
        uint32_t item = 0;
        for (uint32_t g = 0; wk.next(p, b); ++g) {
            const BwdItem &it = *wk.it;
            if ((g & 1u) == (uint32_t)wg) {
                const int s = (int)(g % kStages);
                wait_bar(bar(B_SF + (int)(g % 6u)), (g / 6u) & 1u, abort, c);
                const uint32_t ts = tl + (g % 3u) * 64u;
                wait_bar(bar(B_UF + s), (g / kStages) & 1u, abort, c);  // the statistics
                ptx::tc_fence_after();
                uint32_t sv[64], dv[64];
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    ptx::tmem_ld_32x32b_x32(tl + 192u + (uint32_t)(x * 32), *reinterpret_cast<uint32_t(*)[32]>(dv + 32 * x));
                ptx::tmem_ld_wait();
                // dP first: the next block's may take its place
                ptx::tc_fence_before();
                __syncwarp();
                arrive_if(one, bar(B_TL));
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    ptx::tmem_ld_32x32b_x32(ts + (uint32_t)(x * 32), *reinterpret_cast<uint32_t(*)[32]>(sv + 32 * x));
                ptx::tmem_ld_wait();
                // this key is seen by the block's queries [lo, hi); scores of the others
                // are -inf, so P and dS are 0 (rows past the end were zeroed: dP is 0 there)
                const int pos = it.pos0 + row, p0 = it.off + b.start;
                if (p0 < it.pos0 + kBX - 1 || (it.pos0 <= p0 + kBU - 1 - c.window && it.pos0 + kBX > c.sinks)) {
                    const int lo = clampi(pos - p0, 0, kBU), hi = pos < c.sinks ? kBU : clampi(pos + c.window - p0, 0, kBU);
                    const uint32_t seen[2] = {bits_below(hi, 0) & ~bits_below(lo, 0), bits_below(hi, 32) & ~bits_below(lo, 32)};
                    MaskRow<0, kBU>::apply(sv, seen, __float_as_uint(-INFINITY));
                }
                const float4 *st_l = reinterpret_cast<const float4 *>(sm + L::STAT + s * 512);
                uint32_t pk[32], dk[32];
#pragma unroll
                for (int k = 0; k < kBU; k += 4) {
                    const float4 a = st_l[k / 4], d = st_l[16 + k / 4];
                    float x0, x1, x2, x3, y0, y1, y2, y3;
                    unf2(fma2(f2(__uint_as_float(sv[k]), __uint_as_float(sv[k + 1])), scale2, f2(a.x, a.y)), x0, x1);
                    unf2(fma2(f2(__uint_as_float(sv[k + 2]), __uint_as_float(sv[k + 3])), scale2, f2(a.z, a.w)), x2, x3);
                    const float p0_ = ex2(x0), p1_ = ex2(x1), p2_ = ex2(x2), p3_ = ex2(x3);
                    unf2(mul2(f2(p0_, p1_), add2(f2(__uint_as_float(dv[k]), __uint_as_float(dv[k + 1])), f2(d.x, d.y))), y0, y1);
                    unf2(mul2(f2(p2_, p3_), add2(f2(__uint_as_float(dv[k + 2]), __uint_as_float(dv[k + 3])), f2(d.z, d.w))), y2, y3);
                    pk[k / 2] = pack16<BF16>(p0_, p1_);
                    pk[k / 2 + 1] = pack16<BF16>(p2_, p3_);
                    dk[k / 2] = pack16<BF16>(y0, y1);
                    dk[k / 2 + 1] = pack16<BF16>(y2, y3);
                }
                ptx::tmem_st_32x32b_x32(ts, pk);
                ptx::tmem_st_32x32b_x32(ts + 32u, dk);
                ptx::tmem_st_wait();
                ptx::tc_fence_before();
                __syncwarp();
                arrive_if(one, bar(B_PF + (int)(g % 3u)));
            }
            if (b.last) {  // the item's sums are complete
                wait_bar(bar(B_AF), item & 1u, abort, c);
                ptx::tc_fence_after();
                const bool mine = row < it.n_rows;
                const int64_t r = it.row0 + row;
                // warpgroup 0 writes dK, warpgroup 1 dV
                const Out &o = wg == 0 ? p.dx : p.dy;
                uint16_t *dst = nullptr;
                float *part = nullptr;
                if (it.part >= 0) part = p.part + (((int64_t)it.part * 2 + wg) * kBX + row) * D;
                else if (mine) dst = static_cast<uint16_t *>(o.p) + r * o.token + it.hk * o.head;
#pragma unroll
                for (int x = 0; x < D / 32; ++x)
                    store_cols<BF16>(tl + 256u + (uint32_t)(wg * 128 + x * 32), dst ? dst + x * 32 : nullptr,
                                     part ? part + x * 32 : nullptr, wg == 0 ? c.scale : 1.f);
                ptx::tc_fence_before();
                __syncwarp();
                arrive_if(one, bar(B_OE));
                ++item;
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// -lse log2(e) and -rowsum(dO * O) of each row and head into [head][padded row],
// so that a block's 64 statistics are one aligned run.  Eight lanes a row; a
// group's kPrepRows rows are loaded together (HBM bounds the long inputs, the
// latency of a load the short ones).
constexpr int kPrepRows = 4;
template <bool BF16, int D> __global__ void __launch_bounds__(256) window_prep_kernel(const __grid_constant__ PrepParams p) {
    const PrepTile t = p.tiles[blockIdx.x];
    ptx::grid_wait();
    const int sub = (int)threadIdx.x & 7, grp = (int)threadIdx.x >> 3;
    const uint32_t mask = 0xffu << (threadIdx.x & 24u);
    uint4 x[kPrepRows][D / 64], y[kPrepRows][D / 64];
    float l[kPrepRows];
    int r[kPrepRows], h[kPrepRows];
#pragma unroll
    for (int u = 0; u < kPrepRows; ++u) {
        const int i = ((int)blockIdx.y * kPrepRows + u) * 32 + grp;
        r[u] = i / p.H_q;
        h[u] = i - r[u] * p.H_q;
        l[u] = -INFINITY;
        if (r[u] < t.n_rows) {
            const int64_t row = t.row0 + r[u];
            const uint16_t *a = static_cast<const uint16_t *>(p.o) + row * p.o_token + h[u] * p.o_head + sub * 8;
            const uint16_t *b = static_cast<const uint16_t *>(p.d_o) + row * p.do_token + h[u] * p.do_head + sub * 8;
            l[u] = p.lse[row * p.H_q + h[u]];
#pragma unroll
            for (int k = 0; k < D / 64; ++k) {
                x[u][k] = *reinterpret_cast<const uint4 *>(a + k * 64);
                y[u][k] = *reinterpret_cast<const uint4 *>(b + k * 64);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < kPrepRows; ++u) {
        float v = 0.f;
        if (l[u] != -INFINITY) {  // (a row that sees no key has no gradient)
#pragma unroll
            for (int k = 0; k < D / 64; ++k) {
                const uint32_t xs[4] = {x[u][k].x, x[u][k].y, x[u][k].z, x[u][k].w}, ys[4] = {y[u][k].x, y[u][k].y, y[u][k].z, y[u][k].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float2 e, f;
                    if (BF16) {
                        e = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&xs[j]));
                        f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&ys[j]));
                    } else {
                        e = __half22float2(*reinterpret_cast<const __half2 *>(&xs[j]));
                        f = __half22float2(*reinterpret_cast<const __half2 *>(&ys[j]));
                    }
                    v = fmaf(e.x, f.x, fmaf(e.y, f.y, v));
                }
            }
        }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o);
        if (sub == 0 && r[u] < 64) {
            const int64_t at = (int64_t)h[u] * p.pad_rows + t.pad_row0 + r[u];
            p.nlse2[at] = l[u] == -INFINITY ? -INFINITY : -1.4426950408889634f * l[u];
            p.ndelta[at] = -v;
        }
    }
}

// dK, dV tiles that were summed in parts: the parts in their fixed order
template <bool BF16> __global__ void __launch_bounds__(256) window_sum_kernel(const __grid_constant__ SumParams p) {
    const SumItem it = p.items[blockIdx.x];
    ptx::grid_wait();
    const int per = p.d / 8, rows = 256 / per;  // rows of a block: one vector of eight a thread
    const int r = (int)blockIdx.z * rows + (int)threadIdx.x / per, k = (int)threadIdx.x % per * 8;
    if (r < it.n_rows) {
        float v[8] = {};
#pragma unroll 4
        for (int j = 0; j < it.n_parts; ++j) {
            const float4 *src = reinterpret_cast<const float4 *>(
                p.part + (((int64_t)(it.part0 + j) * 2 + blockIdx.y) * kBX + r) * p.d + k);
            const float4 a = src[0], b = src[1];
            v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
            v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
        }
        const float s = blockIdx.y == 0 ? p.scale : 1.f;
        const Out &o = blockIdx.y == 0 ? p.dk : p.dv;
        uint4 w;
        w.x = pack16<BF16>(v[0] * s, v[1] * s);
        w.y = pack16<BF16>(v[2] * s, v[3] * s);
        w.z = pack16<BF16>(v[4] * s, v[5] * s);
        w.w = pack16<BF16>(v[6] * s, v[7] * s);
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(o.p) + (it.row0 + r) * o.token + it.hk * o.head + k) = w;
    }
}

template <int D, bool BF16> cudaError_t launch(int grid, const BwdParams &p, const BwdMaps &m, cudaStream_t st) {
    return launch_early(window_dkv_kernel<D, BF16>, grid, kThreads, Lay<D>::BYTES, st, p, m);
}
template <int D, bool BF16> cudaError_t prepare() {
    return cudaFuncSetAttribute(window_dkv_kernel<D, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::BYTES);
}

}  // namespace

cudaError_t dkv_prepare(int d, bool bf16) {
    if (d == 64) return bf16 ? prepare<64, true>() : prepare<64, false>();
    return bf16 ? prepare<128, true>() : prepare<128, false>();
}

cudaError_t dkv_launch(int d, bool bf16, int grid, const BwdParams &p, const BwdMaps &m, cudaStream_t st) {
    if (d == 64) return bf16 ? launch<64, true>(grid, p, m, st) : launch<64, false>(grid, p, m, st);
    return bf16 ? launch<128, true>(grid, p, m, st) : launch<128, false>(grid, p, m, st);
}

cudaError_t bwd_prep_launch(bool bf16, int n_tiles, const PrepParams &p, cudaStream_t st) {
    const dim3 grid((unsigned)n_tiles, (unsigned)((64 * p.H_q + 32 * kPrepRows - 1) / (32 * kPrepRows)));
    return launch_early(p.d == 64 ? bf16 ? window_prep_kernel<true, 64> : window_prep_kernel<false, 64>
                        : bf16    ? window_prep_kernel<true, 128>
                                  : window_prep_kernel<false, 128>,
                        grid, 256, 0, st, p);
}

cudaError_t bwd_sum_launch(bool bf16, int n_items, const SumParams &p, cudaStream_t st) {
    const dim3 grid((unsigned)n_items, 2, (unsigned)(kBX * p.d / 8 / 256));
    return launch_early(bf16 ? window_sum_kernel<true> : window_sum_kernel<false>, grid, 256, 0, st, p);
}

}  // namespace window
}  // namespace syn
