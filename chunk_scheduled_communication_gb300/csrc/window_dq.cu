// window_dq.cu -- gradient of Q of the windowed attention (include/syn_window.h;
// the mathematics at window_dkv.cu).
//
// A CTA keeps 128 query rows of a head, X = Q and Y = dO, and streams blocks of
// 128 keys past them, U = K and W = V:
//
//   S = X U^T, dP = Y W^T   128 x 128 each, into TMEM
//   dS = P (dP - rowsum)    by two warpgroups: one query row a thread, half of
//                           the block's keys a warpgroup
//   dQ += dS U              dS read from TMEM as a 16-bit operand
//
//   warp 0        TMA producer: an item's X and Y, each block's U and W (rings)
//   warps 1, 2    issue S = X U^T and dP = Y W^T
//   warp 3        issues dQ += dS U
//   warp 5        zeroes U rows past the sequence's keys
//   warps 8-11, 12-15  the two warpgroups
//
// TMEM (512 columns): S at 0, free again once loaded; dP at 128 or 256 in turn
// with dS over it; the sum at 384.  W is free as soon as dP is made, U when dQ
// is, so U has three stages and W two.
//
// rowsum(dO O) comes from the stored O, whose rounding is that of a whole value
// row where a query sees few keys: there P dP - P rowsum nearly cancels and the
// rounding shows.  A tile that sees one block only has its row's P and dP at
// hand, so it takes rowsum(P dP) instead and leaves it for dK and dV, whose
// kernel runs after this one.
//
// Measured as window_dkv.cu: 625 us, tensor pipe 57 % active (560 us, 62 %, before
// the tiles of one block took their own rowsum; then blocks of 64 keys in one
// ring, as there: 881 us; both tiles in one ring of two: 840 us).
#include "window.cuh"

namespace syn {
namespace window {

namespace {

constexpr int kBQ = 128, kBK = 128;
constexpr int kBox = 128 * 128;
constexpr int kThreads = 512;
constexpr int kUStages = 3, kWStages = 2;

enum {
    B_XF = 0,                  // the item's X, Y landed
    B_XE = 1,                  // X, Y read by the item's last S, dP (a commit of each issuer)
    B_UF = 2,                  // U stage landed
    B_UE = B_UF + kUStages,    // U stage consumed
    B_WF = B_UE + kUStages,    // W stage landed
    B_WE = B_WF + kWStages,    // W stage consumed
    B_ZR = B_WE + kWStages,    // a U block with rows past the end landed
    B_UZ = B_ZR + 1,           // its rows past the end zeroed
    B_SF = B_UZ + 1,           // S written
    B_SL = B_SF + 1,           // S loaded
    B_DF = B_SL + 1,           // dP written (2)
    B_GF = B_DF + 2,           // dS written (2)
    B_DN = B_GF + 2,           // dQ updated: dS read (2)
    B_AF = B_DN + 2,           // the item's sum complete
    B_OE = B_AF + 1,           // the item's sum read out
    B_DRAIN = B_OE + 1,        // every MMA of an issuer completed (3)
    N_BAR = B_DRAIN + 3
};

template <int D> struct Lay {
    static constexpr int kTile = 128 * D * 2;
    static constexpr int X = 0, Y = kTile;
    static constexpr int U = 2 * kTile;
    static constexpr int W = U + kUStages * kTile;
    static constexpr int SUM = W + kWStages * kTile;  // [2][128] halves of rowsum(P dP)
    static constexpr int BAR = SUM + 2 * 128 * 4;
    static constexpr int MISC = BAR + 8 * N_BAR;
    static constexpr int BYTES = MISC + 16 + 1024;
};

// A key block: first key, its valid keys (128: all), keys computed (a multiple of 16)
struct Blk {
    int start, valid, nk;
};

__device__ __forceinline__ int sink_blocks(const BwdItem &it) { return (it.s_end + kBK - 1) / kBK; }
// (query rows that see no key have one block without a valid key)
__device__ __forceinline__ int blocks_of(const BwdItem &it) {
    return max(1, sink_blocks(it) + (it.k_end - it.w_lo + kBK - 1) / kBK);
}
// Block b of an item, from block b - 1 (b > 0)
__device__ __forceinline__ void step(Blk &k, int b, int n_sink, const BwdItem &it) {
    if (b == 0 || b == n_sink) k.start = b < n_sink ? 0 : it.w_lo;
    else k.start += kBK;
    k.valid = min(kBK, (b < n_sink ? it.s_end : it.k_end) - k.start);
    k.nk = (max(k.valid, 1) + 15) & ~15;
}

template <int N> struct Ring {
    int s = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++s == N) {
            s = 0;
            phase ^= 1u;
        }
    }
};

// The first eight warps keep 72 of the 128 registers launched, the two
// warpgroups take 184: 256 * 72 + 256 * 184 = 65,536.
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 72;"); }
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 184;"); }

// 16-bit pairs of columns 2K, 2K + 1 ..: 0 where not seen
template <int K> struct PairRow {
    static __device__ __forceinline__ void apply(uint32_t (&p)[32], const uint32_t (&seen)[2]) {
        p[K] &= keep_if<2 * K % 32>(seen[K / 16], 0x0000ffffu, 0u) | keep_if<2 * K % 32 + 1>(seen[K / 16], 0xffff0000u, 0u);
        if constexpr (K < 31) PairRow<K + 1>::apply(p, seen);
    }
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) window_dq_kernel(const __grid_constant__ BwdParams p,
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
            const bool warps = i == B_SL || i == B_GF || i == B_GF + 1 || i == B_OE;
            ptx::mbar_init(bar(i), warps ? 8 : i == B_XE ? 2 : 1);
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
    const int i0 = p.begin[blockIdx.x], i1 = p.begin[blockIdx.x + 1];
    const uint32_t one = lane == 0 ? 1u : 0u;

    if (warp < 8) {
        regs_dec();
        Blk b = {};
        uint32_t g = 0;
        Ring<kUStages> u;
        Ring<kWStages> w;
        if (warp == 0) {
            // ================= TMA producer =================
            bool stop = false;
            uint32_t n_x = 0, n_w = 0;  // items whose X and Y, blocks whose W has been issued (g: U)
            for (int i = i0; i < i1 && !stop; ++i) {
                const BwdItem &it = p.items[i];
                const int n_sink = sink_blocks(it), n = blocks_of(it), hk = it.hk, row0 = it.stream0, q_row = it.row0, h = it.h0;
                wait_bar(bar(B_XE), ((uint32_t)(i - i0) & 1u) ^ 1u, abort, c);
                if (aborted(abort)) break;
                ++n_x;
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(bar(B_XF), 2 * L::kTile);
                    for (int x = 0; x < D / 64; ++x) {
                        ptx::tma_load_3d(sbase + L::X + (uint32_t)(x * kBox), &m.x, bar(B_XF), x * 64, h, q_row);
                        ptx::tma_load_3d(sbase + L::Y + (uint32_t)(x * kBox), &m.y, bar(B_XF), x * 64, h, q_row);
                    }
                }
                __syncwarp();
                for (int k = 0; k < n; ++k, u.next(), w.next()) {
                    step(b, k, n_sink, it);
                    wait_bar(bar(B_UE + u.s), u.phase ^ 1u, abort, c);
                    stop = aborted(abort);
                    if (stop) break;
                    ++g;
                    if (lane == 0) {
                        ptx::mbar_arrive_expect_tx(bar(B_UF + u.s), L::kTile);
                        for (int x = 0; x < D / 64; ++x)
                            ptx::tma_load_3d(sbase + (uint32_t)(L::U + u.s * L::kTile + x * kBox), &m.u, bar(B_UF + u.s), x * 64, hk,
                                             row0 + b.start);
                    }
                    __syncwarp();
                    wait_bar(bar(B_WE + w.s), w.phase ^ 1u, abort, c);
                    stop = aborted(abort);
                    if (stop) break;
                    ++n_w;
                    if (lane == 0) {
                        ptx::mbar_arrive_expect_tx(bar(B_WF + w.s), L::kTile);
                        for (int x = 0; x < D / 64; ++x)
                            ptx::tma_load_3d(sbase + (uint32_t)(L::W + w.s * L::kTile + x * kBox), &m.w, bar(B_WF + w.s), x * 64, hk,
                                             row0 + b.start);
                    }
                    __syncwarp();
                }
            }
            // every load issued must land before the CTA exits
            if (n_x > 0) drain_bar(bar(B_XF), (n_x - 1u) & 1u, c);
            for (uint32_t s = 0; s < kUStages; ++s)
                if (g > s) drain_bar(bar(B_UF + (int)s), ((g - 1u - s) / kUStages) & 1u, c);
            for (uint32_t s = 0; s < kWStages; ++s)
                if (n_w > s) drain_bar(bar(B_WF + (int)s), ((n_w - 1u - s) / kWStages) & 1u, c);
        } else if (warp == 1) {
            // ================= S = X U^T =================
            const uint32_t x_d = desc_lo(sbase + L::X, 16), u_d = desc_lo(sbase + L::U, 16);
            uint32_t nz = 0;
            for (int i = i0; i < i1; ++i) {
                const BwdItem &it = p.items[i];
                const int n_sink = sink_blocks(it), n = blocks_of(it);
                wait_bar(bar(B_XF), (uint32_t)(i - i0) & 1u, abort, c);
                for (int k = 0; k < n; ++k, ++g, u.next()) {
                    step(b, k, n_sink, it);
                    const uint32_t id_s = ptx::idesc_16bit_f32(BF16, 128, b.nk, false), ud = u_d + (uint32_t)(u.s * L::kTile >> 4);
                    wait_bar(bar(B_UF + u.s), u.phase, abort, c);
                    if (b.valid < kBK) {
                        arrive_if(one, bar(B_ZR));
                        wait_bar(bar(B_UZ), nz++ & 1u, abort, c);
                    }
                    if (g > 0) wait_bar(bar(B_SL), (g - 1u) & 1u, abort, c);  // S of block g - 1 is loaded
                    ptx::tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const int o = (kk >> 2) * kBox + (kk & 3) * 32;
                        umma_if(one, tmem, desc_at(x_d, o), desc_at(ud, o), id_s, kk != 0 ? 1u : 0u);
                    }
                    commit_if(one, bar(B_SF));
                    if (k == n - 1) commit_if(one, bar(B_XE));
                }
            }
            // every MMA issued must complete before TMEM is released
            commit_if(one, bar(B_DRAIN));
            drain_bar(bar(B_DRAIN), 0, c);
        } else if (warp == 2) {
            // ================= dP = Y W^T =================
            const uint32_t y_d = desc_lo(sbase + L::Y, 16), w_d = desc_lo(sbase + L::W, 16);
            for (int i = i0; i < i1; ++i) {
                const BwdItem &it = p.items[i];
                const int n_sink = sink_blocks(it), n = blocks_of(it);
                wait_bar(bar(B_XF), (uint32_t)(i - i0) & 1u, abort, c);
                for (int k = 0; k < n; ++k, ++g, w.next()) {
                    step(b, k, n_sink, it);
                    const uint32_t id_s = ptx::idesc_16bit_f32(BF16, 128, b.nk, false), wd = w_d + (uint32_t)(w.s * L::kTile >> 4);
                    const uint32_t dst = tmem + 128u + (g & 1u) * 128u;
                    wait_bar(bar(B_WF + w.s), w.phase, abort, c);
                    if (g > 1) wait_bar(bar(B_DN + (int)(g & 1u)), ((g >> 1) - 1u) & 1u, abort, c);  // dS of block g - 2 is read
                    ptx::tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const int o = (kk >> 2) * kBox + (kk & 3) * 32;
                        umma_if(one, dst, desc_at(y_d, o), desc_at(wd, o), id_s, kk != 0 ? 1u : 0u);
                    }
                    commit_if(one, bar(B_DF + (int)(g & 1u)));
                    commit_if(one, bar(B_WE + w.s));
                    if (k == n - 1) commit_if(one, bar(B_XE));
                }
            }
            commit_if(one, bar(B_DRAIN + 1));
            drain_bar(bar(B_DRAIN + 1), 0, c);
        } else if (warp == 3) {
            // ================= dQ += dS U =================
            constexpr uint32_t id_a = ptx::idesc_16bit_f32(BF16, 128, D, true);
            const uint32_t u_d = desc_lo(sbase + L::U, kBox);
            for (int i = i0; i < i1; ++i) {
                const BwdItem &it = p.items[i];
                const int n_sink = sink_blocks(it), n = blocks_of(it);
                if (i > i0) wait_bar(bar(B_OE), (uint32_t)(i - i0 - 1) & 1u, abort, c);  // the sum has been read out
                for (int k = 0; k < n; ++k, ++g, u.next()) {
                    step(b, k, n_sink, it);
                    const uint32_t ud = u_d + (uint32_t)(u.s * L::kTile >> 4), src = tmem + 128u + (g & 1u) * 128u;
                    wait_bar(bar(B_UF + u.s), u.phase, abort, c);
                    wait_bar(bar(B_GF + (int)(g & 1u)), (g >> 1) & 1u, abort, c);
                    ptx::tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk)  // (each warpgroup's columns begin 64 on)
                        umma_ts_if(kk * 16 < b.nk ? one : 0u, tmem + 384u, src + (uint32_t)((kk >> 2) * 64 + (kk & 3) * 8),
                                   desc_at(ud, kk * 2048), id_a, (kk != 0 || k != 0) ? 1u : 0u);
                    commit_if(one, bar(B_DN + (int)(g & 1u)));
                    commit_if(one, bar(B_UE + u.s));
                    if (k == n - 1) commit_if(one, bar(B_AF));
                }
            }
            commit_if(one, bar(B_DRAIN + 2));
            drain_bar(bar(B_DRAIN + 2), 0, c);
        } else if (warp == 5) {
            // ================= U rows past the end =================
            // (asked by the issuer of S, which follows every block: this warp sees
            // only some, and a phase of the stage's own barrier could pass it by)
            uint32_t nz = 0;
            for (int i = i0; i < i1; ++i) {
                const BwdItem &it = p.items[i];
                const int n_sink = sink_blocks(it), n = blocks_of(it);
                for (int k = 0; k < n; ++k, u.next()) {
                    step(b, k, n_sink, it);
                    if (b.valid >= kBK) continue;
                    wait_bar(bar(B_ZR), nz++ & 1u, abort, c);
                    zero_rows<D>(sm + L::U + u.s * L::kTile, kBox, b.valid, b.nk, lane);
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    arrive_if(one, bar(B_UZ));
                }
            }
        }
    } else {
        regs_inc();
        // ================= dS of the warpgroup's columns; half of the items' outputs =================
        const int wg = (warp - 8) >> 2;
        const int qd = warp & 3;
        const int row = qd * 32 + lane, co = 64 * wg;  // this thread's row, the warpgroup's first column
        const uint32_t tl = tmem + ((uint32_t)(qd * 32) << 16);
        const uint64_t scale2 = f2(c.scale_log2, c.scale_log2);
        uint32_t g = 0;
        Blk b = {};
        for (int i = i0; i < i1; ++i) {
            const BwdItem &it = p.items[i];
            const int n_sink = sink_blocks(it), n = blocks_of(it), pos0 = it.pos0, pos = pos0 + row;
            const bool mine = row < it.n_rows;
            const int64_t o = (int64_t)it.h0 * p.pad_rows + it.pad_row0 + (mine ? row : 0);
            const float nl = mine ? p.nlse2[o] : -INFINITY, nd = mine ? p.ndelta[o] : 0.f;
            const uint64_t nl2 = f2(nl, nl);
            uint64_t nd2 = f2(nd, nd);
            for (int k = 0; k < n; ++k, ++g) {
                step(b, k, n_sink, it);
                const uint32_t t_d = tl + (uint32_t)(128 + co) + (g & 1u) * 128u;
                // every row of the tile sees every key of the block?
                const bool full = b.valid == kBK && b.start + kBK - 1 <= pos0 &&
                                  (b.start > pos0 + kBQ - 1 - c.window || b.start + kBK <= c.sinks);
                wait_bar(bar(B_SF), g & 1u, abort, c);
                ptx::tc_fence_after();
                uint32_t v[64], d[64];
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    ptx::tmem_ld_32x32b_x32(tl + (uint32_t)(co + x * 32), *reinterpret_cast<uint32_t(*)[32]>(v + 32 * x));
                ptx::tmem_ld_wait();
                ptx::tc_fence_before();
                __syncwarp();
                arrive_if(one, bar(B_SL));
                uint32_t seen[2] = {0xffffffffu, 0xffffffffu};
                if (!full) {  // columns [lo, hi) and those below sk are seen
                    const int hi = clampi(min(b.valid, pos + 1 - b.start) - co, 0, 64);
                    const int lo = clampi(pos - c.window + 1 - b.start - co, 0, 64);
                    const int sk = clampi(c.sinks - b.start - co, 0, 64);
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        seen[x] = bits_below(hi, 32 * x) & (~bits_below(lo, 32 * x) | bits_below(sk, 32 * x));
                    MaskRow<0, 64>::apply(v, seen, __float_as_uint(-INFINITY));
                }
#pragma unroll
                for (int j = 0; j < 64; j += 2) {
                    float x0, x1;
                    unf2(fma2(f2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), scale2, nl2), x0, x1);
                    v[j] = __float_as_uint(ex2(x0));
                    v[j + 1] = __float_as_uint(ex2(x1));
                }
                wait_bar(bar(B_DF + (int)(g & 1u)), (g >> 1) & 1u, abort, c);
                ptx::tc_fence_after();
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    ptx::tmem_ld_32x32b_x32(t_d + (uint32_t)(x * 32), *reinterpret_cast<uint32_t(*)[32]>(d + 32 * x));
                ptx::tmem_ld_wait();
                if (n == 1) {
                    MaskRow<0, 64>::apply(d, seen, __float_as_uint(-nd));
                    uint64_t sum = f2(0.f, 0.f);
#pragma unroll
                    for (int j = 0; j < 64; j += 2)
                        sum = fma2(f2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])),
                                   add2(f2(__uint_as_float(d[j]), __uint_as_float(d[j + 1])), nd2), sum);
                    float s0, s1;
                    unf2(sum, s0, s1);
                    float *halves = reinterpret_cast<float *>(sm + L::SUM);
                    halves[wg * 128 + row] = s0 + s1;
                    asm volatile("bar.sync 1, 256;" ::: "memory");
                    const float exact = nd - (halves[row] + halves[128 + row]);  // (the halves in their order)
                    asm volatile("bar.sync 1, 256;" ::: "memory");               // (read before they are replaced)
                    nd2 = f2(exact, exact);
                    if (wg == 0 && mine) p.ndelta[o] = exact;
                }
                uint32_t pk[32];
#pragma unroll
                for (int j = 0; j < 64; j += 2) {
                    float y0, y1;
                    unf2(mul2(f2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])),
                              add2(f2(__uint_as_float(d[j]), __uint_as_float(d[j + 1])), nd2)), y0, y1);
                    pk[j >> 1] = pack16<BF16>(y0, y1);
                }
                // columns past the keys: dP there is of another sequence's rows, or stale
                if (b.valid < kBK) PairRow<0>::apply(pk, seen);
                ptx::tmem_st_32x32b_x32(t_d, pk);
                ptx::tmem_st_wait();
                ptx::tc_fence_before();
                __syncwarp();
                arrive_if(one, bar(B_GF + (int)(g & 1u)));
            }
            // the item's sum is complete: each warpgroup writes half of its columns
            wait_bar(bar(B_AF), (uint32_t)(i - i0) & 1u, abort, c);
            ptx::tc_fence_after();
            const int64_t r = it.row0 + row;
            uint16_t *dst = mine ? static_cast<uint16_t *>(p.dx.p) + r * p.dx.token + it.h0 * p.dx.head + wg * (D / 2) : nullptr;
#pragma unroll
            for (int x = 0; x < D / 64; ++x)
                store_cols<BF16>(tl + 384u + (uint32_t)(wg * (D / 2) + x * 32), dst ? dst + x * 32 : nullptr, nullptr, c.scale);
            ptx::tc_fence_before();
            __syncwarp();
            arrive_if(one, bar(B_OE));
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

template <int D, bool BF16> cudaError_t launch(int grid, const BwdParams &p, const BwdMaps &m, cudaStream_t st) {
    return launch_early(window_dq_kernel<D, BF16>, grid, kThreads, Lay<D>::BYTES, st, p, m);
}
template <int D, bool BF16> cudaError_t prepare() {
    return cudaFuncSetAttribute(window_dq_kernel<D, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::BYTES);
}

}  // namespace

cudaError_t dq_prepare(int d, bool bf16) {
    if (d == 64) return bf16 ? prepare<64, true>() : prepare<64, false>();
    return bf16 ? prepare<128, true>() : prepare<128, false>();
}

cudaError_t dq_launch(int d, bool bf16, int grid, const BwdParams &p, const BwdMaps &m, cudaStream_t st) {
    if (d == 64) return bf16 ? launch<64, true>(grid, p, m, st) : launch<64, false>(grid, p, m, st);
    return bf16 ? launch<128, true>(grid, p, m, st) : launch<128, false>(grid, p, m, st);
}

}  // namespace window
}  // namespace syn
