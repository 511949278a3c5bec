// window_fwd.cu -- forward of the windowed attention (include/syn_window.h).
//
// A persistent CTA (one per SM) takes its list of work items in turn: two
// 128-row query tiles (t = 0, 1) that read the same key blocks.  With an even
// group of query heads the two tiles are the same rows of two heads of the
// group, so both have the same mask and no block is wasted on one of them;
// else they are consecutive rows of one head.  A block is kBK keys, or a
// multiple of 16 for the sinks and the end of a range, so that four sink keys
// cost a fifth of a block.  The online softmax keeps a running maximum and sum
// per row, one pass over the keys:
//
//   warp 0      TMA producer: an item's Q tiles, each block's K and V (rings)
//   warps 1, 3  MMA issuers, one per tile: S_t = Q_t.K^T, then O_t += P_t.V
//   warp 2      zeroes V rows past the end of a block's keys: their probabilities
//               are 0, and 0 times another sequence's inf or NaN is not
//   warps 4-7   softmax of tile 0 (one query row per thread, its TMEM lane)
//   warps 8-11  softmax of tile 1
//
// TMEM (512 columns) holds each tile's scores, probabilities (16-bit, half as
// many columns) and output side by side, so that the scores of block g+1 are
// computed while the softmax works on block g: it frees the score columns as
// soon as it has loaded them, and nothing waits for P.V but the next block's
// probabilities.  With D 128 that fits blocks of 80 keys (80 + 40 + 128 columns
// a tile), with D 64 blocks of 128 (128 + 64 + 64).  The reference maximum of
// the exponentials may lag the row's by up to 8 (log2 units), so the
// accumulator is rescaled only when a block raises it by more.
#include "window.cuh"

namespace syn {
namespace window {

namespace {

constexpr int kBQ = 128, kTiles = 2;
constexpr int kBoxQ = kBQ * 128;  // 128 rows x 128 bytes
constexpr int kThreads = 384;
constexpr int kSmemItems = 48;   // items of the CTA's list kept in shared memory
constexpr float kRescale = 8.f;

constexpr int kMaxStages = 4;
enum {
    B_QF = 0,                     // the item's Q tiles landed
    B_QE = 1,                     // Q tiles read by the item's last Q.K^T (one commit per issuer)
    B_KF = 2,                     // K stage landed
    B_KE = B_KF + kMaxStages,     // K stage consumed (one commit per issuer)
    B_VF = B_KE + kMaxStages,     // V stage landed
    B_VE = B_VF + kMaxStages,     // V stage consumed (one commit per issuer)
    B_SF = B_VE + kMaxStages,     // tile t's scores written (2)
    B_SL = B_SF + 2,              // tile t's scores loaded into registers (2)
    B_PF = B_SL + 2,              // tile t's probabilities written (2)
    B_PV = B_PF + 2,              // tile t's P.V done (2)
    B_OE = B_PV + 2,              // tile t's accumulator read out (2)
    B_DRAIN = B_OE + 2,           // every MMA of tile t's issuer completed (2)
    B_ZR = B_DRAIN + 2,           // a V block with rows past its keys landed (asked by both issuers)
    B_VZ = B_ZR + 1,              // its rows past the keys zeroed
    N_BAR = B_VZ + 1
};

template <int D> struct Lay {
    static constexpr int kBK = D == 128 ? 80 : 128;  // keys of a block
    static constexpr int kStages = D == 128 ? 3 : 4;
    static constexpr int kBoxK = kBK * 128;
    static constexpr int kTileQ = kBQ * D * 2, kTileK = kBK * D * 2;
    static constexpr int Q = 0;
    static constexpr int K = Q + kTiles * kTileQ;
    static constexpr int V = K + kStages * kTileK;
    static constexpr int ITEMS = V + kStages * kTileK;
    static constexpr int BAR = ITEMS + kSmemItems * (int)sizeof(FwdItem);
    static constexpr int MISC = BAR + 8 * N_BAR;
    static constexpr int USED = MISC + 16;
    static constexpr int BYTES = USED + 1024;  // + the 1024-byte alignment of the tiles
    // TMEM columns of tile t
    __host__ __device__ static constexpr uint32_t S(int t) { return 128u * (uint32_t)t; }
    __host__ __device__ static constexpr uint32_t P(int t) { return D == 128 ? 128u * (uint32_t)t + 80u : 384u + 64u * (uint32_t)t; }
    __host__ __device__ static constexpr uint32_t O(int t) { return 256u + (uint32_t)(D * t); }
};

// One key block of an item
struct Blk {
    int kv0, kend, nk;  // first key, end of its valid keys, keys computed (a multiple of 16)
    bool first, last;
};

// The CTA's walk over its items' blocks; every role makes the same one.
template <int kBK> struct Walk {
    int i, end, b;
    const FwdItem *list;  // shared-memory copy
    const FwdItem *rest;  // global list
    const FwdItem *it;
    __device__ __forceinline__ void load() {
        it = i < kSmemItems ? list + i : rest + i;  // (read only while i < end)
        b = 0;
    }
    __device__ __forceinline__ void init(const FwdParams &p, const FwdItem *smem_items) {
        const int b0 = p.begin[blockIdx.x];
        list = smem_items;
        rest = p.items + b0;
        i = 0;
        end = p.begin[blockIdx.x + 1] - b0;
        load();
    }
    // the next block; `it` is its item until the next call
    __device__ __forceinline__ bool next(Blk &k) {
        if (i < end && b == it->n_blk) {
            ++i;
            load();
        }
        if (i >= end) return false;
        const int n_sink = (it->s_end + kBK - 1) / kBK;
        const bool sink = b < n_sink;
        k.kv0 = sink ? b * kBK : it->w_lo + (b - n_sink) * kBK;
        k.kend = sink ? it->s_end : it->k_end;
        k.nk = min(kBK, (k.kend - k.kv0 + 15) & ~15);
        k.first = b == 0;
        ++b;
        k.last = b == it->n_blk;
        return true;
    }
};

template <bool BF16, int D> __device__ __forceinline__ void store_row(void *dst_row, uint32_t to, float inv) {
    uint4 *dst = reinterpret_cast<uint4 *>(dst_row);
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32];
        ptx::tmem_ld_32x32b_x32(to + (uint32_t)(c * 32), v);
        ptx::tmem_ld_wait();
        if (dst != nullptr) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint4 o;
                o.x = pack16<BF16>(__uint_as_float(v[8 * k + 0]) * inv, __uint_as_float(v[8 * k + 1]) * inv);
                o.y = pack16<BF16>(__uint_as_float(v[8 * k + 2]) * inv, __uint_as_float(v[8 * k + 3]) * inv);
                o.z = pack16<BF16>(__uint_as_float(v[8 * k + 4]) * inv, __uint_as_float(v[8 * k + 5]) * inv);
                o.w = pack16<BF16>(__uint_as_float(v[8 * k + 6]) * inv, __uint_as_float(v[8 * k + 7]) * inv);
                dst[c * 4 + k] = o;
            }
        }
    }
}

// Register split: the launch gives 168 a thread (384 threads); the producer,
// issuer and zeroing warps give theirs down to 96, the softmax warps take 200:
// 128 * 96 + 256 * 200 = 63,488 of 64,512.
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 96;"); }
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 200;"); }

template <bool B> struct Bool {
    static constexpr bool value = B;
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) window_fwd_kernel(const __grid_constant__ FwdParams p,
                                                                 const __grid_constant__ FwdMaps m) {
    using L = Lay<D>;
    constexpr int kBK = L::kBK, kStages = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = ptx::smem_u32(sm);
    const uint32_t bar0 = sbase + L::BAR;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L::MISC);
    volatile int *abort = reinterpret_cast<volatile int *>(sm + L::MISC + 4);
    FwdItem *items = reinterpret_cast<FwdItem *>(sm + L::ITEMS);
    const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
    auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    const Common &c = p.c;

    if (threadIdx.x == 0) {
        *abort = 0;
        for (int i = 0; i < N_BAR; ++i) {
            const bool pair = i == B_QE || i == B_ZR || (i >= B_KE && i < B_KE + kMaxStages) || (i >= B_VE && i < B_VE + kMaxStages);
            const bool warps = i == B_SL || i == B_SL + 1 || i == B_PF || i == B_PF + 1 || i == B_OE || i == B_OE + 1;
            ptx::mbar_init(bar(i), pair ? kTiles : warps ? 4 : 1);
        }
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    {
        const int b0 = p.begin[blockIdx.x], n = min(p.begin[blockIdx.x + 1] - b0, kSmemItems);
        const uint4 *src = reinterpret_cast<const uint4 *>(p.items + b0);
        for (int i = (int)threadIdx.x; i < n * (int)(sizeof(FwdItem) / 16); i += kThreads)
            reinterpret_cast<uint4 *>(items)[i] = src[i];
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t sQ = sbase + L::Q, sK = sbase + L::K, sV = sbase + L::V;

    if (warp < 4) {
        regs_dec();
        Walk<kBK> wk;
        wk.init(p, items);
        Blk b = {};
        if (warp == 0) {
            // ================= TMA producer =================
            if (lane == 0) {
                uint32_t g = 0, ic = 0, nk = 0, nv = 0;
                auto load = [&](uint32_t dst, const CUtensorMap *full, const CUtensorMap *narrow, uint32_t br, int row) {
                    ptx::mbar_arrive_expect_tx(br, (uint32_t)(b.nk * D * 2));
                    for (int x = 0; x < D / 64; ++x) {
                        if (b.nk == kBK) {
                            ptx::tma_load_3d(dst + (uint32_t)(x * L::kBoxK), full, br, x * 64, wk.it->hk, row);
                        } else {
                            for (int r = 0; r < b.nk; r += 16)
                                ptx::tma_load_3d(dst + (uint32_t)(x * L::kBoxK + r * 128), narrow, br, x * 64, wk.it->hk, row + r);
                        }
                    }
                };
                for (; wk.next(b); ++g) {
                    if (b.first) {
                        if (!wait_bar(bar(B_QE), (ic & 1u) ^ 1u, abort, c)) break;
                        ptx::mbar_arrive_expect_tx(bar(B_QF), kTiles * L::kTileQ);
                        for (int t = 0; t < kTiles; ++t)
                            for (int x = 0; x < D / 64; ++x)
                                ptx::tma_load_3d(sQ + (uint32_t)(t * L::kTileQ + x * kBoxQ), &m.q, bar(B_QF), x * 64,
                                                 wk.it->head[t], wk.it->q_row[t]);
                        ++ic;
                    }
                    const int s = (int)(g % kStages);
                    const uint32_t ph = (g / kStages) & 1u;
                    const int row = wk.it->kv_row0 + b.kv0;
                    if (!wait_bar(bar(B_KE + s), ph ^ 1u, abort, c)) break;
                    load(sK + (uint32_t)(s * L::kTileK), &m.k, &m.k16, bar(B_KF + s), row);
                    ++nk;
                    if (!wait_bar(bar(B_VE + s), ph ^ 1u, abort, c)) break;
                    load(sV + (uint32_t)(s * L::kTileK), &m.v, &m.v16, bar(B_VF + s), row);
                    ++nv;
                }
                // every load issued must land before the CTA exits
                if (ic > 0) drain_bar(bar(B_QF), (ic - 1u) & 1u, c);
                for (uint32_t s = 0; s < kStages; ++s) {
                    if (nk > s) drain_bar(bar(B_KF + (int)s), ((nk - 1u - s) / kStages) & 1u, c);
                    if (nv > s) drain_bar(bar(B_VF + (int)s), ((nv - 1u - s) / kStages) & 1u, c);
                }
            }
        } else if (warp == 2) {
            // ================= V rows past a block's keys =================
            // (asked by the issuers, which follow every block: this warp sees only
            // some, and a phase of the stage's own barrier could pass it by)
            uint32_t nz = 0;
            for (uint32_t g = 0; wk.next(b); ++g) {
                if (b.kend - b.kv0 >= b.nk) continue;
                const int s = (int)(g % kStages);
                const bool w = wait_bar(bar(B_ZR), nz++ & 1u, abort, c);
                if (!__all_sync(0xffffffffu, w)) break;
                zero_rows<D>(sm + L::V + s * L::kTileK, L::kBoxK, b.kend - b.kv0, b.nk, lane);
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(B_VZ));
            }
        } else {
            // ================= MMA issuers: warp 1 for tile 0, warp 3 for tile 1 =================
            if (lane == 0) {
                const int t = warp == 1 ? 0 : 1;
                const uint32_t d_s = tmem + L::S(t), a_p = tmem + L::P(t), d_o = tmem + L::O(t);
                const uint32_t q_t = sQ + (uint32_t)(t * L::kTileQ);
                // S_t = Q_t . K_g^T once the softmax has loaded S(g-1)
                auto qk = [&](uint32_t g, const Blk &k) -> bool {
                    const int s = (int)(g % kStages);
                    if (!wait_bar(bar(B_KF + s), (g / kStages) & 1u, abort, c)) return false;
                    if (g > 0 && !wait_bar(bar(B_SL + t), (g - 1u) & 1u, abort, c)) return false;
                    ptx::tc_fence_after();
                    const uint32_t idesc = ptx::idesc_16bit_f32(BF16, 128, k.nk, false);
                    const uint32_t k_s = sK + (uint32_t)(s * L::kTileK);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        ptx::umma_bf16(d_s, kmajor_desc(q_t, kBoxQ, kk), kmajor_desc(k_s, L::kBoxK, kk), idesc, kk != 0 ? 1u : 0u);
                    ptx::umma_commit(bar(B_SF + t));
                    ptx::umma_commit(bar(B_KE + s));
                    if (k.last) ptx::umma_commit(bar(B_QE));
                    return true;
                };
                uint32_t nz = 0;  // zeroed blocks so far
                // O_t (+)= P_t . V_g; an item's first product overwrites O_t once the
                // previous item has been read out
                auto pv = [&](uint32_t g, const Blk &k, uint32_t item) -> bool {
                    const int s = (int)(g % kStages);
                    if (!wait_bar(bar(B_VF + s), (g / kStages) & 1u, abort, c)) return false;
                    if (k.kend - k.kv0 < k.nk) {
                        ptx::mbar_arrive(bar(B_ZR));
                        if (!wait_bar(bar(B_VZ), nz & 1u, abort, c)) return false;
                        ++nz;
                    }
                    if (!wait_bar(bar(B_PF + t), g & 1u, abort, c)) return false;
                    if (k.first && item > 0 && !wait_bar(bar(B_OE + t), (item - 1u) & 1u, abort, c)) return false;
                    ptx::tc_fence_after();
                    constexpr uint32_t idesc = ptx::idesc_16bit_f32(BF16, 128, D, true);
                    for (int kk = 0; kk < k.nk / 16; ++kk)
                        ptx::umma_bf16_ts(d_o, a_p + (uint32_t)(kk * 8),
                                          mnmajor_desc(sV + (uint32_t)(s * L::kTileK), L::kBoxK, kk), idesc,
                                          (kk != 0 || !k.first) ? 1u : 0u);
                    ptx::umma_commit(bar(B_PV + t));
                    ptx::umma_commit(bar(B_VE + s));
                    return true;
                };
                Blk cur = {}, nxt = {};
                bool ok = true, has = wk.next(cur);
                uint32_t g = 0, ic = 0, item = 0;
                if (has) {
                    ok = wait_bar(bar(B_QF), 0u, abort, c);
                    ic = 1;
                    if (ok) ok = qk(0, cur);
                }
                while (ok && has) {
                    const bool has_next = wk.next(nxt);
                    if (has_next && nxt.first) {
                        if (!wait_bar(bar(B_QF), ic & 1u, abort, c)) break;
                        ++ic;
                    }
                    if (has_next) ok = qk(g + 1u, nxt);
                    if (ok) ok = pv(g, cur, item);
                    if (!ok) break;
                    if (has_next && nxt.first) ++item;
                    cur = nxt;
                    has = has_next;
                    ++g;
                }
                // every MMA issued must complete before TMEM is released
                ptx::umma_commit(bar(B_DRAIN + t));
                drain_bar(bar(B_DRAIN + t), 0, c);
            }
        }
    } else {
        regs_inc();
        // ================= softmax of tile t, output rescaling, epilogue =================
        const int t = (warp - 4) >> 2;
        const int qd = warp & 3;
        const int row = qd * 32 + lane;
        const uint32_t tl = tmem + ((uint32_t)(qd * 32) << 16);
        const uint32_t ts = tl + L::S(t), tp = tl + L::P(t), to = tl + L::O(t);
        // tiles none of whose rows see a key
        for (int e = (int)blockIdx.x; e < p.n_empty; e += (int)gridDim.x) {
            const FwdItem &it = p.empty[e];
            if (row < it.n_rows[t]) {
                const int64_t r = it.q_row[t] + row;
                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.o.p) + r * p.o.token + it.head[t] * p.o.head);
                for (int k = 0; k < D / 8; ++k) dst[k] = make_uint4(0, 0, 0, 0);
                if (p.lse != nullptr) p.lse[r * c.H_q + it.head[t]] = -INFINITY;
            }
        }
        float mref = -INFINITY, lrow = 0.f;  // reference max (log2-scaled units), running sum
        const uint64_t scale2 = f2(c.scale_log2, c.scale_log2);
        Walk<kBK> wk;
        wk.init(p, items);
        Blk b = {};
        // one block: FULL, all kBK keys; else its first nk
        auto block = [&](uint32_t g, auto full) -> bool {
            constexpr bool FULL = decltype(full)::value;
            uint32_t v[kBK];
#pragma unroll
            for (int x = 0; x < kBK / 16; ++x) {
                if (FULL || x * 16 < b.nk) {
                    ptx::tmem_ld_32x32b_x16(ts + (uint32_t)(x * 16), v + 16 * x);
                } else {
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[x * 16 + k] = __float_as_uint(-INFINITY);
                }
            }
            ptx::tmem_ld_wait();
            // the scores are in registers: the next block's may overwrite them
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(B_SL + t));
            const int pos0 = wk.it->pos0[t], pos = pos0 + row;
            // some row of the tile does not see every key of the block?
            if (b.kv0 + kBK - 1 > pos0 || b.kend - b.kv0 < kBK ||
                (b.kv0 <= pos0 + kBQ - 1 - c.window && b.kv0 + kBK > c.sinks)) {
                const int hi = clampi(min(b.kend, pos + 1) - b.kv0, 0, kBK);
                const int lo = clampi(pos - c.window + 1 - b.kv0, 0, kBK);
                const int sk = clampi(c.sinks - b.kv0, 0, kBK);
#pragma unroll
                for (int k = 0; k < kBK; ++k)
                    if (k >= hi || (k < lo && k >= sk)) v[k] = __float_as_uint(-INFINITY);
            }
            // row max: eight interleaved partials, two new scores per three-input max
            float mp[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) mp[k] = __uint_as_float(v[k]);
#pragma unroll
            for (int k = 8; k < kBK; k += 2)
                mp[(k >> 1) & 7] = max3(mp[(k >> 1) & 7], __uint_as_float(v[k]), __uint_as_float(v[k + 1]));
            const float mx = fmaxf(max3(mp[0], mp[1], mp[2]), fmaxf(max3(mp[3], mp[4], mp[5]), fmaxf(mp[6], mp[7])));
            const float mcand = mx * c.scale_log2;
            const bool need = !b.first && mcand > mref + kRescale;
            const float alpha = need ? ex2(mref - mcand) : 1.f;
            if (b.first || need) mref = mcand;
            // P.V of the block before: its probabilities and the accumulator are ours
            if (g > 0) {
                const bool w = wait_bar(bar(B_PV + t), (g - 1u) & 1u, abort, c);
                if (!__all_sync(0xffffffffu, w)) return false;
                ptx::tc_fence_after();
            }
            if (__any_sync(0xffffffffu, need)) {
#pragma unroll
                for (int x = 0; x < D / 32; ++x) {
                    uint32_t o[32];
                    ptx::tmem_ld_32x32b_x32(to + (uint32_t)(x * 32), o);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                    ptx::tmem_st_32x32b_x32(to + (uint32_t)(x * 32), o);
                }
            }
            const float base = mref == -INFINITY ? 0.f : mref;
            const uint64_t nbase2 = f2(-base, -base);
            uint64_t sp[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) sp[k] = f2(0.f, 0.f);
#pragma unroll
            for (int x = 0; x < kBK / 16; ++x) {
                if (FULL || x * 16 < b.nk) {
                    uint32_t pk[8];
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                        float x0, x1;
                        unf2(fma2(f2(__uint_as_float(v[x * 16 + k]), __uint_as_float(v[x * 16 + k + 1])), scale2, nbase2), x0, x1);
                        const float p0 = ex2(x0), p1 = ex2(x1);
                        sp[(k >> 1) & 3] = add2(sp[(k >> 1) & 3], f2(p0, p1));
                        pk[k >> 1] = pack16<BF16>(p0, p1);
                    }
                    ptx::tmem_st_32x32b_x8(tp + (uint32_t)(x * 8), pk);
                }
            }
            float s0, s1, s2, s3;
            unf2(add2(sp[0], sp[1]), s0, s1);
            unf2(add2(sp[2], sp[3]), s2, s3);
            lrow = lrow * alpha + ((s0 + s1) + (s2 + s3));
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(B_PF + t));
            return true;
        };
        for (uint32_t g = 0; wk.next(b); ++g) {
            if (b.first) {
                mref = -INFINITY;
                lrow = 0.f;
            }
            bool w = wait_bar(bar(B_SF + t), g & 1u, abort, c);
            if (!__all_sync(0xffffffffu, w)) break;
            ptx::tc_fence_after();
            if (!(b.nk == kBK ? block(g, Bool<true>()) : block(g, Bool<false>()))) break;
            if (b.last) {  // the item's output, after the tile's last P.V
                w = wait_bar(bar(B_PV + t), g & 1u, abort, c);
                if (!__all_sync(0xffffffffu, w)) break;
                ptx::tc_fence_after();
                // a row without a visible key: no sum, output 0, lse -inf
                const bool none = lrow == 0.f;
                const float inv = none ? 0.f : 1.f / lrow;
                const int64_t r = wk.it->q_row[t] + row;
                const int h = wk.it->head[t];
                const bool mine = row < wk.it->n_rows[t];
                uint16_t *dst = mine ? static_cast<uint16_t *>(p.o.p) + r * p.o.token + h * p.o.head : nullptr;
                store_row<BF16, D>(dst, to, inv);
                if (mine && p.lse != nullptr)  // natural log: (m + log2 l) * ln 2
                    p.lse[r * c.H_q + h] = none ? -INFINITY : (mref + log2f(lrow)) * 0.69314718055994531f;
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(B_OE + t));
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

template <int D, bool BF16>
cudaError_t launch(int grid, const FwdParams &p, const FwdMaps &m, cudaStream_t st) {
    window_fwd_kernel<D, BF16><<<grid, kThreads, Lay<D>::BYTES, st>>>(p, m);
    return cudaGetLastError();
}
template <int D, bool BF16> cudaError_t prepare() {
    return cudaFuncSetAttribute(window_fwd_kernel<D, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::BYTES);
}

}  // namespace

int fwd_block(int d) { return d == 64 ? Lay<64>::kBK : Lay<128>::kBK; }
int fwd_smem(int d) { return d == 64 ? Lay<64>::BYTES : Lay<128>::BYTES; }

cudaError_t fwd_prepare(int d, bool bf16) {
    if (d == 64) return bf16 ? prepare<64, true>() : prepare<64, false>();
    return bf16 ? prepare<128, true>() : prepare<128, false>();
}

cudaError_t fwd_launch(int d, bool bf16, int grid, const FwdParams &p, const FwdMaps &m, cudaStream_t st) {
    if (d == 64) return bf16 ? launch<64, true>(grid, p, m, st) : launch<64, false>(grid, p, m, st);
    return bf16 ? launch<128, true>(grid, p, m, st) : launch<128, false>(grid, p, m, st);
}

}  // namespace window
}  // namespace syn
