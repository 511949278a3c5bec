// window_fwd.cu -- forward of the windowed attention (include/syn_window.h).
//
// A persistent CTA (one per SM) takes its list of work items in turn: two
// 128-row query tiles (t = 0, 1) that read the same key blocks.  With an even
// group of query heads the two tiles are the same rows of two heads of the
// group, so both have the same mask and no block is wasted on one of them;
// else they are consecutive rows of one head.  A block is 128 keys, or a
// multiple of 32 for the sinks and the end of a range, so that four sink keys
// cost a quarter of a block.  The online softmax keeps a running maximum and
// sum per row, one pass over the keys:
//
//   warp 0      TMA producer: an item's Q tiles, each block's K and V (two slots)
//   warps 1, 3  MMA issuers, one per tile: S_t = Q_t.K^T, then O_t += P_t.V
//   warp 2      zeroes V rows past the end of a block's keys: their probabilities
//               are 0, and 0 times another sequence's inf or NaN is not
//   warps 4-7   softmax of tile 0 (one query row per thread, its TMEM lane)
//   warps 8-11  softmax of tile 1
//
// TMEM (512 columns): S_t at 128t, O_t at 256 + 128t; the probabilities take
// the upper 64 columns of S_t, from where P.V reads them.  The scores of
// block g+1 are computed in two halves of 64 keys: the lower one as soon as
// the softmax has loaded block g's scores, the upper one once P.V of block g
// has read the probabilities.  The reference maximum of the exponentials may
// lag the row's by up to 8 (log2 units), so the accumulator is rescaled only
// when a block raises it by more.
#include "window.cuh"

namespace syn {
namespace window {

namespace {

constexpr int kBQ = 128, kBK = 128, kTiles = 2;
constexpr int kBox = 128 * 128;  // 128 rows x 128 bytes
constexpr int kThreads = 384;
constexpr int kSmemItems = 48;   // items of the CTA's list kept in shared memory
constexpr float kRescale = 8.f;

enum {
    B_QF = 0,      // the item's Q tiles landed
    B_QE = 1,      // Q tiles read by the item's last Q.K^T (one commit per issuer)
    B_KF = 2,      // K slot s landed (2)
    B_KE = 4,      // K slot s consumed (2; one commit per issuer)
    B_VF = 6,      // V slot s landed (2)
    B_VE = 8,      // V slot s consumed (2; one commit per issuer)
    B_SF = 10,     // tile t's scores written (2)
    B_PF = 12,     // tile t's probabilities written (2)
    B_PV = 14,     // tile t's P.V done (2)
    B_OE = 16,     // tile t's accumulator read out (2)
    B_DRAIN = 18,  // every MMA of tile t's issuer completed (2)
    B_XD = 20,     // tile t's exponentials of a block done (2): the tiles take turns
    B_SL = 22,     // tile t's scores loaded into registers (2)
    B_ZR = 24,     // a V block with rows past its keys landed (asked by both issuers)
    B_VZ = 25,     // its rows past the keys zeroed
    N_BAR = 26
};

template <int D> struct Lay {
    static constexpr int kTile = 128 * D * 2;
    static constexpr int Q = 0;
    static constexpr int K = Q + kTiles * kTile;
    static constexpr int V = K + 2 * kTile;
    static constexpr int ITEMS = V + 2 * kTile;
    static constexpr int BAR = ITEMS + kSmemItems * (int)sizeof(FwdItem);
    static constexpr int MISC = BAR + 8 * N_BAR;
    static constexpr int USED = MISC + 16;
    static constexpr int BYTES = USED + 1024;  // + the 1024-byte alignment of the tiles
};

// One key block of an item
struct Blk {
    int kv0, kend, nk;  // first key, end of its valid keys, keys computed (a multiple of 32)
    bool first, last;
};

// The CTA's walk over its items' blocks; every role makes the same one.
struct Walk {
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
        k.nk = min(kBK, (k.kend - k.kv0 + 31) & ~31);
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

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) window_fwd_kernel(const __grid_constant__ FwdParams p,
                                                                 const __grid_constant__ FwdMaps m) {
    using L = Lay<D>;
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
        ptx::mbar_init(bar(B_QF), 1);
        ptx::mbar_init(bar(B_QE), kTiles);
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(bar(B_KF + s), 1);
            ptx::mbar_init(bar(B_KE + s), kTiles);
            ptx::mbar_init(bar(B_VF + s), 1);
            ptx::mbar_init(bar(B_VE + s), kTiles);
            ptx::mbar_init(bar(B_SF + s), 1);
            ptx::mbar_init(bar(B_PF + s), 4);
            ptx::mbar_init(bar(B_PV + s), 1);
            ptx::mbar_init(bar(B_OE + s), 4);
            ptx::mbar_init(bar(B_DRAIN + s), 1);
            ptx::mbar_init(bar(B_XD + s), 4);
            ptx::mbar_init(bar(B_SL + s), 4);
        }
        ptx::mbar_init(bar(B_ZR), kTiles);
        ptx::mbar_init(bar(B_VZ), 1);
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
        Walk wk;
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
                            ptx::tma_load_3d(dst + (uint32_t)(x * kBox), full, br, x * 64, wk.it->hk, row);
                        } else {
                            for (int r = 0; r < b.nk; r += 32)
                                ptx::tma_load_3d(dst + (uint32_t)(x * kBox + r * 128), narrow, br, x * 64, wk.it->hk, row + r);
                        }
                    }
                };
                for (; wk.next(b); ++g) {
                    if (b.first) {
                        if (!wait_bar(bar(B_QE), (ic & 1u) ^ 1u, abort, c)) break;
                        ptx::mbar_arrive_expect_tx(bar(B_QF), kTiles * L::kTile);
                        for (int t = 0; t < kTiles; ++t)
                            for (int x = 0; x < D / 64; ++x)
                                ptx::tma_load_3d(sQ + (uint32_t)(t * L::kTile + x * kBox), &m.q, bar(B_QF), x * 64,
                                                 wk.it->head[t], wk.it->q_row[t]);
                        ++ic;
                    }
                    const int s = (int)(g & 1u);
                    const uint32_t ph = (g >> 1) & 1u;
                    const int row = wk.it->kv_row0 + b.kv0;
                    if (!wait_bar(bar(B_KE + s), ph ^ 1u, abort, c)) break;
                    load(sK + (uint32_t)(s * L::kTile), &m.k, &m.k32, bar(B_KF + s), row);
                    ++nk;
                    if (!wait_bar(bar(B_VE + s), ph ^ 1u, abort, c)) break;
                    load(sV + (uint32_t)(s * L::kTile), &m.v, &m.v32, bar(B_VF + s), row);
                    ++nv;
                }
                // every load issued must land before the CTA exits
                if (ic > 0) drain_bar(bar(B_QF), (ic - 1u) & 1u, c);
                for (uint32_t s = 0; s < 2; ++s) {
                    if (nk > s) drain_bar(bar(B_KF + (int)s), ((s + ((nk - 1u - s) / 2u) * 2u) >> 1) & 1u, c);
                    if (nv > s) drain_bar(bar(B_VF + (int)s), ((s + ((nv - 1u - s) / 2u) * 2u) >> 1) & 1u, c);
                }
            }
        } else if (warp == 2) {
            // ================= V rows past a block's keys =================
            // (asked by the issuers, which follow every block: this warp sees only
            // some, and a phase of the slot's own barrier could pass it by)
            uint32_t nz = 0;
            for (uint32_t g = 0; wk.next(b); ++g) {
                if (b.kend - b.kv0 >= b.nk) continue;
                const int s = (int)(g & 1u);
                const bool w = wait_bar(bar(B_ZR), nz++ & 1u, abort, c);
                if (!__all_sync(0xffffffffu, w)) break;
                zero_rows<D>(sm + L::V + s * L::kTile, kBox, b.kend - b.kv0, b.nk, lane);
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(B_VZ));
            }
        } else {
            // ================= MMA issuers: warp 1 for tile 0, warp 3 for tile 1 =================
            if (lane == 0) {
                const int t = warp == 1 ? 0 : 1;
                const uint32_t d_s = tmem + (uint32_t)(t * 128);         // S_t, then P_t
                const uint32_t d_o = tmem + 256u + (uint32_t)(t * 128);  // O_t
                const uint32_t q_t = sQ + (uint32_t)(t * L::kTile);
                // S_t = Q_t . K_g^T in two halves of up to 64 keys: the lower once the
                // softmax has loaded S(g-1), the upper once P.V(g-1) has read P(g-1)
                auto qk_half = [&](uint32_t g, const Blk &k, int half) -> bool {
                    const int s = (int)(g & 1u);
                    const int n = min(k.nk - 64 * half, 64);
                    if (half == 0) {
                        if (!wait_bar(bar(B_KF + s), (g >> 1) & 1u, abort, c)) return false;
                        if (g > 0 && !wait_bar(bar(B_SL + t), (g - 1u) & 1u, abort, c)) return false;
                    } else if (g > 0 && !wait_bar(bar(B_PV + t), (g - 1u) & 1u, abort, c)) {
                        return false;
                    }
                    ptx::tc_fence_after();
                    if (n > 0) {
                        const uint32_t idesc = ptx::idesc_16bit_f32(BF16, 128, n, false);
                        const uint32_t k_h = sK + (uint32_t)(s * L::kTile + half * 8192);  // key rows 64 * half ..
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            ptx::umma_bf16(d_s + (uint32_t)(half * 64), kmajor_desc(q_t, kBox, kk), kmajor_desc(k_h, kBox, kk),
                                           idesc, kk != 0 ? 1u : 0u);
                    }
                    if (half == 1) {
                        ptx::umma_commit(bar(B_SF + t));
                        ptx::umma_commit(bar(B_KE + s));
                    }
                    return true;
                };
                uint32_t nz = 0;  // zeroed blocks so far
                // O_t (+)= P_t . V_g; an item's first product overwrites O_t once the
                // previous item has been read out
                auto pv = [&](uint32_t g, const Blk &k, uint32_t item) -> bool {
                    const int s = (int)(g & 1u);
                    if (!wait_bar(bar(B_VF + s), (g >> 1) & 1u, abort, c)) return false;
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
                        ptx::umma_bf16_ts(d_o, d_s + 64u + (uint32_t)(kk * 8),
                                          mnmajor_desc(sV + (uint32_t)(s * L::kTile), kBox, kk), idesc,
                                          (kk != 0 || !k.first) ? 1u : 0u);
                    ptx::umma_commit(bar(B_PV + t));
                    ptx::umma_commit(bar(B_VE + s));
                    return true;
                };
                Blk cur, nxt;
                bool ok = true, has = wk.next(cur);
                uint32_t g = 0, ic = 0, item_cur = 0;
                if (has) {
                    ok = wait_bar(bar(B_QF), 0u, abort, c);
                    ic = 1;
                    if (ok) ok = qk_half(0, cur, 0);
                    if (ok) ok = qk_half(0, cur, 1);
                    if (ok && cur.last) ptx::umma_commit(bar(B_QE));
                }
                while (ok && has) {
                    const bool has_next = wk.next(nxt);
                    if (has_next && nxt.first) {
                        if (!wait_bar(bar(B_QF), ic & 1u, abort, c)) break;
                        ++ic;
                    }
                    if (has_next) ok = qk_half(g + 1u, nxt, 0);
                    if (ok) ok = pv(g, cur, item_cur);
                    if (ok && has_next) ok = qk_half(g + 1u, nxt, 1);
                    if (!ok) break;
                    if (has_next && nxt.last) ptx::umma_commit(bar(B_QE));
                    if (has_next && nxt.first) ++item_cur;
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
        const uint32_t ts = tl + (uint32_t)(t * 128);
        const uint32_t to = tl + 256u + (uint32_t)(t * 128);
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
        Walk wk;
        wk.init(p, items);
        Blk b;
        for (uint32_t g = 0; wk.next(b); ++g) {
            if (b.first) {
                mref = -INFINITY;
                lrow = 0.f;
            }
            bool w = wait_bar(bar(B_SF + t), g & 1u, abort, c);
            if (!__all_sync(0xffffffffu, w)) break;
            ptx::tc_fence_after();
            const int pos0 = wk.it->pos0[t], pos = pos0 + row;
            // every row of the tile sees every key of the block?
            const bool masked = b.kv0 + kBK - 1 > pos0 || b.kend - b.kv0 < kBK ||
                                (b.kv0 <= pos0 + kBQ - 1 - c.window && b.kv0 + kBK > c.sinks);
            uint32_t v[kBK];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                if (x * 32 < b.nk) {
                    ptx::tmem_ld_32x32b_x32(ts + (uint32_t)(x * 32), *reinterpret_cast<uint32_t(*)[32]>(v + 32 * x));
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[x * 32 + k] = __float_as_uint(-INFINITY);
                }
            }
            ptx::tmem_ld_wait();
            // the scores are in registers: the next block's lower half may overwrite them
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(B_SL + t));
            if (masked) {
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
            const float mx = fmaxf(fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3])),
                                   fmaxf(fmaxf(mp[4], mp[5]), fmaxf(mp[6], mp[7])));
            const float mcand = mx * c.scale_log2;
            const bool need = !b.first && mcand > mref + kRescale;
            const float alpha = need ? ex2(mref - mcand) : 1.f;
            if (b.first || need) mref = mcand;
            if (__any_sync(0xffffffffu, need)) {
                // P.V(g-1) completed before this block's Q.K^T could overwrite the
                // scores, so the accumulator is stable: rescale it
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
            // the tiles take turns at the exponentials, so each runs them alone while
            // the other tile's products run on the tensor pipe
            if (t == 1 || g > 0) {
                w = wait_bar(bar(B_XD + (1 - t)), (t == 1 ? g : g - 1u) & 1u, abort, c);
                if (!__all_sync(0xffffffffu, w)) break;
            }
            const float base = mref == -INFINITY ? 0.f : mref;
            const uint64_t scale2 = f2(c.scale_log2, c.scale_log2), nbase2 = f2(-base, -base);
            uint64_t sp[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) sp[k] = f2(0.f, 0.f);
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                if (hh * 64 < b.nk) {
                    uint32_t pk[32];
#pragma unroll
                    for (int k = 0; k < 64; k += 2) {
                        float x0, x1;
                        unf2(fma2(f2(__uint_as_float(v[hh * 64 + k]), __uint_as_float(v[hh * 64 + k + 1])), scale2, nbase2),
                             x0, x1);
                        const float p0 = ex2(x0), p1 = ex2(x1);
                        sp[(k >> 1) & 3] = add2(sp[(k >> 1) & 3], f2(p0, p1));
                        pk[k >> 1] = pack16<BF16>(p0, p1);
                    }
                    ptx::tmem_st_32x32b_x32(ts + 64u + (uint32_t)(hh * 32), pk);
                }
            }
            float s0, s1, s2, s3, s4, s5, s6, s7;
            unf2(sp[0], s0, s1);
            unf2(sp[1], s2, s3);
            unf2(sp[2], s4, s5);
            unf2(sp[3], s6, s7);
            const float sum = ((s0 + s1) + (s2 + s3)) + ((s4 + s5) + (s6 + s7));
            lrow = lrow * alpha + sum;
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(bar(B_PF + t));
                ptx::mbar_arrive(bar(B_XD + t));
            }
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
