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
//   warp 0        TMA producer: an item's Q tiles, each block's K and V (a ring)
//   warps 1, 2    issue S_t = Q_t.K^T of tile 0, 1
//   warps 3, 4    issue O_t += P_t.V of tile 0, 1
//   warp 5        zeroes V rows past the end of a block's keys: their probabilities
//                 are 0, and 0 times another sequence's inf or NaN is not
//   warps 8-11    softmax of tile 0 (one query row per thread, its TMEM lane)
//   warps 12-15   softmax of tile 1
//
// Each product has an issuing warp of its own because a warp's waits, commits
// and branches cost more than the tensor pipe needs for a block: one issuer a
// tile, or one for all, left the pipe idle for a third of the time.
//
// TMEM (512 columns) holds each tile's scores, probabilities (16-bit, half as
// many columns) and output side by side, so that the scores of block g+1 are
// computed while the softmax works on block g: it frees the score columns as
// soon as it has loaded them, and nothing waits for P.V but the next block's
// probabilities.  With D 128 that fits blocks of 80 keys (80 + 40 + 128 columns a
// tile); at D 64 more scores a thread would spill registers.  The reference
// maximum of the exponentials may lag the row's by up to 8 (log2 units), so the
// accumulator is rescaled only when a block raises it by more.
//
// Measured on one GB300 (bf16, 16384 tokens, 32 query and 8 kv heads of 128, 4
// sinks): window 4096 710 us alone, 1356 TFLOP/s over the visible pairs, 0.70 of
// the measured burst peak, and 735 to 754 in long runs, under the power cap; window
// 2048 444 us.  Tensor pipe 60 % active: a product of
// 80 columns costs it 52 cycles where 40 would be the peak's pace (128 columns:
// 64), but blocks of 128 keys would leave the probabilities no columns but the
// scores', and each step would wait for the last one's P.V.  A step takes the
// softmax warps about as long as the products: without either 640 to 730 us.
#include "window.cuh"

namespace syn {
namespace window {

namespace {

constexpr int kBQ = 128, kTiles = 2;
constexpr int kBoxQ = kBQ * 128;  // 128 rows x 128 bytes
constexpr int kThreads = 512;
constexpr int kSmemItems = 48;   // items of the CTA's list kept in shared memory
constexpr float kRescale = 8.f;

constexpr int kMaxStages = 4;
enum {
    B_QF = 0,                     // the item's Q tiles landed
    B_QE = 1,                     // Q tiles read by the item's last Q.K^T (one commit per tile)
    B_KF = 2,                     // stage landed: a block's K and V
    B_KE = B_KF + kMaxStages,     // stage consumed (one commit per tile, after its P.V)
    B_SF = B_KE + kMaxStages,     // tile t's scores written (2)
    B_SL = B_SF + 2,              // tile t's scores loaded into registers (2)
    B_PF = B_SL + 2,              // tile t's probabilities written (2)
    B_PV = B_PF + 2,              // tile t's P.V done (2)
    B_OE = B_PV + 2,              // tile t's accumulator read out (2)
    B_DRAIN = B_OE + 2,           // every MMA of an issuer completed (4)
    B_ZR = B_DRAIN + 4,           // a block with V rows past its keys landed (asked by both P.V issuers)
    B_VZ = B_ZR + 1,              // its rows past the keys zeroed
    N_BAR = B_VZ + 1
};

template <int D> struct Lay {
    static constexpr int kBK = 80;  // keys of a block
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

// A key block: first key, end of its valid keys, keys computed (a multiple of 16)
struct Blk {
    int kv0, kend, nk;
};

// Block b of an item, from block b - 1 (b > 0)
template <int kBK> __device__ __forceinline__ void step(Blk &k, int b, int n_sink, const FwdItem &it) {
    if (b == n_sink) {
        k.kv0 = it.w_lo;
        k.kend = it.k_end;
    } else if (b == 0) {
        k.kv0 = 0;
        k.kend = it.s_end;
    } else {
        k.kv0 += kBK;
    }
    k.nk = min(kBK, (k.kend - k.kv0 + 15) & ~15);
}

// Every role walks the CTA's items and their blocks: g counts the blocks, `item`
// the items, and stage and phase follow g.
struct Ring {
    int s = 0;
    uint32_t phase = 0;
    template <int kStages> __device__ __forceinline__ void next() {
        if (++s == kStages) {
            s = 0;
            phase ^= 1u;
        }
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

// Register split: the launch gives 128 a thread (512 threads); the first eight
// warps keep 64, the softmax warps take 192: 256 * 64 + 256 * 192 = 65,536.
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 64;"); }
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 192;"); }

template <int V> struct Int {
    static constexpr int value = V;
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
            const bool pair = i == B_QE || i == B_ZR || (i >= B_KE && i < B_KE + kMaxStages);
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
    ptx::grid_wait();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t sQ = sbase + L::Q, sK = sbase + L::K, sV = sbase + L::V;

    const int first_item = p.begin[blockIdx.x], n_items = p.begin[blockIdx.x + 1] - first_item;
    auto item_at = [&](int i) -> const FwdItem & { return i < kSmemItems ? items[i] : p.items[first_item + i]; };
    const uint32_t one = lane == 0 ? 1u : 0u;

    if (warp < 8) {
        regs_dec();
        Ring r;
        Blk b = {};
        uint32_t g = 0;
        if (warp == 0) {
            // ================= TMA producer =================
            bool stop = false;
            int n_q = 0;  // items whose Q has been issued
            for (int i = 0; i < n_items && !stop; ++i) {
                const FwdItem &it = item_at(i);
                const int n_blk = it.n_blk, n_sink = (it.s_end + kBK - 1) / kBK, hk = it.hk, row0 = it.kv_row0;
                wait_bar(bar(B_QE), ((uint32_t)i & 1u) ^ 1u, abort, c);
                if (aborted(abort)) break;
                ++n_q;
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(bar(B_QF), kTiles * L::kTileQ);
                    for (int t = 0; t < kTiles; ++t)
                        for (int x = 0; x < D / 64; ++x)
                            ptx::tma_load_3d(sQ + (uint32_t)(t * L::kTileQ + x * kBoxQ), &m.q, bar(B_QF), x * 64, it.head[t],
                                             it.q_row[t]);
                }
                __syncwarp();
                for (int k = 0; k < n_blk; ++k, ++g, r.next<kStages>()) {
                    step<kBK>(b, k, n_sink, it);
                    wait_bar(bar(B_KE + r.s), r.phase ^ 1u, abort, c);
                    stop = aborted(abort);
                    if (stop) break;
                    if (lane == 0) {
                        const uint32_t br = bar(B_KF + r.s), dk = sK + (uint32_t)(r.s * L::kTileK), dv = sV + (uint32_t)(r.s * L::kTileK);
                        ptx::mbar_arrive_expect_tx(br, (uint32_t)(2 * b.nk * D * 2));
                        for (int x = 0; x < D / 64; ++x) {
                            const uint32_t o = (uint32_t)(x * L::kBoxK);
                            if (b.nk == kBK) {
                                ptx::tma_load_3d(dk + o, &m.k, br, x * 64, hk, row0 + b.kv0);
                                ptx::tma_load_3d(dv + o, &m.v, br, x * 64, hk, row0 + b.kv0);
                            } else {
                                for (int y = 0; y < b.nk; y += 16) {
                                    ptx::tma_load_3d(dk + o + (uint32_t)(y * 128), &m.k16, br, x * 64, hk, row0 + b.kv0 + y);
                                    ptx::tma_load_3d(dv + o + (uint32_t)(y * 128), &m.v16, br, x * 64, hk, row0 + b.kv0 + y);
                                }
                            }
                        }
                    }
                    __syncwarp();
                }
            }
            // every load issued must land before the CTA exits
            if (n_q > 0) drain_bar(bar(B_QF), (uint32_t)(n_q - 1) & 1u, c);
            for (uint32_t s = 0; s < kStages; ++s)
                if (g > s) drain_bar(bar(B_KF + (int)s), ((g - 1u - s) / kStages) & 1u, c);
        } else if (warp <= 2) {
            // ================= S_t = Q_t . K^T =================
            const int t = warp - 1;
            const uint32_t d_s = tmem + L::S(t), q_d = desc_lo(sQ + (uint32_t)(t * L::kTileQ), 16), k_d0 = desc_lo(sK, 16);
            for (int i = 0; i < n_items; ++i) {
                const FwdItem &it = item_at(i);
                const int n_blk = it.n_blk, n_sink = (it.s_end + kBK - 1) / kBK;
                wait_bar(bar(B_QF), (uint32_t)i & 1u, abort, c);
                for (int k = 0; k < n_blk; ++k, ++g, r.next<kStages>()) {
                    step<kBK>(b, k, n_sink, it);
                    const uint32_t idesc = ptx::idesc_16bit_f32(BF16, 128, b.nk, false);
                    const uint32_t k_d = k_d0 + (uint32_t)(r.s * L::kTileK >> 4);
                    wait_bar(bar(B_KF + r.s), r.phase, abort, c);
                    if (g > 0) wait_bar(bar(B_SL + t), (g - 1u) & 1u, abort, c);  // the softmax has loaded S of block g - 1
                    ptx::tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        umma_if(one, d_s, desc_at(q_d, (kk >> 2) * kBoxQ + (kk & 3) * 32),
                                desc_at(k_d, (kk >> 2) * L::kBoxK + (kk & 3) * 32), idesc, kk != 0 ? 1u : 0u);
                    commit_if(one, bar(B_SF + t));
                    if (k == n_blk - 1) commit_if(one, bar(B_QE));
                }
            }
            // every MMA issued must complete before TMEM is released
            commit_if(one, bar(B_DRAIN + t));
            drain_bar(bar(B_DRAIN + t), 0, c);
        } else if (warp <= 4) {
            // ================= O_t (+)= P_t . V =================
            const int t = warp - 3;
            const uint32_t a_p = tmem + L::P(t), d_o = tmem + L::O(t), v_d0 = desc_lo(sV, L::kBoxK);
            constexpr uint32_t idesc = ptx::idesc_16bit_f32(BF16, 128, D, true);
            uint32_t nz = 0;  // zeroed blocks so far
            for (int i = 0; i < n_items; ++i) {
                const FwdItem &it = item_at(i);
                const int n_blk = it.n_blk, n_sink = (it.s_end + kBK - 1) / kBK;
                // the first product overwrites O_t once the previous item has been read out
                if (i > 0) wait_bar(bar(B_OE + t), (uint32_t)(i - 1) & 1u, abort, c);
                for (int k = 0; k < n_blk; ++k, ++g, r.next<kStages>()) {
                    step<kBK>(b, k, n_sink, it);
                    const uint32_t v_d = v_d0 + (uint32_t)(r.s * L::kTileK >> 4);
                    wait_bar(bar(B_KF + r.s), r.phase, abort, c);
                    if (b.kend - b.kv0 < b.nk) {
                        arrive_if(one, bar(B_ZR));
                        wait_bar(bar(B_VZ), nz & 1u, abort, c);
                        ++nz;
                    }
                    wait_bar(bar(B_PF + t), g & 1u, abort, c);
                    ptx::tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk)
                        umma_ts_if(kk * 16 < b.nk ? one : 0u, d_o, a_p + (uint32_t)(kk * 8), desc_at(v_d, kk * 2048), idesc,
                                   (kk != 0 || k != 0) ? 1u : 0u);
                    commit_if(one, bar(B_PV + t));
                    commit_if(one, bar(B_KE + r.s));
                }
            }
            commit_if(one, bar(B_DRAIN + 2 + t));
            drain_bar(bar(B_DRAIN + 2 + t), 0, c);
        } else if (warp == 5) {
            // ================= V rows past a block's keys =================
            // (asked by the issuers, which follow every block: this warp sees only
            // some, and a phase of the stage's own barrier could pass it by)
            uint32_t nz = 0;
            for (int i = 0; i < n_items; ++i) {
                const FwdItem &it = item_at(i);
                const int n_blk = it.n_blk, n_sink = (it.s_end + kBK - 1) / kBK;
                for (int k = 0; k < n_blk; ++k, r.next<kStages>()) {
                    step<kBK>(b, k, n_sink, it);
                    if (b.kend - b.kv0 >= b.nk) continue;
                    wait_bar(bar(B_ZR), nz++ & 1u, abort, c);
                    zero_rows<D>(sm + L::V + r.s * L::kTileK, L::kBoxK, b.kend - b.kv0, b.nk, lane);
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    arrive_if(one, bar(B_VZ));
                }
            }
        }
    } else {
        regs_inc();
        // ================= softmax of tile t, output rescaling, epilogue =================
        const int t = (warp - 8) >> 2;
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
        __syncwarp();
        float mref = -INFINITY, lrow = 0.f;  // reference max (log2-scaled units), running sum
        const uint64_t scale2 = f2(c.scale_log2, c.scale_log2);
        const int window = c.window, sinks = c.sinks;
        int pos0 = 0;                        // position of the tile's first row
        uint32_t g = 0;
        Blk b = {};
        // one block of N score columns (kBK, or 16 where that covers its keys): with
        // MASK, those that the row sees (columns past nk are stale, and masked).  A
        // body of its own without the masks, whose selects take as long as the rest.
        auto block = [&](bool first, auto cols, auto masked) {
            constexpr int N = decltype(cols)::value;
            constexpr bool MASK = decltype(masked)::value;
            uint32_t v[N];
#pragma unroll
            for (int x = 0; x < N / 16; ++x) ptx::tmem_ld_32x32b_x16(ts + (uint32_t)(x * 16), v + 16 * x);
            ptx::tmem_ld_wait();
            // the scores are in registers: the next block's may overwrite them
            ptx::tc_fence_before();
            __syncwarp();
            arrive_if(one, bar(B_SL + t));
            if constexpr (MASK) {
                const int pos = pos0 + row;
                const int hi = clampi(min(b.kend, pos + 1) - b.kv0, 0, kBK);
                const int lo = clampi(pos - window + 1 - b.kv0, 0, kBK);
                const int sk = clampi(sinks - b.kv0, 0, kBK);
                uint32_t seen[(N + 31) / 32];
#pragma unroll
                for (int x = 0; x < (N + 31) / 32; ++x)
                    seen[x] = bits_below(hi, 32 * x) & (~bits_below(lo, 32 * x) | bits_below(sk, 32 * x));
                MaskRow<0, N>::apply(v, seen, __float_as_uint(-INFINITY));
            }
            // row max: eight interleaved partials, two new scores per three-input max
            float mp[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) mp[k] = __uint_as_float(v[k]);
#pragma unroll
            for (int k = 8; k < N; k += 2)
                mp[(k >> 1) & 7] = max3(mp[(k >> 1) & 7], __uint_as_float(v[k]), __uint_as_float(v[k + 1]));
            const float mx = fmaxf(max3(mp[0], mp[1], mp[2]), fmaxf(max3(mp[3], mp[4], mp[5]), fmaxf(mp[6], mp[7])));
            const float mcand = mx * c.scale_log2;
            const bool need = !first && mcand > mref + kRescale;
            const float alpha = need ? ex2(mref - mcand) : 1.f;
            if (first || need) mref = mcand;
            const float base = mref == -INFINITY ? 0.f : mref;
            const uint64_t nbase2 = f2(-base, -base);
            uint64_t sp[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) sp[k] = f2(0.f, 0.f);
            uint32_t pk[N / 2];
#pragma unroll
            for (int k = 0; k < N; k += 2) {
                float x0, x1;
                unf2(fma2(f2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), scale2, nbase2), x0, x1);
                const float p0 = ex2(x0), p1 = ex2(x1);
                sp[(k >> 1) & 3] = add2(sp[(k >> 1) & 3], f2(p0, p1));
                pk[k >> 1] = pack16<BF16>(p0, p1);
            }
            // P.V of the block before, by now long under way: then its
            // probabilities may be replaced and the accumulator rescaled
            if (g > 0) {
                wait_bar(bar(B_PV + t), (g - 1u) & 1u, abort, c);
                ptx::tc_fence_after();
            }
            if (__any_sync(0xffffffffu, need)) {
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    uint32_t o[16];
                    ptx::tmem_ld_32x32b_x16(to + (uint32_t)(x * 16), o);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                    ptx::tmem_st_32x32b_x8(to + (uint32_t)(x * 16), o);
                    ptx::tmem_st_32x32b_x8(to + (uint32_t)(x * 16 + 8), o + 8);
                }
            }
#pragma unroll
            for (int x = 0; x < N / 16; ++x) ptx::tmem_st_32x32b_x8(tp + (uint32_t)(x * 8), pk + x * 8);
            float s0, s1, s2, s3;
            unf2(add2(sp[0], sp[1]), s0, s1);
            unf2(add2(sp[2], sp[3]), s2, s3);
            lrow = lrow * alpha + ((s0 + s1) + (s2 + s3));
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            arrive_if(one, bar(B_PF + t));
        };
        for (int i = 0; i < n_items; ++i) {
            const FwdItem &it = item_at(i);
            const int n_blk = it.n_blk, n_sink = (it.s_end + kBK - 1) / kBK;
            mref = -INFINITY;
            lrow = 0.f;
            pos0 = it.pos0[t];
            for (int k = 0; k < n_blk; ++k, ++g) {
                step<kBK>(b, k, n_sink, it);
                // every row of the tile sees every key of the block?
                const bool full = b.kv0 + kBK - 1 <= pos0 && b.kend - b.kv0 >= kBK &&
                                  (b.kv0 > pos0 + kBQ - 1 - window || b.kv0 + kBK <= sinks);
                wait_bar(bar(B_SF + t), g & 1u, abort, c);
                ptx::tc_fence_after();
                if (full) block(k == 0, Int<kBK>(), Int<0>());
                else if (b.nk > 16) block(k == 0, Int<kBK>(), Int<1>());
                else block(k == 0, Int<16>(), Int<1>());
            }
            // the item's output, after the tile's last P.V
            wait_bar(bar(B_PV + t), (g - 1u) & 1u, abort, c);
            ptx::tc_fence_after();
            // a row without a visible key: no sum, output 0, lse -inf
            const bool none = lrow == 0.f;
            const float inv = none ? 0.f : 1.f / lrow;
            const int64_t r = it.q_row[t] + row;
            const int h = it.head[t];
            const bool mine = row < it.n_rows[t];
            uint16_t *dst = mine ? static_cast<uint16_t *>(p.o.p) + r * p.o.token + h * p.o.head : nullptr;
            store_row<BF16, D>(dst, to, inv);
            if (mine && p.lse != nullptr)  // natural log: (m + log2 l) * ln 2
                p.lse[r * c.H_q + h] = none ? -INFINITY : (mref + log2f(lrow)) * 0.69314718055994531f;
            ptx::tc_fence_before();
            __syncwarp();
            arrive_if(one, bar(B_OE + t));
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
    return launch_early(window_fwd_kernel<D, BF16>, grid, kThreads, Lay<D>::BYTES, st, p, m);
}
template <int D, bool BF16> cudaError_t prepare() {
    return cudaFuncSetAttribute(window_fwd_kernel<D, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::BYTES);
}

}  // namespace

int fwd_block(int d) { return d == 64 ? Lay<64>::kBK : Lay<128>::kBK; }
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
