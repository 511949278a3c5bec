// window.cu -- plans and C ABI of the windowed attention over ragged sequences
// (include/syn_window.h; kernels in window_fwd.cu, window_dkv.cu and window_dq.cu).
//
// A plan turns the sequences' lengths into work items and deals them out to
// one persistent CTA per SM: the largest first, each to the CTA with the least
// work so far, so that the CTAs end together although the first query tiles of
// a sequence and the last key tiles see less.  In the gradient a key tile whose
// queries are many (the sinks: every later query) or whose items would be too
// few to fill the SMs is cut into parts with sums of their own, added in a
// fixed order at the end.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <memory>
#include <new>
#include <queue>
#include <string>
#include <vector>

#include "host_util.h"
#include "syn_window.h"
#include "window.cuh"

using namespace syn;
using namespace syn::window;

struct syn_window_plan_s {
    syn_window_cfg_t cfg;
    syn_window_info_t info;
    int device = 0, num_sms = 0;
    bool bf16 = true;
    int grid_f = 0, grid_k = 0, grid_q = 0;  // CTAs of the forward, dK/dV and dQ kernels
    int n_empty = 0, n_prep = 0, n_sums = 0;
    int64_t pad_rows = 0;
    FwdItem *d_items = nullptr, *d_empty = nullptr;
    BwdItem *d_key_items = nullptr, *d_query_items = nullptr;
    int32_t *d_begin = nullptr, *d_key_begin = nullptr, *d_query_begin = nullptr;
    PrepTile *d_prep = nullptr;
    SumItem *d_sums = nullptr;
    float *d_stats = nullptr;  // [2][H_q][pad_rows]
    float *d_part = nullptr;
    int32_t *d_err = nullptr;
};

namespace {

#define WIN_CK(call)                                                                                  \
    do {                                                                                              \
        cudaError_t e__ = (call);                                                                     \
        if (e__ != cudaSuccess) return host_fail(SYN_ERR_CUDA, std::string(#call) + ": " + cudaGetErrorString(e__)); \
    } while (0)

constexpr int64_t kMaxLen = (int64_t)1 << 29;  // positions and window sums stay within 32 bits
constexpr int64_t kMaxItems = (int64_t)1 << 28;  // of a work list (16 GB): its indexes stay within 32 bits

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

void free_plan(syn_window_plan_s *pl) {
    for (void *x : {(void *)pl->d_items, (void *)pl->d_empty, (void *)pl->d_key_items, (void *)pl->d_query_items,
                    (void *)pl->d_begin, (void *)pl->d_key_begin, (void *)pl->d_query_begin, (void *)pl->d_prep,
                    (void *)pl->d_sums, (void *)pl->d_stats, (void *)pl->d_part, (void *)pl->d_err})
        cudaFree(x);
    delete pl;
}

template <typename T> cudaError_t upload(T **dst, const std::vector<T> &v) {
    cudaError_t e = cudaMalloc(reinterpret_cast<void **>(dst), std::max<size_t>(v.size(), 1) * sizeof(T));
    if (e == cudaSuccess && !v.empty()) e = cudaMemcpy(*dst, v.data(), v.size() * sizeof(T), cudaMemcpyHostToDevice);
    return e;
}

// Deal items out to at most `ctas` CTAs: the costliest first (equal costs in
// the list's order, so that neighbours run at the same time and share their
// keys in L2), each to the CTA with the least cost so far.  Reorders `items`
// by CTA; `begin` has one entry a CTA and the end.
template <typename T>
void deal(std::vector<T> &items, const std::vector<int> &cost, int ctas, std::vector<int32_t> &begin) {
    const int n = (int)items.size(), grid = std::min(ctas, n);
    std::vector<int> order((size_t)n);
    for (int i = 0; i < n; ++i) order[(size_t)i] = i;
    std::stable_sort(order.begin(), order.end(), [&](int a, int b) { return cost[(size_t)a] > cost[(size_t)b]; });
    std::vector<std::vector<int>> of((size_t)grid);
    typedef std::pair<int64_t, int> Load;
    std::priority_queue<Load, std::vector<Load>, std::greater<Load>> q;
    for (int i = 0; i < grid; ++i) q.push(Load(0, i));
    for (int i : order) {
        Load l = q.top();
        q.pop();
        of[(size_t)l.second].push_back(i);
        l.first += cost[(size_t)i];
        q.push(l);
    }
    std::vector<T> out;
    out.reserve(items.size());
    begin.assign(1, 0);
    for (int i = 0; i < grid; ++i) {
        for (int j : of[(size_t)i]) out.push_back(items[(size_t)j]);
        begin.push_back((int32_t)out.size());
    }
    items.swap(out);
}

struct Lists {
    std::vector<FwdItem> fwd, empty;
    std::vector<BwdItem> keys, queries;
    std::vector<PrepTile> prep;
    std::vector<SumItem> sums;
    std::vector<int> fwd_cost, key_cost, query_cost;
    int n_parts = 0;
    int64_t pad_rows = 0;
};

// Key ranges that query positions [p0, p1] (p1 >= 0) of a sequence see: the
// sinks [0, s_end) and [w_lo, k_end)
void key_ranges(int64_t p0, int64_t p1, int64_t window, int sinks, int32_t &s_end, int32_t &w_lo, int32_t &k_end) {
    const int64_t lo = std::max<int64_t>(std::max<int64_t>(p0, 0) - window + 1, 0);
    w_lo = (int32_t)lo;
    s_end = (int32_t)std::min<int64_t>(sinks, lo);
    k_end = (int32_t)(p1 + 1);
}

// Items that build_forward makes of ql queries
int64_t forward_items(const syn_window_cfg_t &c, int64_t ql) {
    return c.H_q / c.H_kv % 2 == 0 ? (int64_t)c.H_q / 2 * ceil_div(ql, 128) : (int64_t)c.H_q * ceil_div(ql, 256);
}

void build_forward(Lists &l, const syn_window_cfg_t &c, int64_t window, int64_t q0, int64_t k0, int64_t ql, int64_t kl) {
    const int G = c.H_q / c.H_kv;
    const int64_t off = kl - ql;
    const int bk = fwd_block(c.d);
    const bool heads = G % 2 == 0;  // the two tiles: two heads, else consecutive rows
    const int64_t step = heads ? 128 : 256;
    for (int hk = 0; hk < c.H_kv; ++hk)
        for (int64_t i0 = 0; i0 < ql; i0 += step)
            for (int h = 0; h < G; h += heads ? 2 : 1) {
                FwdItem it;
                std::memset(&it, 0, sizeof(it));
                int64_t last = i0;
                for (int t = 0; t < 2; ++t) {
                    const int64_t i = heads ? i0 : std::min(i0 + 128 * t, ql);
                    it.n_rows[t] = (int32_t)std::min<int64_t>(128, ql - i);
                    it.q_row[t] = (int32_t)(q0 + i);
                    it.pos0[t] = (int32_t)(off + i);
                    it.head[t] = hk * G + h + (heads ? t : 0);
                    last = std::max(last, i + it.n_rows[t] - 1);
                }
                it.kv_row0 = (int32_t)k0;
                it.hk = hk;
                if (off + last < 0) {
                    l.empty.push_back(it);
                    continue;
                }
                key_ranges(off + i0, off + last, window, c.sinks, it.s_end, it.w_lo, it.k_end);
                it.n_blk = ceil_div(it.s_end, bk) + ceil_div(it.k_end - it.w_lo, bk);
                l.fwd.push_back(it);
                l.fwd_cost.push_back(ceil_div(it.s_end, 16) + ceil_div(it.k_end - it.w_lo, 16) + 8);
            }
}

int64_t pad_to_block(int64_t rows) { return (rows + 63) / 64 * 64; }

void build_queries(Lists &l, const syn_window_cfg_t &c, int64_t window, int64_t q0, int64_t k0, int64_t ql, int64_t kl) {
    const int G = c.H_q / c.H_kv;
    const int64_t off = kl - ql;
    for (int64_t i0 = 0; i0 < pad_to_block(ql); i0 += 64)
        l.prep.push_back({(int32_t)(q0 + i0), (int32_t)std::max<int64_t>(0, std::min<int64_t>(64, ql - i0)), (int32_t)(l.pad_rows + i0), 0});
    for (int hk = 0; hk < c.H_kv; ++hk)
        for (int64_t i0 = 0; i0 < ql; i0 += 128)
            for (int h = hk * G; h < (hk + 1) * G; ++h) {
                BwdItem it;
                std::memset(&it, 0, sizeof(it));
                const int64_t last = std::min(i0 + 128, ql) - 1;
                it.row0 = (int32_t)(q0 + i0);
                it.n_rows = (int32_t)(last - i0 + 1);
                it.pos0 = (int32_t)(off + i0);
                it.hk = hk;
                it.h0 = h;
                it.stream0 = (int32_t)k0;
                it.stream_len = (int32_t)kl;
                it.off = (int32_t)off;
                it.pad_row0 = (int32_t)(l.pad_rows + i0);
                it.part = -1;
                if (off + last >= 0) key_ranges(off + i0, off + last, window, c.sinks, it.s_end, it.w_lo, it.k_end);
                l.queries.push_back(it);
                l.query_cost.push_back(ceil_div(it.s_end, 128) + ceil_div(it.k_end - it.w_lo, 128) + 1);
            }
}

// Query blocks of 64 rows that see keys [j0, j1) of a sequence; false: none
bool query_blocks(int64_t j0, int64_t j1, int64_t ql, int64_t off, int64_t window, int sinks, int64_t &b0, int64_t &b1) {
    const int64_t lo = std::max<int64_t>(j0 - off, 0);
    const int64_t hi = j0 < sinks ? ql - 1 : std::min(ql - 1, j1 - 1 + window - 1 - off);
    if (lo > hi) return false;
    b0 = lo / 64;
    b1 = hi / 64 + 1;
    return true;
}

// A key tile's `G` heads x `blocks` cut into head ranges x block ranges of at
// most `most` blocks (>= 1): the fewest parts, and of those the most even
void cut(int G, int64_t blocks, int64_t most, int &by_head, int64_t &by_block) {
    int64_t parts = INT64_MAX, largest = INT64_MAX;
    for (int h = 1; h <= G; ++h) {
        const int64_t heads = (G + h - 1) / h, fit = most / heads;
        if (fit < 1) continue;
        const int64_t b = (blocks + fit - 1) / fit, size = heads * ((blocks + b - 1) / b);
        if (h * b < parts || (h * b == parts && size < largest)) {
            parts = h * b;
            largest = size;
            by_head = h;
            by_block = b;
        }
    }
}

// What an item of dK, dV costs beside its blocks, in blocks (its K and V, the
// start and end of its pipeline); a part's fp32 sums cost 1 / kPartsPerBlock of a
// CTA's block each (written and read again, 256 KB).
constexpr int kItemCost = 4, kPartsPerBlock = 28;

// The largest part of a key tile, in blocks.  Where there are few tiles a CTA,
// the one of a ladder around a CTA's share that gives the least cost of the
// busiest CTA and the sums; the costs alone are dealt out.  (Sequences of 1024,
// 517, 63 and 1531 tokens, 14/2 heads, window 300, against parts of 16 blocks:
// busiest CTA 32 -> 25 blocks, 184 -> 132 parts, gradient 77.1 -> 69.6 us; four
// of 2048, causal, 32/8 heads 464.8 -> 429.2; one of 257, 16/4 heads 33.4 -> 28.5;
// the plan takes 0.1 to 0.4 ms longer.)  Where there are many the order costliest first evens them out.
int64_t part_size(const std::vector<int64_t> &tiles, int G, int num_sms) {
    int64_t blocks = 0;
    for (int64_t t : tiles) blocks += t * G;
    const int64_t share = std::max<int64_t>(blocks / num_sms, 1);
    if (tiles.size() > 4 * (size_t)num_sms) return std::max<int64_t>(share / 2, 16);
    int64_t best = share, least = INT64_MAX;
    std::vector<int> cost;
    for (int64_t most = std::max<int64_t>(share / 6, 4); most <= 2 * share + 24; most += std::max<int64_t>(most / 5, 2)) {
        cost.clear();
        int64_t parts = 0;
        for (int64_t t : tiles) {
            int h;
            int64_t b;
            cut(G, t, most, h, b);
            for (int x = 0; x < h; ++x)
                for (int64_t y = 0; y < b; ++y)
                    cost.push_back((int)((G * (x + 1) / h - G * x / h) * (t * (y + 1) / b - t * y / b)) + kItemCost);
            parts += h * b > 1 ? h * b : 0;
        }
        std::sort(cost.begin(), cost.end(), std::greater<int>());
        std::vector<int64_t> load((size_t)std::min<int64_t>(num_sms, (int64_t)cost.size()), 0);
        std::priority_queue<int64_t, std::vector<int64_t>, std::greater<int64_t>> q(std::greater<int64_t>(), std::move(load));
        int64_t busiest = 0;
        for (int x : cost) {
            const int64_t v = q.top() + x;
            q.pop();
            q.push(v);
            busiest = std::max(busiest, v);
        }
        if (busiest * kPartsPerBlock + parts < least) {
            least = busiest * kPartsPerBlock + parts;
            best = most;
        }
    }
    return best;
}

void build_keys(Lists &l, const syn_window_cfg_t &c, int64_t window, int64_t q0, int64_t k0, int64_t ql, int64_t kl,
                int64_t most) {
    const int G = c.H_q / c.H_kv;
    const int64_t off = kl - ql;
    for (int hk = 0; hk < c.H_kv; ++hk)
        for (int64_t j0 = 0; j0 < kl; j0 += 128) {
            const int64_t j1 = std::min(j0 + 128, kl);
            int64_t b0 = 0, b1 = 0;
            SumItem sum;
            std::memset(&sum, 0, sizeof(sum));
            sum.row0 = (int32_t)(k0 + j0);
            sum.n_rows = (int32_t)(j1 - j0);
            sum.hk = hk;
            sum.part0 = l.n_parts;
            if (!query_blocks(j0, j1, ql, off, window, c.sinks, b0, b1)) {
                l.sums.push_back(sum);  // seen by no query: zero gradients
                continue;
            }
            int by_head;
            int64_t by_block;
            cut(G, b1 - b0, most, by_head, by_block);
            const int64_t parts = by_head * by_block;
            for (int x = 0; x < by_head; ++x)
                for (int64_t y = 0; y < by_block; ++y) {
                    BwdItem it;
                    std::memset(&it, 0, sizeof(it));
                    it.row0 = sum.row0;
                    it.n_rows = sum.n_rows;
                    it.pos0 = (int32_t)j0;
                    it.hk = hk;
                    it.h0 = hk * G + G * x / by_head;
                    it.h1 = hk * G + G * (x + 1) / by_head;
                    it.stream0 = (int32_t)q0;
                    it.stream_len = (int32_t)ql;
                    it.off = (int32_t)off;
                    it.b0 = (int32_t)(b0 + (b1 - b0) * y / by_block);
                    it.b1 = (int32_t)(b0 + (b1 - b0) * (y + 1) / by_block);
                    it.pad_row0 = (int32_t)l.pad_rows;
                    it.part = parts > 1 ? l.n_parts++ : -1;
                    l.keys.push_back(it);
                    l.key_cost.push_back((it.h1 - it.h0) * (it.b1 - it.b0) + kItemCost);
                }
            if (parts > 1) {
                sum.n_parts = (int32_t)parts;
                l.sums.push_back(sum);
            }
        }
}

// (query row, visible key) pairs of a sequence
int64_t count_pairs(int64_t ql, int64_t kl, int64_t window, int sinks) {
    int64_t n = 0;
    for (int64_t p = std::max<int64_t>(kl - ql, 0); p < kl; ++p) {
        const int64_t lo = std::max<int64_t>(p - window + 1, 0);
        n += p + 1 - lo + std::min<int64_t>(lo, sinks);
    }
    return n;
}

bool al16(const void *x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; }

int check_rows(const char *name, const syn_window_rows_t *r, int64_t rows, int heads) {
    if (r == nullptr || (rows > 0 && r->p == nullptr)) return host_fail(SYN_ERR_INVALID, std::string(name) + ": null operand");
    if (!al16(r->p)) return host_fail(SYN_ERR_INVALID, std::string(name) + ": operand not 16-byte aligned");
    const bool token = rows > 1, head = heads > 1;
    if ((token && (r->token <= 0 || r->token % 8 != 0)) || (head && (r->head <= 0 || r->head % 8 != 0)))
        return host_fail(SYN_ERR_INVALID, std::string(name) + ": strides must be positive multiples of 8 elements");
    if ((token && r->token >= (int64_t)1 << 38) || (head && r->head >= (int64_t)1 << 38))
        return host_fail(SYN_ERR_UNSUPPORTED, std::string(name) + ": stride of 2^38 elements or more");
    return SYN_OK;
}

// Written rows may not overlap
int check_written(const char *name, const syn_window_rows_t *r, int64_t rows, int heads, int d) {
    if ((rows > 1 && r->token < d) || (heads > 1 && r->head < d)) return host_fail(SYN_ERR_INVALID, std::string(name) + ": output rows overlap");
    return SYN_OK;
}

int encode(CUtensorMap *m, const syn_window_plan_s *pl, const syn_window_rows_t &r, int64_t rows, int heads, uint32_t box_rows) {
    // a stride of an axis with one entry is never used; keep it valid
    const int64_t d = pl->cfg.d, head = heads > 1 ? r.head : d, token = rows > 1 ? r.token : d * heads;
    return host_encode_3d(m, r.p, pl->bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (uint64_t)d,
                          (uint64_t)heads, (uint64_t)rows, (uint64_t)head * 2, (uint64_t)token * 2, 64, box_rows,
                          CU_TENSOR_MAP_SWIZZLE_128B);
}

Common common_of(const syn_window_plan_s *pl) {
    const syn_window_cfg_t &c = pl->cfg;
    Common x;
    std::memset(&x, 0, sizeof(x));
    x.window = (int32_t)c.window;
    x.sinks = c.sinks;
    x.H_q = c.H_q;
    x.G = c.H_q / c.H_kv;
    x.scale = c.scale;
    x.scale_log2 = c.scale * 1.4426950408889634f;
    x.timeout_ns = c.timeout_ns;
    x.err = pl->d_err;
    return x;
}

Out out_of(const syn_window_rows_t *r) { return {r->p, r->token, r->head}; }

}  // namespace

extern "C" {

int syn_window_cfg_default(syn_window_cfg_t *c) {
    if (c == nullptr) return host_fail(SYN_ERR_INVALID, "null cfg");
    std::memset(c, 0, sizeof(*c));
    c->dtype = SYN_DTYPE_BF16;
    c->H_q = c->H_kv = 1;
    c->d = 128;
    return SYN_OK;
}

int syn_window_plan_create(syn_window_plan_t *out, const syn_window_cfg_t *cfg, int n_seqs, const int64_t *q_lens,
                           const int64_t *k_lens) try {
    if (out == nullptr || cfg == nullptr) return host_fail(SYN_ERR_INVALID, "null argument");
    *out = nullptr;
    syn_window_cfg_t c = *cfg;
    if (n_seqs < 0 || (n_seqs > 0 && (q_lens == nullptr || k_lens == nullptr)))
        return host_fail(SYN_ERR_INVALID, "need q_lens and k_lens of n_seqs >= 0 sequences");
    if (c.dtype == SYN_DTYPE_F32) return host_fail(SYN_ERR_UNSUPPORTED, "attention takes bf16 or fp16");
    if (c.dtype != SYN_DTYPE_BF16 && c.dtype != SYN_DTYPE_F16) return host_fail(SYN_ERR_INVALID, "unknown dtype");
    if (c.H_q < 1 || c.H_kv < 1 || c.H_q % c.H_kv != 0) return host_fail(SYN_ERR_INVALID, "need H_q % H_kv == 0");
    if (c.H_q > 1024) return host_fail(SYN_ERR_UNSUPPORTED, "H_q > 1024");
    if (c.d != 64 && c.d != 128) return host_fail(SYN_ERR_UNSUPPORTED, "head dimension must be 64 or 128");
    if (c.window < 0 || c.sinks < 0) return host_fail(SYN_ERR_INVALID, "window and sinks must not be negative");
    if (!(c.scale >= 0.f) || !std::isfinite(c.scale)) return host_fail(SYN_ERR_INVALID, "bad scale");
    if (c.backward != 0 && c.backward != 1) return host_fail(SYN_ERR_INVALID, "backward must be 0 or 1");
    int64_t q_rows = 0, k_rows = 0, n_fwd = 0, n_queries = 0, n_keys = 0;
    for (int s = 0; s < n_seqs; ++s) {
        if (q_lens[s] < 0 || k_lens[s] < 0) return host_fail(SYN_ERR_INVALID, "negative length");
        if (q_lens[s] >= kMaxLen || k_lens[s] >= kMaxLen) return host_fail(SYN_ERR_UNSUPPORTED, "length of 2^29 or more");
        q_rows += q_lens[s];
        k_rows += k_lens[s];
        n_fwd += forward_items(c, q_lens[s]);
        n_queries += (int64_t)c.H_q * ceil_div(q_lens[s], 128);
        n_keys += (int64_t)c.H_kv * ceil_div(k_lens[s], 128);
    }
    if (q_rows >= (int64_t)1 << 30 || k_rows >= (int64_t)1 << 30) return host_fail(SYN_ERR_UNSUPPORTED, "2^30 or more rows");
    if (n_fwd >= kMaxItems || (c.backward && (n_queries >= kMaxItems || n_keys >= kMaxItems)))
        return host_fail(SYN_ERR_UNSUPPORTED, "2^28 or more tiles");
    if (c.window == 0 || c.window > kNoWindow) c.window = kNoWindow;
    c.sinks = (int)std::min<int64_t>(c.sinks, kMaxLen);
    if (c.scale == 0.f) c.scale = 1.f / std::sqrt((float)c.d);
    if (c.timeout_ns == 0) c.timeout_ns = host_timeout_ns();
    std::vector<int64_t> tiles;  // query blocks of each tile of keys
    for (int s = 0; c.backward && s < n_seqs; ++s)
        for (int64_t j0 = 0; j0 < k_lens[s]; j0 += 128) {
            int64_t b0, b1;
            if (query_blocks(j0, std::min(j0 + 128, k_lens[s]), q_lens[s], k_lens[s] - q_lens[s], c.window, c.sinks, b0, b1))
                tiles.insert(tiles.end(), (size_t)c.H_kv, b1 - b0);
        }
    int rc = host_load_driver();
    if (rc != SYN_OK) return rc;

    syn_window_plan_s *pl = new syn_window_plan_s();
    std::unique_ptr<syn_window_plan_s, void (*)(syn_window_plan_s *)> unfinished(pl, free_plan);
#define PL_CK(call)                                                                                                     \
    do {                                                                                                                \
        cudaError_t e__ = (call);                                                                                       \
        if (e__ != cudaSuccess) return host_fail(SYN_ERR_CUDA, std::string("window plan: ") + cudaGetErrorString(e__)); \
    } while (0)
    pl->cfg = c;
    pl->bf16 = c.dtype == SYN_DTYPE_BF16;
    PL_CK(cudaGetDevice(&pl->device));
    PL_CK(cudaDeviceGetAttribute(&pl->num_sms, cudaDevAttrMultiProcessorCount, pl->device));
    PL_CK(fwd_prepare(c.d, pl->bf16));
    if (c.backward) {
        PL_CK(dkv_prepare(c.d, pl->bf16));
        PL_CK(dq_prepare(c.d, pl->bf16));
    }

    const int64_t most = part_size(tiles, c.H_q / c.H_kv, pl->num_sms);
    Lists l;
    int64_t q0 = 0, k0 = 0, pairs = 0;
    for (int s = 0; s < n_seqs; ++s) {
        const int64_t ql = q_lens[s], kl = k_lens[s];
        build_forward(l, c, c.window, q0, k0, ql, kl);
        if (c.backward) {
            build_queries(l, c, c.window, q0, k0, ql, kl);
            build_keys(l, c, c.window, q0, k0, ql, kl, most);
            l.pad_rows += pad_to_block(ql);
        }
        pairs += count_pairs(ql, kl, c.window, c.sinks);
        q0 += ql;
        k0 += kl;
    }
    std::vector<int32_t> begin, key_begin, query_begin;
    deal(l.fwd, l.fwd_cost, pl->num_sms, begin);
    deal(l.keys, l.key_cost, pl->num_sms, key_begin);
    deal(l.queries, l.query_cost, pl->num_sms, query_begin);
    pl->grid_f = (int)begin.size() - 1;
    pl->grid_k = (int)key_begin.size() - 1;
    pl->grid_q = (int)query_begin.size() - 1;
    if (pl->grid_f == 0 && !l.empty.empty()) {  // only empty tiles: CTAs without items
        pl->grid_f = (int)std::min<size_t>(l.empty.size(), (size_t)pl->num_sms);
        begin.assign((size_t)pl->grid_f + 1, 0);
    }
    pl->n_empty = (int)l.empty.size();
    pl->n_prep = (int)l.prep.size();
    pl->n_sums = (int)l.sums.size();
    pl->pad_rows = l.pad_rows;
    const size_t stats = (size_t)2 * (size_t)c.H_q * (size_t)l.pad_rows * sizeof(float);
    const size_t part = (size_t)l.n_parts * 2 * 128 * (size_t)c.d * sizeof(float);
    PL_CK(upload(&pl->d_items, l.fwd));
    PL_CK(upload(&pl->d_empty, l.empty));
    PL_CK(upload(&pl->d_begin, begin));
    if (c.backward) {
        PL_CK(upload(&pl->d_key_items, l.keys));
        PL_CK(upload(&pl->d_key_begin, key_begin));
        PL_CK(upload(&pl->d_query_items, l.queries));
        PL_CK(upload(&pl->d_query_begin, query_begin));
        PL_CK(upload(&pl->d_prep, l.prep));
        PL_CK(upload(&pl->d_sums, l.sums));
        PL_CK(cudaMalloc(&pl->d_stats, std::max<size_t>(stats, 16)));
        PL_CK(cudaMalloc(&pl->d_part, std::max<size_t>(part, 16)));
    }
    PL_CK(cudaMalloc(&pl->d_err, 4 * sizeof(int32_t)));
    PL_CK(cudaMemset(pl->d_err, 0, 4 * sizeof(int32_t)));
    PL_CK(cudaDeviceSynchronize());
#undef PL_CK
    syn_window_info_t &f = pl->info;
    std::memset(&f, 0, sizeof(f));
    f.n_seqs = n_seqs;
    f.n_items = (int)l.fwd.size();
    f.n_bwd_items = (int)(l.keys.size() + l.queries.size());
    f.n_parts = l.n_parts;
    f.grid = pl->grid_f;
    f.q_rows = q_rows;
    f.k_rows = k_rows;
    f.pairs = pairs;
    f.workspace_bytes = (int64_t)(c.backward ? stats + part : 0);
    unfinished.release();
    *out = pl;
    return SYN_OK;
} catch (const std::bad_alloc &) {  // (the lists grow with the lengths)
    return host_fail(SYN_ERR_UNSUPPORTED, "not enough host memory for the work lists");
}

int syn_window_plan_destroy(syn_window_plan_t pl) {
    if (pl != nullptr) free_plan(pl);
    return SYN_OK;
}

int syn_window_plan_query(syn_window_plan_t pl, syn_window_info_t *info) {
    if (pl == nullptr || info == nullptr) return host_fail(SYN_ERR_INVALID, "null argument");
    *info = pl->info;
    return SYN_OK;
}

int syn_window_attention(syn_window_plan_t pl, const syn_window_rows_t *Q, const syn_window_rows_t *K,
                         const syn_window_rows_t *V, const syn_window_rows_t *O, float *lse, void *stream) {
    if (pl == nullptr) return host_fail(SYN_ERR_INVALID, "null plan");
    const syn_window_cfg_t &c = pl->cfg;
    const int64_t nq = pl->info.q_rows, nk = pl->info.k_rows;
    int rc;
    if ((rc = check_rows("Q", Q, nq, c.H_q)) != SYN_OK || (rc = check_rows("K", K, nk, c.H_kv)) != SYN_OK ||
        (rc = check_rows("V", V, nk, c.H_kv)) != SYN_OK || (rc = check_rows("O", O, nq, c.H_q)) != SYN_OK ||
        (rc = check_written("O", O, nq, c.H_q, c.d)) != SYN_OK)
        return rc;
    if ((reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return host_fail(SYN_ERR_INVALID, "lse: not aligned");
    if (nq == 0) return SYN_OK;
    FwdMaps m;
    const uint32_t bk = (uint32_t)fwd_block(c.d);
    // without any key no item reads K or V
    const syn_window_rows_t &k = nk > 0 ? *K : *Q, &v = nk > 0 ? *V : *Q;
    const int64_t rows = nk > 0 ? nk : nq;
    const int heads = nk > 0 ? c.H_kv : c.H_q;
    if ((rc = encode(&m.q, pl, *Q, nq, c.H_q, 128)) != SYN_OK || (rc = encode(&m.k, pl, k, rows, heads, bk)) != SYN_OK ||
        (rc = encode(&m.k16, pl, k, rows, heads, 16)) != SYN_OK || (rc = encode(&m.v, pl, v, rows, heads, bk)) != SYN_OK ||
        (rc = encode(&m.v16, pl, v, rows, heads, 16)) != SYN_OK)
        return rc;
    FwdParams p;
    std::memset(&p, 0, sizeof(p));
    p.c = common_of(pl);
    p.items = pl->d_items;
    p.begin = pl->d_begin;
    p.empty = pl->d_empty;
    p.n_empty = pl->n_empty;
    p.o = out_of(O);
    p.lse = lse;
    WIN_CK(fwd_launch(c.d, pl->bf16, pl->grid_f, p, m, static_cast<cudaStream_t>(stream)));
    return SYN_OK;
}

int syn_window_attention_backward(syn_window_plan_t pl, const syn_window_rows_t *dO, const syn_window_rows_t *Q,
                                  const syn_window_rows_t *K, const syn_window_rows_t *V, const syn_window_rows_t *O,
                                  const float *lse, const syn_window_rows_t *dQ, const syn_window_rows_t *dK,
                                  const syn_window_rows_t *dV, void *stream) {
    if (pl == nullptr) return host_fail(SYN_ERR_INVALID, "null plan");
    const syn_window_cfg_t &c = pl->cfg;
    if (!c.backward) return host_fail(SYN_ERR_INVALID, "the plan was made without backward");
    const int64_t nq = pl->info.q_rows, nk = pl->info.k_rows;
    int rc;
    if ((rc = check_rows("dO", dO, nq, c.H_q)) != SYN_OK || (rc = check_rows("Q", Q, nq, c.H_q)) != SYN_OK ||
        (rc = check_rows("K", K, nk, c.H_kv)) != SYN_OK || (rc = check_rows("V", V, nk, c.H_kv)) != SYN_OK ||
        (rc = check_rows("O", O, nq, c.H_q)) != SYN_OK || (rc = check_rows("dQ", dQ, nq, c.H_q)) != SYN_OK ||
        (rc = check_rows("dK", dK, nk, c.H_kv)) != SYN_OK || (rc = check_rows("dV", dV, nk, c.H_kv)) != SYN_OK ||
        (rc = check_written("dQ", dQ, nq, c.H_q, c.d)) != SYN_OK || (rc = check_written("dK", dK, nk, c.H_kv, c.d)) != SYN_OK ||
        (rc = check_written("dV", dV, nk, c.H_kv, c.d)) != SYN_OK)
        return rc;
    if (nq > 0 && (lse == nullptr || (reinterpret_cast<uintptr_t>(lse) & 3u) != 0))
        return host_fail(SYN_ERR_INVALID, "lse: null or not aligned");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    BwdParams p;
    std::memset(&p, 0, sizeof(p));
    p.c = common_of(pl);
    p.nlse2 = pl->d_stats;
    p.ndelta = pl->d_stats + (int64_t)c.H_q * pl->pad_rows;
    p.pad_rows = pl->pad_rows;
    p.part = pl->d_part;
    if (nq > 0) {
        PrepParams r;
        std::memset(&r, 0, sizeof(r));
        r.tiles = pl->d_prep;
        r.o = O->p;
        r.o_token = O->token;
        r.o_head = O->head;
        r.d_o = dO->p;
        r.do_token = dO->token;
        r.do_head = dO->head;
        r.lse = lse;
        r.nlse2 = pl->d_stats;
        r.ndelta = pl->d_stats + (int64_t)c.H_q * pl->pad_rows;
        r.pad_rows = pl->pad_rows;
        r.H_q = c.H_q;
        r.d = c.d;
        WIN_CK(bwd_prep_launch(pl->bf16, pl->n_prep, r, st));
    }
    if (nq > 0 && nk > 0) {
        BwdMaps keys, queries;
        if ((rc = encode(&keys.x, pl, *K, nk, c.H_kv, 128)) != SYN_OK || (rc = encode(&keys.y, pl, *V, nk, c.H_kv, 128)) != SYN_OK ||
            (rc = encode(&keys.u, pl, *Q, nq, c.H_q, 64)) != SYN_OK || (rc = encode(&keys.w, pl, *dO, nq, c.H_q, 64)) != SYN_OK ||
            (rc = encode(&queries.x, pl, *Q, nq, c.H_q, 128)) != SYN_OK || (rc = encode(&queries.y, pl, *dO, nq, c.H_q, 128)) != SYN_OK ||
            (rc = encode(&queries.u, pl, *K, nk, c.H_kv, 128)) != SYN_OK || (rc = encode(&queries.w, pl, *V, nk, c.H_kv, 128)) != SYN_OK)
            return rc;
        if (pl->grid_q > 0) {
            p.items = pl->d_query_items;
            p.begin = pl->d_query_begin;
            p.dx = out_of(dQ);
            WIN_CK(dq_launch(c.d, pl->bf16, pl->grid_q, p, queries, st));
        }
        if (pl->grid_k > 0) {
            p.items = pl->d_key_items;
            p.begin = pl->d_key_begin;
            p.dx = out_of(dK);
            p.dy = out_of(dV);
            WIN_CK(dkv_launch(c.d, pl->bf16, pl->grid_k, p, keys, st));
        }
    } else if (nq > 0) {  // no key at all: dQ = 0
        for (int h = 0; h < c.H_q; ++h)
            WIN_CK(cudaMemset2DAsync(static_cast<uint16_t *>(dQ->p) + (c.H_q > 1 ? h * dQ->head : 0),
                                     (size_t)(nq > 1 ? dQ->token : c.d) * 2, 0, (size_t)c.d * 2, (size_t)nq, st));
    }
    if (pl->n_sums > 0) {
        SumParams s;
        std::memset(&s, 0, sizeof(s));
        s.items = pl->d_sums;
        s.part = pl->d_part;
        s.dk = out_of(dK);
        s.dv = out_of(dV);
        s.scale = c.scale;
        s.d = c.d;
        WIN_CK(bwd_sum_launch(pl->bf16, pl->n_sums, s, st));
    }
    return SYN_OK;
}

int syn_window_sync_status(syn_window_plan_t pl, void *stream) {
    if (pl == nullptr) return host_fail(SYN_ERR_INVALID, "null plan");
    WIN_CK(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)));
    int32_t e[4] = {0, 0, 0, 0};
    WIN_CK(cudaMemcpy(e, pl->d_err, sizeof(e), cudaMemcpyDeviceToHost));
    if (e[0] == 0) return SYN_OK;
    WIN_CK(cudaMemset(pl->d_err, 0, sizeof(e)));
    WIN_CK(cudaDeviceSynchronize());  // (cleared before a later call, of whatever stream, can report)
    return host_fail(e[0], std::string("device error ") + syn_status_string(e[0]) + " at site " + std::to_string(e[1]) +
                               " in CTA " + std::to_string(e[2]) + " (info " + std::to_string(e[3]) + ")");
}

}  // extern "C"
