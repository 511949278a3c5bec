// ffn.cu -- plans and C ABI of the gated feed-forward block (include/syn_ffn.h;
// kernels in ffn_fwd.cu and ffn_bwd.cu).
#include <algorithm>
#include <cstring>
#include <new>
#include <string>
#include <utility>

#include "ffn.cuh"
#include "host_util.h"
#include "syn_ffn.h"

using namespace syn;
using namespace syn::ffn;

struct syn_ffn_plan_s {
    syn_ffn_cfg_t cfg;
    int device = 0, pairs = 0;
    bool bf16 = true, wide = false;  // wide: G and U in fp32
    int32_t *d_err = nullptr;
    Parts parts = {nullptr, nullptr};  // of as many items as there are pairs
};

namespace {

#define FFN_CK(call)                                                                                  \
    do {                                                                                              \
        cudaError_t e__ = (call);                                                                     \
        if (e__ != cudaSuccess) return host_fail(SYN_ERR_CUDA, std::string(#call) + ": " + cudaGetErrorString(e__)); \
    } while (0)

constexpr int kMaxCols = 1 << 20;

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

int check_mat(const char *name, const syn_ffn_mat_t *m, int64_t rows, int cols, bool written, int multiple = 8) {
    if (m == nullptr || (rows > 0 && m->p == nullptr)) return host_fail(SYN_ERR_INVALID, std::string(name) + ": null operand");
    if ((reinterpret_cast<uintptr_t>(m->p) & 15u) != 0) return host_fail(SYN_ERR_INVALID, std::string(name) + ": operand not 16-byte aligned");
    if (rows < 2) return SYN_OK;
    if (m->row <= 0 || m->row % multiple != 0)
        return host_fail(SYN_ERR_INVALID, std::string(name) + ": row stride must be a positive multiple of " + std::to_string(multiple) + " elements");
    if (m->row >= (int64_t)1 << 38) return host_fail(SYN_ERR_UNSUPPORTED, std::string(name) + ": stride of 2^38 elements or more");
    if (written && m->row < cols) return host_fail(SYN_ERR_INVALID, std::string(name) + ": output rows overlap");
    return SYN_OK;
}

// An operand of a call.  `place`: an output each of whose elements is written by the
// thread that has read it, so that it may take the place of a `replaced` input.
struct Mat {
    const char *name;
    const syn_ffn_mat_t *m;
    int64_t rows;
    int cols;
    bool written, needed;
    int multiple = 8;
    bool replaced = false, place = false;
};
// Operands as above, no output in the place of another operand (matrices may lie
// between each other's rows, so that only their beginnings tell)
int check_mats(const Mat *mats, int n) {
    int rc;
    for (int i = 0; i < n; ++i)
        if (mats[i].needed && (rc = check_mat(mats[i].name, mats[i].m, mats[i].rows, mats[i].cols, mats[i].written, mats[i].multiple)) != SYN_OK)
            return rc;
    for (int j = 0; j < n; ++j)
        for (int i = 0; i < j; ++i) {
            const Mat &a = mats[i], &b = mats[j];
            if (!a.needed || !b.needed || !(a.written || b.written) || a.rows == 0 || b.rows == 0 || a.m->p != b.m->p) continue;
            if (!(a.replaced && b.place && a.multiple == b.multiple && (a.rows < 2 || a.m->row == b.m->row)))
                return host_fail(SYN_ERR_INVALID, std::string(b.name) + " cannot take the place of " + a.name);
        }
    return SYN_OK;
}

int check_call(const syn_ffn_plan_s *pl, int64_t n_tokens) {
    if (pl == nullptr) return host_fail(SYN_ERR_INVALID, "null plan");
    int device = -1;
    FFN_CK(cudaGetDevice(&device));
    if (device != pl->device) return host_fail(SYN_ERR_INVALID, "the plan belongs to another device than the current one");
    if (n_tokens < 0) return host_fail(SYN_ERR_INVALID, "negative token count");
    if (n_tokens >= (int64_t)1 << 30) return host_fail(SYN_ERR_UNSUPPORTED, "2^30 or more tokens in one call");
    return SYN_OK;
}

// Boxes of 64 columns x 64 rows to load (of fewer: `box`), x 32 rows to store
int encode(CUtensorMap *m, const syn_ffn_plan_s *pl, const syn_ffn_mat_t &x, int64_t rows, int cols, bool store, int box = 64) {
    const int64_t row = rows > 1 ? x.row : cols;  // (never used otherwise; kept valid)
    return host_encode_rows(m, x.p, pl->bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (uint64_t)cols,
                            (uint64_t)rows, (uint64_t)row * 2, 64, store ? 32 : (uint32_t)box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Boxes of 32 columns x 32 rows of an fp32 matrix to store
int encode_wide(CUtensorMap *m, const syn_ffn_mat_t &x, int64_t rows, int cols) {
    const int64_t row = rows > 1 ? x.row : cols;
    return host_encode_rows(m, x.p, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, (uint64_t)cols, (uint64_t)rows, (uint64_t)row * 4, 32, 32,
                            CU_TENSOR_MAP_SWIZZLE_128B);
}

Common common_of(const syn_ffn_plan_s *pl) { return {pl->d_err, pl->cfg.timeout_ns}; }

// r / n for r < 2^31 as r * magic >> shift
void divisor(uint32_t n, uint32_t &magic, uint32_t &shift) {
    uint32_t bits = 0;
    while (((uint64_t)1 << bits) < n) ++bits;
    shift = 31 + bits;
    magic = (uint32_t)((((uint64_t)1 << shift) + n - 1) / n);
}

// Row tiles of a band: those of a wave of pairs and as many columns
int band_of(int pairs, int tiles_m) {
    int b = 1;
    while (b * b < pairs) ++b;
    return std::min(b, std::max(tiles_m, 1));
}

constexpr size_t kPartBytes = (size_t)kTileM * 256 * sizeof(float);  // of an item, the widest
constexpr size_t kStrips = 8;                                        // of a tile: quarters of two CTAs, each counted by itself

// Times of tiles in parts, in us: a stage, having parts at all, each part of a tile (the
// last quarter to arrive joins them all), each part of any tile (all pairs leave and join
// theirs at once).  Fitted to forward calls, and to the gradient's, whose stages are
// twice as large and run beside other tiles.
struct Costs {
    double stage, any, part, item;
};
// A stage takes longer where the rows that it brings do not begin at whole 32-byte sectors
// (300 tokens in one piece, 2752 -> 704: 11.5 us, 2672 -> 728: 15.5), 16 rows of X or
// fewer aside.  Told by the sizes, as rows lie one behind the other, and not by addresses:
// the parts decide the bits of a result.
Costs fwd_costs(int64_t n_tokens, int d, int d_ff) {
    return {0.3 + (n_tokens > 16 && d % 16 != 0 ? 0.12 : 0.0) + (d_ff % 16 != 0 ? 0.12 : 0.0), 2.9, 1.0, 0.015};
}
// (The gradient, dX and dW, whole tiles against this rule's parts: 120 tokens, 512 -> 14400
// 147 us, 42 in 12 parts; 200, 1024 -> 8192 86, 37 in 8; 9000, 264 -> 520 63, 39.5 in 4;
// 30000, 512 -> 512 167, 77 in 7; 128, 4096 -> 14336 162, 106 in 4; 2116, 312 -> 2920 48, 42
// in 2; but 277, 4024 -> 6808 89.6, 92.2 in 2.)
constexpr Costs kBwdCosts = {0.6, 0.0, 0.5, 0.25};

// Parts of each of `tiles` tiles of `stages` stages, where they leave pairs without
// work (18 tiles of 39 stages 25.1 -> 16.3 us in four parts, 512 tokens, 3256 -> 456: 16
// of 26 19.0 -> 14.6 in three; but 19 tiles of 28 stages 13.4 -> 15.2, 37 in two parts
// 16.5 -> 17.5).
int parts_of(int tiles, int stages, int pairs, const Costs &c) {
    int best = 1;
    double least = c.stage * stages;
    for (int s = 2; s <= 16 && tiles * s <= pairs && s <= stages; ++s) {
        const double cost = c.stage * ((stages + s - 1) / s) + c.any + c.part * s + c.item * (tiles * s);
        if (cost < least) {
            least = cost;
            best = s;
        }
    }
    return best;
}

// Rounds of the shorter kind's tiles in which every pair takes part, so that the pairs
// with one item of the longer kind more end with the others
int even_rounds(int pairs, int items1, int tiles2, int cost1, int cost2) {
    const int more = items1 % pairs, others = pairs - more;
    int best = 0;
    int64_t least = INT64_MAX;
    for (int e = 0; (int64_t)(e - 1) * pairs < tiles2; ++e) {
        const int64_t left = std::max<int64_t>(tiles2 - (int64_t)e * pairs, 0);
        const int64_t a = (more > 0 ? cost1 : 0) + (int64_t)e * cost2, b = (e + (left + others - 1) / others) * (int64_t)cost2;
        if (std::max(a, b) < least) {
            least = std::max(a, b);
            best = e;
        }
    }
    return best;
}

// A forward's tiles: columns of a product, rows and columns of tiles (n 0: too many), parts
struct FwdTiles {
    int width, m, n, split;
};
FwdTiles fwd_tiles(const syn_ffn_plan_s *pl, int64_t n_tokens) {
    const syn_ffn_cfg_t &c = pl->cfg;
    const int m = ceil_div(n_tokens, kTileM), wide = ceil_div(c.d_ff, 128), narrow = ceil_div(c.d_ff, 64);
    if ((int64_t)m * narrow >= (int64_t)1 << 30) return {0, m, 0, 1};
    // a round of narrow tiles takes 0.58 of one of wide ones (8 tokens: 3 rounds of narrow
    // ones for 2; 1003 tokens, 3584 -> 2368: 1 of wide ones for 2)
    const int64_t rounds_w = ceil_div((int64_t)m * wide, pl->pairs), rounds_n = ceil_div((int64_t)m * narrow, pl->pairs);
    if (n_tokens > 64 && rounds_n * 58 >= rounds_w * 100) return {256, m, wide, 1};
    return {128, m, narrow, parts_of(m * narrow, ceil_div(c.d, 128), pl->pairs, fwd_costs(n_tokens, c.d, c.d_ff))};
}

// The gradient's tiles of dX and of dW: those of the longer kind first, in parts
constexpr int kEnd = 2;  // (stages that a tile's start and end cost, about)
struct BwdDeal {
    bool dw_first;
    int n1, n2, stages1, stages2, split;
};
BwdDeal bwd_deal(const syn_ffn_plan_s *pl, int64_t n_tokens, int dx, int dw) {
    const int tiles[2] = {dx, dw}, stages[2] = {2 * ceil_div(pl->cfg.d_ff, 128), ceil_div(n_tokens, 128)};
    const bool first = dx == 0 || (dw > 0 && stages[1] > stages[0]);
    BwdDeal t = {first, tiles[first], tiles[!first], stages[first], stages[!first], 1};
    // the longer kind's tiles are cut where the pairs would wait for one of them
    if (((int64_t)t.n1 * (t.stages1 + kEnd) + (int64_t)t.n2 * (t.stages2 + kEnd)) / pl->pairs < t.stages1 + kEnd)
        t.split = parts_of(t.n1, t.stages1, pl->pairs, kBwdCosts);
    return t;
}
int dx_tiles(const syn_ffn_plan_s *pl, int64_t n_tokens, int &m, int &n) {
    m = ceil_div(n_tokens, kTileM);
    n = ceil_div(pl->cfg.d, 256);
    return (int64_t)m * n >= (int64_t)1 << 30 ? host_fail(SYN_ERR_UNSUPPORTED, "2^30 or more tiles") : SYN_OK;
}
void dw_tiles(const syn_ffn_plan_s *pl, int &m, int &n) {
    m = ceil_div(pl->cfg.d, kTileM);
    n = 2 * ceil_div(pl->cfg.d_ff, 256);
}

}  // namespace

extern "C" {

int syn_ffn_cfg_default(syn_ffn_cfg_t *c) {
    if (c == nullptr) return host_fail(SYN_ERR_INVALID, "null cfg");
    std::memset(c, 0, sizeof(*c));
    c->dtype = SYN_DTYPE_BF16;
    c->d = 4096;
    c->d_ff = 14336;
    c->act = SYN_ACT_SILU;
    c->backward = 1;
    return SYN_OK;
}

int syn_ffn_plan_create(syn_ffn_plan_t *out, const syn_ffn_cfg_t *cfg) {
    if (out == nullptr || cfg == nullptr) return host_fail(SYN_ERR_INVALID, "null argument");
    *out = nullptr;
    syn_ffn_cfg_t c = *cfg;
    if (c.dtype == SYN_DTYPE_F32) return host_fail(SYN_ERR_UNSUPPORTED, "the gated block takes bf16 or fp16");
    if (c.dtype != SYN_DTYPE_BF16 && c.dtype != SYN_DTYPE_F16) return host_fail(SYN_ERR_INVALID, "unknown dtype");
    if (c.d < 1 || c.d_ff < 1) return host_fail(SYN_ERR_INVALID, "d and d_ff must be positive");
    if (c.d % 8 != 0 || c.d_ff % 8 != 0) return host_fail(SYN_ERR_UNSUPPORTED, "d and d_ff must be multiples of 8");
    if (c.d > kMaxCols || c.d_ff > kMaxCols) return host_fail(SYN_ERR_UNSUPPORTED, "d or d_ff above 2^20");
    if (c.act < SYN_ACT_SILU || c.act > SYN_ACT_GELU_TANH) return host_fail(SYN_ERR_INVALID, "unknown activation");
    if (c.backward != 0 && c.backward != 1) return host_fail(SYN_ERR_INVALID, "backward must be 0 or 1");
    if (c.saved_f32 != 0 && c.saved_f32 != 1) return host_fail(SYN_ERR_INVALID, "saved_f32 must be 0 or 1");
    if (c.timeout_ns == 0) c.timeout_ns = host_timeout_ns();
    const int rc = host_load_driver();
    if (rc != SYN_OK) return rc;
    syn_ffn_plan_s *pl = new (std::nothrow) syn_ffn_plan_s();
    if (pl == nullptr) return host_fail(SYN_ERR_UNSUPPORTED, "not enough host memory");
    pl->cfg = c;
    pl->bf16 = c.dtype == SYN_DTYPE_BF16;
    pl->wide = c.saved_f32 == 1;
    int sms = 0;
    cudaError_t e = cudaGetDevice(&pl->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, pl->device);
    if (e == cudaSuccess) e = fwd_prepare(c.act);
    if (e == cudaSuccess && c.backward) e = bwd_prepare();
    if (e == cudaSuccess) e = cudaMalloc(&pl->d_err, 4 * sizeof(int32_t));
    if (e == cudaSuccess) e = cudaMemset(pl->d_err, 0, 4 * sizeof(int32_t));
    pl->pairs = sms / 2;
    if (e == cudaSuccess) e = cudaMalloc(&pl->parts.sums, (size_t)pl->pairs * kPartBytes / (c.backward ? 1 : 2));
    if (e == cudaSuccess) e = cudaMalloc(&pl->parts.arrived, (size_t)pl->pairs * kStrips * sizeof(uint32_t));
    if (e == cudaSuccess) e = cudaMemset(pl->parts.arrived, 0, (size_t)pl->pairs * kStrips * sizeof(uint32_t));
    // (the clearing may return before it has reached the device, which other streams would not wait for)
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) {
        syn_ffn_plan_destroy(pl);
        return host_fail(SYN_ERR_CUDA, std::string("ffn plan: ") + cudaGetErrorString(e));
    }
    *out = pl;
    return SYN_OK;
}

int syn_ffn_plan_destroy(syn_ffn_plan_t pl) {
    if (pl == nullptr) return SYN_OK;
    cudaFree(pl->d_err);
    cudaFree(pl->parts.sums);
    cudaFree(pl->parts.arrived);
    delete pl;
    return SYN_OK;
}

int syn_ffn_plan_parts(syn_ffn_plan_t pl, int64_t n_tokens, int want, int *forward, int *backward) {
    int rc = check_call(pl, n_tokens);
    if (rc != SYN_OK) return rc;
    if (want < 0 || want > 3) return host_fail(SYN_ERR_INVALID, "want must be 0 to 3");
    if (forward != nullptr) {
        const FwdTiles t = n_tokens == 0 ? FwdTiles{0, 0, 1, 1} : fwd_tiles(pl, n_tokens);
        if (t.n == 0) return host_fail(SYN_ERR_UNSUPPORTED, "2^30 or more tiles");
        *forward = t.split;
    }
    if (backward != nullptr) {
        int x[2] = {0, 0}, w[2] = {0, 0};
        if ((want & 1) != 0 && (rc = dx_tiles(pl, n_tokens, x[0], x[1])) != SYN_OK) return rc;
        if ((want & 2) != 0) dw_tiles(pl, w[0], w[1]);
        *backward = want == 0 || n_tokens == 0 || !pl->cfg.backward ? 1 : bwd_deal(pl, n_tokens, x[0] * x[1], w[0] * w[1]).split;
    }
    return SYN_OK;
}

int syn_gated_ffn(syn_ffn_plan_t pl, const syn_ffn_mat_t *X, const syn_ffn_mat_t *Wg, const syn_ffn_mat_t *Wu,
                  const syn_ffn_mat_t *H, const syn_ffn_mat_t *G, const syn_ffn_mat_t *U, int64_t n_tokens, void *stream) {
    int rc = check_call(pl, n_tokens);
    if (rc != SYN_OK) return rc;
    const syn_ffn_cfg_t &c = pl->cfg;
    if ((G == nullptr) != (U == nullptr)) return host_fail(SYN_ERR_INVALID, "G and U go together");
    const bool keep = G != nullptr;
    const int saved = pl->wide ? 4 : 8;
    const Mat mats[] = {{"X", X, n_tokens, c.d, false, true}, {"Wg", Wg, c.d, c.d_ff, false, true}, {"Wu", Wu, c.d, c.d_ff, false, true},
                        {"H", H, n_tokens, c.d_ff, true, true}, {"G", G, n_tokens, c.d_ff, true, keep, saved},
                        {"U", U, n_tokens, c.d_ff, true, keep, saved}};
    if ((rc = check_mats(mats, 6)) != SYN_OK) return rc;
    if (n_tokens == 0) return SYN_OK;
    FwdMaps m;
    const int x_rows = n_tokens < 64 ? (int)((n_tokens + 7) / 8 * 8) : 64;
    if ((rc = encode(&m.x, pl, *X, n_tokens, c.d, false, x_rows)) != SYN_OK || (rc = encode(&m.wg, pl, *Wg, c.d, c.d_ff, false)) != SYN_OK ||
        (rc = encode(&m.wu, pl, *Wu, c.d, c.d_ff, false)) != SYN_OK || (rc = encode(&m.h, pl, *H, n_tokens, c.d_ff, true)) != SYN_OK)
        return rc;
    m.g = m.u = m.h;
    if (G != nullptr)
        for (auto x : {std::make_pair(&m.g, G), std::make_pair(&m.u, U)})
            if ((rc = pl->wide ? encode_wide(x.first, *x.second, n_tokens, c.d_ff) : encode(x.first, pl, *x.second, n_tokens, c.d_ff, true)) != SYN_OK)
                return rc;
    FwdParams p;
    std::memset(&p, 0, sizeof(p));
    p.c = common_of(pl);
    p.m = (int32_t)n_tokens;
    p.k = c.d;
    p.f = c.d_ff;
    const FwdTiles t = fwd_tiles(pl, n_tokens);
    if (t.n == 0) return host_fail(SYN_ERR_UNSUPPORTED, "2^30 or more tiles");
    const int nt = t.width;
    p.tiles_m = t.m;
    p.tiles_n = t.n;
    p.band = band_of(pl->pairs, p.tiles_m);
    p.x_rows = x_rows;
    p.keep = G == nullptr ? 0 : pl->wide ? 2 : 1;
    p.bf16 = pl->bf16;
    p.split = t.split;
    p.parts = pl->parts;
    FFN_CK(fwd_launch(c.act, nt, std::min(pl->pairs, p.tiles_m * p.tiles_n * p.split), p, m, static_cast<cudaStream_t>(stream)));
    return SYN_OK;
}

int syn_gated_ffn_backward(syn_ffn_plan_t pl, const syn_ffn_mat_t *dH, const syn_ffn_mat_t *X, const syn_ffn_mat_t *Wg,
                           const syn_ffn_mat_t *Wu, const syn_ffn_mat_t *G, const syn_ffn_mat_t *U,
                           const syn_ffn_mat_t *dG, const syn_ffn_mat_t *dU, const syn_ffn_mat_t *dX,
                           const syn_ffn_mat_t *dWg, const syn_ffn_mat_t *dWu, int64_t n_tokens, void *stream) {
    int rc = check_call(pl, n_tokens);
    if (rc != SYN_OK) return rc;
    const syn_ffn_cfg_t &c = pl->cfg;
    if (!c.backward) return host_fail(SYN_ERR_INVALID, "the plan was made without backward");
    if ((dWg == nullptr) != (dWu == nullptr)) return host_fail(SYN_ERR_INVALID, "dWg and dWu go together");
    const bool dx = dX != nullptr, dw = dWg != nullptr;
    const int saved = pl->wide ? 4 : 8;
    const Mat mats[] = {{"dH", dH, n_tokens, c.d_ff, false, true, 8, true}, {"X", X, n_tokens, c.d, false, dw},
                        {"Wg", Wg, c.d, c.d_ff, false, dx}, {"Wu", Wu, c.d, c.d_ff, false, dx},
                        {"G", G, n_tokens, c.d_ff, false, true, saved, true}, {"U", U, n_tokens, c.d_ff, false, true, saved, true},
                        {"dG", dG, n_tokens, c.d_ff, true, true, 8, false, true}, {"dU", dU, n_tokens, c.d_ff, true, true, 8, false, true},
                        {"dX", dX, n_tokens, c.d, true, dx}, {"dWg", dWg, c.d, c.d_ff, true, dw}, {"dWu", dWu, c.d, c.d_ff, true, dw}};
    if ((rc = check_mats(mats, 11)) != SYN_OK) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (n_tokens == 0) {
        for (const syn_ffn_mat_t *w : {dWg, dWu})
            if (w != nullptr)
                FFN_CK(cudaMemset2DAsync(w->p, (size_t)(c.d > 1 ? w->row : c.d_ff) * 2, 0, (size_t)c.d_ff * 2, (size_t)c.d, st));
        return SYN_OK;
    }
    const int64_t vecs = n_tokens * (c.d_ff / 8);
    if (vecs >= (int64_t)1 << 31) return host_fail(SYN_ERR_UNSUPPORTED, "2^34 or more elements of dH in one call");
    BwdParams p;
    std::memset(&p, 0, sizeof(p));
    p.c = common_of(pl);
    p.m = (int32_t)n_tokens;
    p.k = c.d;
    p.f = c.d_ff;
    p.bf16 = pl->bf16;
    BwdMaps m;
    std::memset(&m, 0, sizeof(m));
    if ((rc = encode(&m.dg, pl, *dG, n_tokens, c.d_ff, false)) != SYN_OK || (rc = encode(&m.du, pl, *dU, n_tokens, c.d_ff, false)) != SYN_OK)
        return rc;
    if (dX != nullptr) {
        if ((rc = encode(&m.wg, pl, *Wg, c.d, c.d_ff, false)) != SYN_OK || (rc = encode(&m.wu, pl, *Wu, c.d, c.d_ff, false)) != SYN_OK ||
            (rc = encode(&m.dx, pl, *dX, n_tokens, c.d, true)) != SYN_OK)
            return rc;
        if ((rc = dx_tiles(pl, n_tokens, p.dx_m, p.dx_n)) != SYN_OK) return rc;
    }
    if (dWg != nullptr) {
        if ((rc = encode(&m.x, pl, *X, n_tokens, c.d, false)) != SYN_OK || (rc = encode(&m.dwg, pl, *dWg, c.d, c.d_ff, true)) != SYN_OK ||
            (rc = encode(&m.dwu, pl, *dWu, c.d, c.d_ff, true)) != SYN_OK)
            return rc;
        dw_tiles(pl, p.dw_m, p.dw_n);
    }
    ActParams a;
    std::memset(&a, 0, sizeof(a));
    a.dh = dH->p;
    a.g = G->p;
    a.u = U->p;
    a.dg = dG->p;
    a.du = dU->p;
    a.dh_row = n_tokens > 1 ? dH->row : 0;
    a.g_row = n_tokens > 1 ? G->row : 0;
    a.u_row = n_tokens > 1 ? U->row : 0;
    a.dg_row = n_tokens > 1 ? dG->row : 0;
    a.du_row = n_tokens > 1 ? dU->row : 0;
    a.n = (uint32_t)vecs;
    a.per_row = (uint32_t)(c.d_ff / 8);
    divisor(a.per_row, a.magic, a.shift);
    FFN_CK(act_grad_launch(c.act, pl->bf16, pl->wide, a, st));
    if (p.dx_m * p.dx_n + p.dw_m * p.dw_n == 0) return SYN_OK;
    const BwdDeal deal = bwd_deal(pl, n_tokens, p.dx_m * p.dx_n, p.dw_m * p.dw_n);
    const int n1 = deal.n1, n2 = deal.n2;
    p.dw_first = deal.dw_first;
    p.split = deal.split;
    p.items1 = n1 * p.split;
    p.tiles2 = n2;
    p.parts = pl->parts;
    const int pairs = std::min(pl->pairs, p.items1 + p.tiles2);
    p.even = even_rounds(pairs, p.items1, p.tiles2, deal.stages1 / p.split + kEnd, deal.stages2 + kEnd);
    p.rest = p.items1 % pairs;
    p.band = band_of(pairs, std::max(p.dx_m, p.dw_m));
    FFN_CK(bwd_launch(pairs, p, m, st));
    return SYN_OK;
}

int syn_ffn_sync_status(syn_ffn_plan_t pl, void *stream) {
    if (pl == nullptr) return host_fail(SYN_ERR_INVALID, "null plan");
    FFN_CK(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)));
    int32_t e[4] = {0, 0, 0, 0};
    FFN_CK(cudaMemcpy(e, pl->d_err, sizeof(e), cudaMemcpyDeviceToHost));
    if (e[0] == 0) return SYN_OK;
    // (parts that never arrived are counted anew)
    FFN_CK(cudaMemset(pl->parts.arrived, 0, (size_t)pl->pairs * kStrips * sizeof(uint32_t)));
    FFN_CK(cudaMemset(pl->d_err, 0, sizeof(e)));
    FFN_CK(cudaDeviceSynchronize());  // (cleared before a later call, of whatever stream, can report)
    return host_fail(e[0], std::string("device error ") + syn_status_string(e[0]) + " at site " + std::to_string(e[1]) +
                               " in CTA " + std::to_string(e[2]) + " (info " + std::to_string(e[3]) + ")");
}

}  // extern "C"
