// rope.cu -- rotary positions of query and key heads, alone or with a norm of
// each head in the same pass, and their gradients (C ABI: include/syn_rope.h).
//
// Every operator here reads each element of a head once and writes it once
// (the norm's gradient reads two), so HBM bounds it at long inputs and the
// launch at a token.  A head (row) belongs to a group of L lanes; a lane holds
// one slot of the row: 2 * VEC elements as two 16-byte vectors that contain
// both members of each of its VEC pairs, so that the turn needs no exchange
// between lanes and the norm's sum one shuffle tree over L lanes.  A group
// takes a unit of up to `rows` heads of one token, computes the unit's cosines
// and sines once into registers and walks the heads.
//
// The angle of position p and frequency f is p * f mod 2 pi.  f / 2 pi is kept
// as a 64-bit fraction of a turn; the 64-bit product with p drops whole turns
// exactly, and the upper 32 bits give the angle in half turns to sincospif.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <string>
#include <vector>

#include "host_util.h"
#include "syn.h"
#include "syn_rope.h"

namespace syn {
namespace rope {

constexpr int kThreads = 256;
constexpr int kMaxD = 256;
constexpr int kRows = 8;            // heads that share one computation of the angles
constexpr int kBlocksPerSm = 4;

struct Tensor {
    const void *x, *dy;  // dy: the gradient kernel only
    void *y;             // the gradient kernel: dx
    int64_t xt, xh, gt, gh, yt, yh;
    const void *w;
    int32_t heads, splits;
    int32_t copy, scatter, norm;
};

struct Args {
    Tensor t[3];
    int32_t n_tensors, rows, d, d_rot, interleaved;
    uint32_t n_tokens;
    const int64_t *pos, *slots;
    int64_t pos0, n_slots;
    const uint64_t *step;  // [d_rot / 2] turns per position, as 64-bit fractions
    float factor, sign, eps;
    float *partial;        // [grid][2][kMaxD] weight-gradient sums
};

template <typename T> struct Num;
template <> struct Num<__nv_bfloat16> {
    static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <> struct Num<__half> {
    static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
};
template <> struct Num<float> {
    static __device__ __forceinline__ float get(float v) { return v; }
    static __device__ __forceinline__ float put(float v) { return v; }
};

// VEC elements as they lie in memory
template <typename T, int VEC> struct alignas(sizeof(T) * VEC) Pack {
    T v[VEC];
};

// Where a lane's slots lie in a row.  Slot s of the rotated part holds VEC
// pairs with frequencies s * VEC ..: half layout, elements s * VEC .. and
// d_rot/2 + s * VEC ..; interleaved, 2 * VEC consecutive ones.  The slots after
// them hold 2 * VEC consecutive elements that pass through.
template <int VEC, int L, int NS> struct Slots {
    int o0[NS], o1[NS], f0[NS];
    bool rot[NS], has0[NS], has1[NS];
    __device__ __forceinline__ void init(const Args &a, bool copy, int sub) {
        const int d_rot = copy ? 0 : a.d_rot;
        const int n_rot = d_rot / (2 * VEC);
#pragma unroll
        for (int n = 0; n < NS; ++n) {
            const int s = sub + n * L;
            rot[n] = s < n_rot;
            f0[n] = s * VEC;
            if (rot[n]) {
                o0[n] = a.interleaved ? 2 * s * VEC : s * VEC;
                o1[n] = a.interleaved ? o0[n] + VEC : d_rot / 2 + s * VEC;
            } else {
                o0[n] = d_rot + 2 * (s - n_rot) * VEC;
                o1[n] = o0[n] + VEC;
            }
            has0[n] = o0[n] + VEC <= a.d;
            has1[n] = o1[n] + VEC <= a.d;
        }
    }
};

template <typename T, int VEC, int L, int NS>
__device__ __forceinline__ void load_row(Pack<T, VEC> (&raw)[NS][2], const T *row, const Slots<VEC, L, NS> &s) {
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        if (s.has0[n]) raw[n][0] = *reinterpret_cast<const Pack<T, VEC> *>(row + s.o0[n]);
        if (s.has1[n]) raw[n][1] = *reinterpret_cast<const Pack<T, VEC> *>(row + s.o1[n]);
    }
}

template <typename T, int VEC, int L, int NS>
__device__ __forceinline__ void widen(float (&e)[NS][2 * VEC], const Pack<T, VEC> (&raw)[NS][2],
                                      const Slots<VEC, L, NS> &s) {
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            e[n][i] = s.has0[n] ? Num<T>::get(raw[n][0].v[i]) : 0.f;
            e[n][VEC + i] = s.has1[n] ? Num<T>::get(raw[n][1].v[i]) : 0.f;
        }
}

template <typename T, int VEC, int L, int NS>
__device__ __forceinline__ void store_row(T *row, const float (&e)[NS][2 * VEC], const Slots<VEC, L, NS> &s) {
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        Pack<T, VEC> a, b;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            a.v[i] = Num<T>::put(e[n][i]);
            b.v[i] = Num<T>::put(e[n][VEC + i]);
        }
        if (s.has0[n]) *reinterpret_cast<Pack<T, VEC> *>(row + s.o0[n]) = a;
        if (s.has1[n]) *reinterpret_cast<Pack<T, VEC> *>(row + s.o1[n]) = b;
    }
}

// (cos, sin) of the unit's position for the lane's pairs, times the factor
template <int VEC, int L, int NS>
__device__ __forceinline__ void angles(float (&cs)[NS][VEC], float (&sn)[NS][VEC], const Args &a, int64_t pos,
                                       const Slots<VEC, L, NS> &s) {
#pragma unroll
    for (int n = 0; n < NS; ++n)
        if (s.rot[n]) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const uint64_t turn = (uint64_t)pos * a.step[s.f0[n] + i];
                const float half_turns = (float)(int32_t)(uint32_t)(turn >> 32) * 4.656612873077393e-10f;  // 2^-31
                float c, si;
                sincospif(half_turns, &si, &c);
                cs[n][i] = c * a.factor;
                sn[n][i] = si * a.factor * a.sign;
            }
        }
}

template <int VEC, int L, int NS>
__device__ __forceinline__ void turn(float (&e)[NS][2 * VEC], const float (&cs)[NS][VEC], const float (&sn)[NS][VEC],
                                     const Args &a, const Slots<VEC, L, NS> &s) {
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        if (!s.rot[n]) continue;
        if (a.interleaved) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float u = e[n][2 * i], v = e[n][2 * i + 1];
                e[n][2 * i] = u * cs[n][i] - v * sn[n][i];
                e[n][2 * i + 1] = u * sn[n][i] + v * cs[n][i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float u = e[n][i], v = e[n][VEC + i];
                e[n][i] = u * cs[n][i] - v * sn[n][i];
                e[n][VEC + i] = u * sn[n][i] + v * cs[n][i];
            }
        }
    }
}

// sum over the group's L lanes, in every lane
template <int L> __device__ __forceinline__ float group_sum(float v, uint32_t mask) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o);
    return v;
}

template <typename T, int VEC, int L, int NS>
__device__ __forceinline__ void load_weight(float (&w)[NS][2 * VEC], const Tensor &x, const Slots<VEC, L, NS> &s) {
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            w[n][i] = x.w != nullptr && s.has0[n] ? Num<T>::get(static_cast<const T *>(x.w)[s.o0[n] + i]) : 1.f;
            w[n][VEC + i] = x.w != nullptr && s.has1[n] ? Num<T>::get(static_cast<const T *>(x.w)[s.o1[n] + i]) : 1.f;
        }
}

// The forward of both operators (and, with sign -1, the gradient of the rotation).
template <typename T, int VEC, int L, int NS, bool NORM>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ Args a) {
    constexpr int U = VEC == 1 ? 1 : 2;  // rows whose loads are in flight together
    const int sub = (int)threadIdx.x % L;
    const uint32_t mask = L == 32 ? 0xffffffffu : ((1u << L) - 1u) << ((threadIdx.x & 31u) & ~(uint32_t)(L - 1));
    uint32_t total = 0;
    for (int x = 0; x < a.n_tensors; ++x) total += a.n_tokens * (uint32_t)a.t[x].splits;
    const uint32_t groups = gridDim.x * (kThreads / L);
    for (uint32_t u = blockIdx.x * (kThreads / L) + threadIdx.x / L; u < total; u += groups) {
        uint32_t v = u;
        int x = 0;
        while (v >= a.n_tokens * (uint32_t)a.t[x].splits) v -= a.n_tokens * (uint32_t)a.t[x++].splits;
        const Tensor &t = a.t[x];
        const uint32_t tok = v / (uint32_t)t.splits;
        const int h0 = (int)(v - tok * (uint32_t)t.splits) * a.rows;
        const int h1 = min(h0 + a.rows, t.heads);
        int64_t to = tok;
        if (t.scatter) {
            to = a.slots[tok];
            if (to < 0 || to >= a.n_slots) continue;
        }
        Slots<VEC, L, NS> s;
        s.init(a, t.copy != 0, sub);
        float cs[NS][VEC], sn[NS][VEC], w[NS][2 * VEC];
        angles(cs, sn, a, a.pos != nullptr ? a.pos[tok] : a.pos0 + (int64_t)tok, s);
        if (NORM && t.norm) load_weight<T>(w, t, s);
        const T *src = static_cast<const T *>(t.x) + (int64_t)tok * t.xt;
        T *dst = static_cast<T *>(t.y) + to * t.yt;
        for (int h = h0; h < h1; h += U) {
            Pack<T, VEC> raw[U][NS][2];
#pragma unroll
            for (int r = 0; r < U; ++r)
                if (h + r < h1) load_row(raw[r], src + (h + r) * t.xh, s);
#pragma unroll
            for (int r = 0; r < U; ++r) {
                if (h + r >= h1) break;
                float e[NS][2 * VEC];
                widen(e, raw[r], s);
                if (NORM && t.norm) {
                    float q = 0.f;
#pragma unroll
                    for (int n = 0; n < NS; ++n)
#pragma unroll
                        for (int i = 0; i < 2 * VEC; ++i) q = fmaf(e[n][i], e[n][i], q);
                    const float inv = rsqrtf(group_sum<L>(q, mask) / (float)a.d + a.eps);
#pragma unroll
                    for (int n = 0; n < NS; ++n)
#pragma unroll
                        for (int i = 0; i < 2 * VEC; ++i) e[n][i] *= inv * w[n][i];
                }
                turn(e, cs, sn, a, s);
                store_row(dst + (h + r) * t.yh, e, s);
            }
        }
    }
}

// The gradient of norm and rotation.  With g = R^T dy, r = rsqrt(mean x^2 + eps):
// dx = r (g w - x r mean(g w x r)), dw = sum over rows of g x r.  A lane sums
// its elements' dw over all its rows in registers, a block its groups' sums in
// shared memory, and norm_dw_kernel the blocks' -- each in a fixed order.
template <typename T, int VEC, int L, int NS>
__global__ void __launch_bounds__(kThreads) norm_grad_kernel(const __grid_constant__ Args a) {
    constexpr int G = kThreads / L;
    __shared__ float sums[kThreads * NS * 2 * VEC];  // [group][element]
    const int sub = (int)threadIdx.x % L, grp = (int)threadIdx.x / L;
    const uint32_t mask = L == 32 ? 0xffffffffu : ((1u << L) - 1u) << ((threadIdx.x & 31u) & ~(uint32_t)(L - 1));
    const uint32_t groups = gridDim.x * G;
    Slots<VEC, L, NS> s;
    s.init(a, false, sub);
    for (int x = 0; x < a.n_tensors; ++x) {
        const Tensor &t = a.t[x];
        float w[NS][2 * VEC], acc[NS][2 * VEC];
        load_weight<T>(w, t, s);
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < 2 * VEC; ++i) acc[n][i] = 0.f;
        const uint32_t units = a.n_tokens * (uint32_t)t.splits;
        for (uint32_t u = blockIdx.x * G + grp; u < units; u += groups) {
            const uint32_t tok = u / (uint32_t)t.splits;
            const int h0 = (int)(u - tok * (uint32_t)t.splits) * a.rows;
            const int h1 = min(h0 + a.rows, t.heads);
            float cs[NS][VEC], sn[NS][VEC];
            angles(cs, sn, a, a.pos != nullptr ? a.pos[tok] : a.pos0 + (int64_t)tok, s);
            const T *src = static_cast<const T *>(t.x) + (int64_t)tok * t.xt;
            const T *grd = static_cast<const T *>(t.dy) + (int64_t)tok * t.gt;
            T *dst = static_cast<T *>(t.y) + (int64_t)tok * t.yt;
            for (int h = h0; h < h1; ++h) {
                Pack<T, VEC> rx[NS][2], rg[NS][2];
                load_row(rx, src + h * t.xh, s);
                load_row(rg, grd + h * t.gh, s);
                float e[NS][2 * VEC], g[NS][2 * VEC];
                widen(e, rx, s);
                widen(g, rg, s);
                turn(g, cs, sn, a, s);
                float q = 0.f, m = 0.f;  // sums of x^2 and of g w x
#pragma unroll
                for (int n = 0; n < NS; ++n)
#pragma unroll
                    for (int i = 0; i < 2 * VEC; ++i) {
                        q = fmaf(e[n][i], e[n][i], q);
                        m = fmaf(g[n][i] * w[n][i], e[n][i], m);
                    }
                const float inv = rsqrtf(group_sum<L>(q, mask) / (float)a.d + a.eps);
                const float mean = group_sum<L>(m, mask) * inv / (float)a.d;
#pragma unroll
                for (int n = 0; n < NS; ++n)
#pragma unroll
                    for (int i = 0; i < 2 * VEC; ++i) {
                        const float xh = e[n][i] * inv;
                        acc[n][i] = fmaf(g[n][i], xh, acc[n][i]);
                        e[n][i] = inv * (g[n][i] * w[n][i] - xh * mean);
                    }
                store_row(dst + h * t.yh, e, s);
            }
        }
        __syncthreads();  // the previous tensor's sums have been read
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                if (s.has0[n]) sums[grp * a.d + s.o0[n] + i] = acc[n][i];
                if (s.has1[n]) sums[grp * a.d + s.o1[n] + i] = acc[n][VEC + i];
            }
        __syncthreads();
        for (int j = (int)threadIdx.x; j < a.d; j += kThreads) {
            float v = 0.f;
            for (int k = 0; k < G; ++k) v += sums[k * a.d + j];
            a.partial[((int64_t)blockIdx.x * 2 + x) * kMaxD + j] = v;
        }
    }
}

// dw[j] of tensor blockIdx.y: the blocks' partial sums, 32 interleaved chains
// joined in a fixed order.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float *partial, int n, int d, float *dw0, float *dw1) {
    __shared__ float sums[32][33];
    const int j = (int)(blockIdx.x * 32 + threadIdx.x);
    float *dw = blockIdx.y == 0 ? dw0 : dw1;
    if (dw == nullptr) return;
    float v = 0.f;
    if (j < d)
        for (int k = (int)threadIdx.y; k < n; k += 32) v += partial[((int64_t)k * 2 + blockIdx.y) * kMaxD + j];
    sums[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y == 0 && j < d) {
        v = 0.f;
        for (int k = 0; k < 32; ++k) v += sums[k][threadIdx.x];
        dw[j] = v;
    }
}

}  // namespace rope
}  // namespace syn

using namespace syn;
using namespace syn::rope;

struct syn_rope_plan_s {
    syn_rope_cfg_t cfg;
    int device = 0, num_sms = 0;
    double factor = 1.0;
    std::vector<double> f;
    uint64_t *d_step = nullptr;
    float *d_partial = nullptr;
};

namespace {

#define ROPE_CK(call)                                                                                 \
    do {                                                                                              \
        cudaError_t e__ = (call);                                                                     \
        if (e__ != cudaSuccess) return host_fail(SYN_ERR_CUDA, std::string(#call) + ": " + cudaGetErrorString(e__)); \
    } while (0)

constexpr double kPi = 3.14159265358979323846;

// f_i in radians per position and the factor on the rotated elements
void frequencies(const syn_rope_cfg_t &c, std::vector<double> &f, double &factor) {
    const int n = c.d_rot / 2;
    double base = c.base;
    if (c.scaling == SYN_ROPE_SCALE_NTK) base *= std::pow(c.factor, (double)c.d_rot / (double)(c.d_rot - 2));
    f.resize((size_t)n);
    double lo = 0, hi = 0;
    if (c.scaling == SYN_ROPE_SCALE_YARN) {
        auto index = [&](double turns) {
            return c.d_rot * std::log(c.original_context / (2 * kPi * turns)) / (2 * std::log(c.base));
        };
        lo = std::max(std::floor(index(c.beta_fast)), 0.0);
        hi = std::min(std::ceil(index(c.beta_slow)), (double)(c.d_rot - 1));
    }
    for (int i = 0; i < n; ++i) {
        double v = std::pow(base, -2.0 * i / c.d_rot);
        if (c.scaling == SYN_ROPE_SCALE_LINEAR) {
            v /= c.factor;
        } else if (c.scaling == SYN_ROPE_SCALE_LLAMA3) {
            double t = (c.original_context * v / (2 * kPi) - c.low_freq_factor) / (c.high_freq_factor - c.low_freq_factor);
            t = std::min(std::max(t, 0.0), 1.0);
            v = (1 - t) * v / c.factor + t * v;
        } else if (c.scaling == SYN_ROPE_SCALE_YARN) {
            const double r = std::min(std::max((i - lo) / std::max(hi - lo, 1e-3), 0.0), 1.0);
            v = v / c.factor * r + v * (1 - r);
        }
        f[(size_t)i] = v;
    }
    factor = c.attn_factor != 0 ? c.attn_factor
             : c.scaling == SYN_ROPE_SCALE_YARN ? 0.1 * std::log(c.factor) + 1.0 : 1.0;
}

int elem_size(int dtype) { return dtype == SYN_DTYPE_F32 ? 4 : 2; }

// Whether rows at `p` with these strides can be read and written as 16-byte vectors
bool vector_rows(const void *p, int64_t token, int64_t head, int size) {
    const int vec = 16 / size;
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && token % vec == 0 && head % vec == 0;
}

int check_rows(const char *name, const void *p, int size, int heads, bool any) {
    if (heads < 0) return host_fail(SYN_ERR_INVALID, std::string(name) + ": negative head count");
    if (heads > 0 && any && p == nullptr) return host_fail(SYN_ERR_INVALID, std::string(name) + ": null operand");
    if (reinterpret_cast<uintptr_t>(p) % (uintptr_t)size != 0)
        return host_fail(SYN_ERR_INVALID, std::string(name) + ": operand not aligned to its element");
    return SYN_OK;
}

// Units of up to a.rows heads of one token: few heads while that is what fills
// the SMs (the angles are computed again for each unit), up to kRows after.
void split_rows(Args &a, int num_sms, int lanes) {
    int64_t rows = 0;
    for (int x = 0; x < a.n_tensors; ++x) rows += (int64_t)a.n_tokens * a.t[x].heads;
    const int64_t fill = (int64_t)num_sms * 1024 / lanes;
    a.rows = (int32_t)std::min<int64_t>(kRows, std::max<int64_t>(1, rows / fill));
    for (int x = 0; x < a.n_tensors; ++x) a.t[x].splits = (a.t[x].heads + a.rows - 1) / a.rows;
}

int64_t units_of(const Args &a) {
    int64_t n = 0;
    for (int x = 0; x < a.n_tensors; ++x) n += (int64_t)a.n_tokens * a.t[x].splits;
    return n;
}

enum Kind { kTurn, kNorm, kNormGrad };

template <typename T, int VEC, int L, int NS> int launch(syn_rope_plan_s *pl, Args &a, Kind kind, cudaStream_t st, int &grid) {
    split_rows(a, pl->num_sms, L);
    const int64_t units = units_of(a);
    grid = (int)std::min<int64_t>((units + kThreads / L - 1) / (kThreads / L), (int64_t)pl->num_sms * kBlocksPerSm);
    if (kind == kTurn) rope_kernel<T, VEC, L, NS, false><<<grid, kThreads, 0, st>>>(a);
    else if (kind == kNorm) rope_kernel<T, VEC, L, NS, true><<<grid, kThreads, 0, st>>>(a);
    else norm_grad_kernel<T, VEC, L, NS><<<grid, kThreads, 0, st>>>(a);
    ROPE_CK(cudaGetLastError());
    return SYN_OK;
}

// A lane's slot is two 16-byte vectors where every row, stride and both parts
// of the head allow it, else single elements.
template <typename T> int dispatch(syn_rope_plan_s *pl, Args &a, Kind kind, bool vec, cudaStream_t st, int &grid) {
    constexpr int V = 16 / (int)sizeof(T);
    if (!vec) return launch<T, 1, 32, 4>(pl, a, kind, st, grid);
    const int slots = a.d / (2 * V);
    if (slots <= 4) return launch<T, V, 4, 1>(pl, a, kind, st, grid);
    if (slots <= 8) return launch<T, V, 8, 1>(pl, a, kind, st, grid);
    if (slots <= 16) return launch<T, V, 16, 1>(pl, a, kind, st, grid);
    return launch<T, V, 32, 1>(pl, a, kind, st, grid);
}

int run(syn_rope_plan_s *pl, Args &a, Kind kind, cudaStream_t st, int &grid) {
    const syn_rope_cfg_t &c = pl->cfg;
    grid = 0;
    a.d = c.d;
    a.d_rot = c.d_rot;
    a.interleaved = c.layout == SYN_ROPE_INTERLEAVED;
    a.step = pl->d_step;
    a.factor = (float)pl->factor;
    a.partial = pl->d_partial;
    const int size = elem_size(c.dtype);
    bool vec = c.d % (32 / size) == 0 && c.d_rot % (32 / size) == 0;
    int64_t rows = 0;
    for (int x = 0; x < a.n_tensors; ++x) {
        const Tensor &t = a.t[x];
        vec = vec && vector_rows(t.x, t.xt, t.xh, size) && vector_rows(t.y, t.yt, t.yh, size) &&
              (t.dy == nullptr || vector_rows(t.dy, t.gt, t.gh, size));
        rows += (int64_t)a.n_tokens * t.heads;
    }
    if (rows == 0) return SYN_OK;
    if (rows >= (int64_t)1 << 31) return host_fail(SYN_ERR_UNSUPPORTED, "2^31 or more rows in one call");
    if (c.dtype == SYN_DTYPE_BF16) return dispatch<__nv_bfloat16>(pl, a, kind, vec, st, grid);
    if (c.dtype == SYN_DTYPE_F16) return dispatch<__half>(pl, a, kind, vec, st, grid);
    return dispatch<float>(pl, a, kind, vec, st, grid);
}

int add(Args &a, const char *name, const syn_rope_rows_t *r, const void *w, int size, bool copy, bool scatter, bool norm) {
    if (r == nullptr) return SYN_OK;
    int rc;
    if ((rc = check_rows(name, r->x, size, r->heads, a.n_tokens > 0)) != SYN_OK || (rc = check_rows(name, r->y, size, r->heads, a.n_tokens > 0)) != SYN_OK ||
        (rc = check_rows(name, w, size, 0, false)) != SYN_OK)
        return rc;
    if (r->heads == 0) return SYN_OK;
    Tensor &t = a.t[a.n_tensors++];
    std::memset(&t, 0, sizeof(t));
    t.x = r->x;
    t.y = r->y;
    t.xt = r->x_token;
    t.xh = r->x_head;
    t.yt = r->y_token;
    t.yh = r->y_head;
    t.w = w;
    t.heads = r->heads;
    t.copy = copy;
    t.scatter = scatter;
    t.norm = norm;
    return SYN_OK;
}

int begin(syn_rope_plan_s *pl, Args &a, const int64_t *positions, int64_t pos0, int64_t n_tokens) {
    if (pl == nullptr) return host_fail(SYN_ERR_INVALID, "null plan");
    if (n_tokens < 0) return host_fail(SYN_ERR_INVALID, "negative token count");
    if (n_tokens >= (int64_t)1 << 31) return host_fail(SYN_ERR_UNSUPPORTED, "2^31 or more tokens in one call");
    std::memset(&a, 0, sizeof(a));
    a.pos = positions;
    a.pos0 = pos0;
    a.n_tokens = (uint32_t)n_tokens;
    a.sign = 1.f;
    return SYN_OK;
}

int forward(syn_rope_plan_s *pl, Kind kind, const syn_rope_rows_t *q, const void *wq, const syn_rope_rows_t *k,
            const void *wk, float eps, const syn_rope_rows_t *v, const int64_t *positions, int64_t pos0,
            const int64_t *slots, int64_t n_slots, int64_t n_tokens, void *stream) {
    Args a;
    int rc = begin(pl, a, positions, pos0, n_tokens);
    if (rc != SYN_OK) return rc;
    if (slots != nullptr && n_slots < 0) return host_fail(SYN_ERR_INVALID, "negative slot count");
    if (!(eps >= 0.f) || !std::isfinite(eps)) return host_fail(SYN_ERR_INVALID, "eps must be finite and not negative");
    const int size = elem_size(pl->cfg.dtype);
    const bool norm = kind == kNorm, scatter = slots != nullptr;
    if ((rc = add(a, "q", q, wq, size, false, false, norm)) != SYN_OK ||
        (rc = add(a, "k", k, wk, size, false, scatter, norm)) != SYN_OK ||
        (rc = add(a, "v", v, nullptr, size, true, scatter, false)) != SYN_OK)
        return rc;
    a.slots = slots;
    a.n_slots = n_slots;
    a.eps = eps;
    int grid;
    return run(pl, a, kind, static_cast<cudaStream_t>(stream), grid);
}

}  // namespace

extern "C" {

int syn_rope_cfg_default(syn_rope_cfg_t *c) {
    if (c == nullptr) return host_fail(SYN_ERR_INVALID, "null cfg");
    std::memset(c, 0, sizeof(*c));
    c->dtype = SYN_DTYPE_BF16;
    c->d = c->d_rot = 128;
    c->layout = SYN_ROPE_HALF;
    c->base = 10000.0;
    c->scaling = SYN_ROPE_SCALE_NONE;
    c->factor = 1.0;
    c->low_freq_factor = 1.0;
    c->high_freq_factor = 4.0;
    c->original_context = 8192.0;
    c->beta_fast = 32.0;
    c->beta_slow = 1.0;
    return SYN_OK;
}

int syn_rope_plan_create(syn_rope_plan_t *out, const syn_rope_cfg_t *cfg) {
    if (out == nullptr || cfg == nullptr) return host_fail(SYN_ERR_INVALID, "null argument");
    *out = nullptr;
    const syn_rope_cfg_t &c = *cfg;
    if (c.dtype < SYN_DTYPE_BF16 || c.dtype > SYN_DTYPE_F32) return host_fail(SYN_ERR_INVALID, "unknown dtype");
    if (c.d < 1) return host_fail(SYN_ERR_INVALID, "d must be positive");
    if (c.d > kMaxD) return host_fail(SYN_ERR_UNSUPPORTED, "d > 256");
    if (c.d_rot < 0 || c.d_rot > c.d || c.d_rot % 2 != 0) return host_fail(SYN_ERR_INVALID, "d_rot must be even and in [0, d]");
    if (c.layout != SYN_ROPE_HALF && c.layout != SYN_ROPE_INTERLEAVED) return host_fail(SYN_ERR_INVALID, "unknown layout");
    if (!(c.base > 1.0) || !std::isfinite(c.base)) return host_fail(SYN_ERR_INVALID, "base must be above 1");
    if (c.scaling < SYN_ROPE_SCALE_NONE || c.scaling > SYN_ROPE_SCALE_YARN) return host_fail(SYN_ERR_INVALID, "unknown scaling");
    if (c.scaling != SYN_ROPE_SCALE_NONE && (!(c.factor >= 1.0) || !std::isfinite(c.factor)))
        return host_fail(SYN_ERR_INVALID, "factor must be at least 1");
    if (c.scaling == SYN_ROPE_SCALE_NTK && c.d_rot < 4) return host_fail(SYN_ERR_INVALID, "NTK scaling needs d_rot >= 4");
    if ((c.scaling == SYN_ROPE_SCALE_LLAMA3 || c.scaling == SYN_ROPE_SCALE_YARN) &&
        (!(c.original_context > 0) || !std::isfinite(c.original_context)))
        return host_fail(SYN_ERR_INVALID, "original_context must be positive");
    if (c.scaling == SYN_ROPE_SCALE_LLAMA3 &&
        !(c.low_freq_factor > 0 && c.high_freq_factor > c.low_freq_factor && std::isfinite(c.high_freq_factor)))
        return host_fail(SYN_ERR_INVALID, "need 0 < low_freq_factor < high_freq_factor");
    if (c.scaling == SYN_ROPE_SCALE_YARN && !(c.beta_slow > 0 && c.beta_fast > c.beta_slow && std::isfinite(c.beta_fast)))
        return host_fail(SYN_ERR_INVALID, "need 0 < beta_slow < beta_fast");
    if (!(c.attn_factor >= 0) || !std::isfinite(c.attn_factor)) return host_fail(SYN_ERR_INVALID, "bad attn_factor");
    syn_rope_plan_s *pl = new syn_rope_plan_s();
    pl->cfg = c;
    frequencies(c, pl->f, pl->factor);
    std::vector<uint64_t> step(pl->f.size());
    for (size_t i = 0; i < step.size(); ++i) step[i] = (uint64_t)std::ldexp(pl->f[i] / (2 * kPi), 64);
    cudaError_t e = cudaGetDevice(&pl->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&pl->num_sms, cudaDevAttrMultiProcessorCount, pl->device);
    if (e == cudaSuccess) e = cudaMalloc(&pl->d_step, std::max<size_t>(step.size(), 1) * sizeof(uint64_t));
    if (e == cudaSuccess)
        e = cudaMalloc(&pl->d_partial, (size_t)pl->num_sms * kBlocksPerSm * 2 * kMaxD * sizeof(float));
    if (e == cudaSuccess && !step.empty())
        e = cudaMemcpy(pl->d_step, step.data(), step.size() * sizeof(uint64_t), cudaMemcpyHostToDevice);
    if (e != cudaSuccess) {
        syn_rope_plan_destroy(pl);
        return host_fail(SYN_ERR_CUDA, std::string("rope plan: ") + cudaGetErrorString(e));
    }
    *out = pl;
    return SYN_OK;
}

int syn_rope_plan_destroy(syn_rope_plan_t pl) {
    if (pl == nullptr) return SYN_OK;
    cudaFree(pl->d_step);
    cudaFree(pl->d_partial);
    delete pl;
    return SYN_OK;
}

int syn_rope_plan_frequencies(syn_rope_plan_t pl, double *f, double *attn_factor) {
    if (pl == nullptr) return host_fail(SYN_ERR_INVALID, "null plan");
    if (f != nullptr) std::copy(pl->f.begin(), pl->f.end(), f);
    if (attn_factor != nullptr) *attn_factor = pl->factor;
    return SYN_OK;
}

int syn_rope(syn_rope_plan_t pl, const syn_rope_rows_t *q, const syn_rope_rows_t *k, const syn_rope_rows_t *v,
             const int64_t *positions, int64_t pos0, const int64_t *slots, int64_t n_slots, int64_t n_tokens,
             void *stream) {
    return forward(pl, kTurn, q, nullptr, k, nullptr, 0.f, v, positions, pos0, slots, n_slots, n_tokens, stream);
}

int syn_qk_norm_rope(syn_rope_plan_t pl, const syn_rope_rows_t *q, const void *wq, const syn_rope_rows_t *k,
                     const void *wk, float eps, const syn_rope_rows_t *v, const int64_t *positions, int64_t pos0,
                     const int64_t *slots, int64_t n_slots, int64_t n_tokens, void *stream) {
    return forward(pl, kNorm, q, wq, k, wk, eps, v, positions, pos0, slots, n_slots, n_tokens, stream);
}

int syn_rope_backward(syn_rope_plan_t pl, const syn_rope_rows_t *dq, const syn_rope_rows_t *dk,
                      const int64_t *positions, int64_t pos0, int64_t n_tokens, void *stream) {
    Args a;
    int rc = begin(pl, a, positions, pos0, n_tokens);
    if (rc != SYN_OK) return rc;
    const int size = elem_size(pl->cfg.dtype);
    if ((rc = add(a, "dq", dq, nullptr, size, false, false, false)) != SYN_OK ||
        (rc = add(a, "dk", dk, nullptr, size, false, false, false)) != SYN_OK)
        return rc;
    a.sign = -1.f;
    int grid;
    return run(pl, a, kTurn, static_cast<cudaStream_t>(stream), grid);
}

int syn_qk_norm_rope_backward(syn_rope_plan_t pl, const syn_rope_grad_t *q, const syn_rope_grad_t *k, float eps,
                              const int64_t *positions, int64_t pos0, int64_t n_tokens, void *stream) {
    Args a;
    int rc = begin(pl, a, positions, pos0, n_tokens);
    if (rc != SYN_OK) return rc;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return host_fail(SYN_ERR_INVALID, "eps must be finite and not negative");
    const int size = elem_size(pl->cfg.dtype);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    float *dw[2] = {nullptr, nullptr};
    float *empty[2] = {nullptr, nullptr};  // gradients of weights without any row
    int x = 0;
    for (const syn_rope_grad_t *g : {q, k}) {
        const char *name = x++ == 0 ? "q" : "k";
        if (g == nullptr) continue;
        if ((rc = check_rows(name, g->x, size, g->heads, n_tokens > 0)) != SYN_OK || (rc = check_rows(name, g->dy, size, g->heads, n_tokens > 0)) != SYN_OK ||
            (rc = check_rows(name, g->dx, size, g->heads, n_tokens > 0)) != SYN_OK || (rc = check_rows(name, g->w, size, 0, false)) != SYN_OK ||
            (rc = check_rows(name, g->dw, 4, 0, false)) != SYN_OK)
            return rc;
        if (g->heads == 0 || n_tokens == 0) {
            empty[x - 1] = g->dw;
            continue;
        }
        dw[a.n_tensors] = g->dw;
        Tensor &t = a.t[a.n_tensors++];
        t.x = g->x;
        t.xt = g->x_token;
        t.xh = g->x_head;
        t.dy = g->dy;
        t.gt = g->dy_token;
        t.gh = g->dy_head;
        t.y = g->dx;
        t.yt = g->dx_token;
        t.yh = g->dx_head;
        t.w = g->w;
        t.heads = g->heads;
        t.norm = 1;
    }
    for (float *p : empty)
        if (p != nullptr) ROPE_CK(cudaMemsetAsync(p, 0, (size_t)pl->cfg.d * sizeof(float), st));
    a.sign = -1.f;
    a.eps = eps;
    int grid = 0;
    rc = run(pl, a, kNormGrad, st, grid);
    if (rc != SYN_OK || a.n_tensors == 0 || (dw[0] == nullptr && dw[1] == nullptr)) return rc;
    norm_dw_kernel<<<dim3((unsigned)(pl->cfg.d + 31) / 32, (unsigned)a.n_tensors), dim3(32, 32), 0, st>>>(
        pl->d_partial, grid, pl->cfg.d, dw[0], dw[1]);
    ROPE_CK(cudaGetLastError());
    return SYN_OK;
}

}  // extern "C"
