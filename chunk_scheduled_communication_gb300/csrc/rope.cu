// rope.cu -- rotary positions of query and key heads, alone or with a norm of
// each head in the same pass, and their gradients (C ABI: include/syn_rope.h).
//
// Every operator here reads each element of a head once and writes it once
// (the norm's gradient reads two), so HBM bounds it at long inputs and the
// launch at a token.  A head (row) belongs to a group of L lanes; a lane holds
// one slot of the row: 2 * VEC elements as two 16-byte vectors that contain
// both members of each of its VEC pairs, so that the turn needs no exchange
// between lanes and the norm's sum one shuffle tree over L lanes.  A block
// takes a few tokens with all their heads, of all tensors as one run of rows
// (tensor by tensor the keys' few rows were a pass of their own: the gradient
// of 5003 tokens 16.5 against 14.5 us): its threads issue the loads of their
// first rows, compute the tokens' cosines and sines into shared memory while
// these are under way, and then walk the rows.
//
// Measured on one GB300 (bf16, heads of 128; back-to-back calls): the rotation of
// 32768 tokens x 40 heads 98.2 us, 6.8 TB/s, the measured copy rate;
// with the norm, 16384 tokens 57.6 us, 5.8 TB/s (0.86: 310 instructions for a
// warp's four rows fill two thirds of the issue slots); its gradient 91.3 us,
// 5.5 TB/s (0.81: 125 registers, 16 warps an SM).  A call on a few tokens takes
// 2.4-3.0 us in a graph and 6.6-9.0 us with its host side.
//
// The angle of position p and frequency f is p * f mod 2 pi.  f / 2 pi is kept
// as a 64-bit fraction of a turn; the 64-bit product with p drops whole turns
// exactly, and the upper 32 bits give the angle in half turns to sincospif.  What
// remains is the rounding of f / 2 pi to 53 bits, about 3e-16 p f radians, and
// that of the angle to fp32, about 1e-7.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <string>
#include <vector>

#include "host_util.h"
#include "syn.h"
#include "syn_rope.h"
#include "window.cuh"

namespace syn {
namespace rope {

constexpr int kThreads = 256;
constexpr int kMaxD = 256;
constexpr int kNormPasses = 5;      // passes of a block with the norm at most
constexpr int kNormBlocksPerSm = 4;
constexpr int kRowsPerLane = 4;     // rows whose loads a lane has under way at long inputs
constexpr int kGradRowsPerLane = 3; // (gradient: of the step ahead)
constexpr int kGradThreads = 128;
constexpr int kGradBlocksPerSm = 4; // persistent blocks of the gradient kernel
constexpr int kTableBytes = 12 * 1024;  // cosines and sines of a block's tokens at most

struct Tensor {
    const void *x, *dy;  // dy: the gradient kernel only
    void *y;             // the gradient kernel: dx
    int64_t xt, xh, gt, gh, yt, yh;
    const void *w;
    int32_t heads;
    uint32_t magic, shift;  // r / heads = r * magic >> shift
    int32_t copy, scatter, norm;
};

struct Args {
    Tensor t[3];
    int32_t n_tensors, d, d_rot, interleaved;
    uint32_t n_tokens;
    uint32_t heads, magic, shift;  // of all tensors together; as Tensor::magic (forward)
    uint32_t tokens_of;    // tokens of a block (forward)
    uint32_t table_tokens; // tokens that half of the table of angles holds (gradient), at least 2
    const int64_t *pos, *slots;
    int64_t pos0, n_slots;
    const uint64_t *step;  // [d_rot / 2] turns per position, as 64-bit fractions
    float factor, sign, eps, inv_d;
    float *partial;        // [grid][2][kMaxD] weight-gradient sums (nullptr: not wanted)
};

template <typename T> struct Num;
template <> struct Num<__nv_bfloat16> {
    static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
    static __device__ __forceinline__ void get2(uint32_t w, float &a, float &b) {
        a = __uint_as_float(w << 16);
        b = __uint_as_float(w & 0xffff0000u);
    }
    static __device__ __forceinline__ uint32_t put2(float a, float b) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};
template <> struct Num<__half> {
    static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
    static __device__ __forceinline__ void get2(uint32_t w, float &a, float &b) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        a = v.x;
        b = v.y;
    }
    static __device__ __forceinline__ uint32_t put2(float a, float b) {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};
template <> struct Num<float> {
    static __device__ __forceinline__ float get(float v) { return v; }
    static __device__ __forceinline__ float put(float v) { return v; }
};

// VEC elements as they lie in memory: 16 bytes, or one element
template <typename T, int VEC> struct Pack {
    uint4 v;
    __device__ __forceinline__ void load(const T *p) { v = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<uint4 *>(p) = v; }
    __device__ __forceinline__ void widen(float *e) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 2) Num<T>::get2(w[i], e[2 * i], e[2 * i + 1]);
            else e[i] = __uint_as_float(w[i]);
        }
    }
    __device__ __forceinline__ void narrow(const float *e) {
        if constexpr (sizeof(T) == 2)
            v = make_uint4(Num<T>::put2(e[0], e[1]), Num<T>::put2(e[2], e[3]), Num<T>::put2(e[4], e[5]),
                           Num<T>::put2(e[6], e[7]));
        else
            v = make_uint4(__float_as_uint(e[0]), __float_as_uint(e[1]), __float_as_uint(e[2]), __float_as_uint(e[3]));
    }
};
template <typename T> struct Pack<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T *p) { v = *p; }
    __device__ __forceinline__ void store(T *p) const { *p = v; }
    __device__ __forceinline__ void widen(float *e) const { *e = Num<T>::get(v); }
    __device__ __forceinline__ void narrow(const float *e) { v = Num<T>::put(*e); }
};

// Where a lane's slots lie in a row.  Slot s of the rotated part holds VEC
// pairs with frequencies s * VEC ..: half layout, elements s * VEC .. and
// d_rot/2 + s * VEC ..; interleaved, 2 * VEC consecutive ones.  The slots after
// them hold 2 * VEC consecutive elements that pass through.
template <int VEC, int L, int NS> struct Slots {
    int o0[NS], o1[NS], f0[NS];
    bool rot[NS], has0[NS], has1[NS];
    __device__ __forceinline__ void init(const Args &a, int sub) {
        const int d_rot = a.d_rot, n_rot = d_rot / (2 * VEC);
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
__device__ __forceinline__ void store_row(T *row, const float (&e)[NS][2 * VEC], const Slots<VEC, L, NS> &s) {
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        Pack<T, VEC> a, b;
        a.narrow(e[n]);
        b.narrow(e[n] + VEC);
        if (s.has0[n]) a.store(row + s.o0[n]);
        if (s.has1[n]) b.store(row + s.o1[n]);
    }
}

// Two fp32 operations in one instruction (f32x2) on neighbouring elements
using window::add2;
using window::f2;
using window::fma2;
using window::mul2;
using window::unf2;
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
template <int N> __device__ __forceinline__ uint64_t at2(const float (&e)[N], int i) { return f2(e[i], e[i + 1]); }

// 16 bytes (or one element) of global memory into this thread's own slot of
// shared memory, asynchronously
template <typename T, int VEC> __device__ __forceinline__ void stage(Pack<T, VEC> *dst, const T *src) {
    if constexpr (VEC == 1) {
        dst->load(src);
    } else {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
    }
}
__device__ __forceinline__ void stage_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void stage_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A lane's slots of a row: staged as [slot][2][thread] packs, then widened
template <int TH, typename T, int VEC, int L, int NS>
__device__ __forceinline__ void stage_row(Pack<T, VEC> *st, const T *row, const Slots<VEC, L, NS> &s) {
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        if (s.has0[n]) stage(st + (2 * n) * TH + threadIdx.x, row + s.o0[n]);
        if (s.has1[n]) stage(st + (2 * n + 1) * TH + threadIdx.x, row + s.o1[n]);
    }
}

// The packs that no row fills read as zeros: set once, so that no row needs a
// choice for each element
template <int TH, typename T, int VEC, int L, int NS>
__device__ __forceinline__ void clear_rest(Pack<T, VEC> *st, const Slots<VEC, L, NS> &s) {
    float zero[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) zero[i] = 0.f;
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        if (!s.has0[n]) st[(2 * n) * TH + threadIdx.x].narrow(zero);
        if (!s.has1[n]) st[(2 * n + 1) * TH + threadIdx.x].narrow(zero);
    }
}

template <int TH, typename T, int VEC, int L, int NS>
__device__ __forceinline__ void widen(float (&e)[NS][2 * VEC], const Pack<T, VEC> *st, const Slots<VEC, L, NS> &s) {
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        st[(2 * n) * TH + threadIdx.x].widen(e[n]);
        st[(2 * n + 1) * TH + threadIdx.x].widen(e[n] + VEC);
    }
}

// r / heads for r < 2^31 (Tensor::magic, shift)
__device__ __forceinline__ uint32_t divide(uint32_t r, uint32_t magic, uint32_t shift) {
    return (uint32_t)(((uint64_t)r * magic) >> shift);
}

// The cosines and sines of tokens tok0 .. tok0 + n - 1, times the factor, by the
// whole block: table[token][2][d_rot / 2].
template <int TH>
__device__ __forceinline__ void fill_table(float *table, const Args &a, uint32_t tok0, uint32_t n) {
    const uint32_t half = (uint32_t)a.d_rot / 2;
    for (uint32_t i = threadIdx.x; i < n * half; i += TH) {
        const uint32_t t = i / half, f = i - t * half;
        const int64_t pos = a.pos != nullptr ? a.pos[tok0 + t] : a.pos0 + (int64_t)(tok0 + t);
        const uint64_t turn = (uint64_t)pos * a.step[f];
        const float half_turns = (float)(int32_t)(uint32_t)(turn >> 32) * 4.656612873077393e-10f;  // 2^-31
        float c, s;
        sincospif(half_turns, &s, &c);
        table[2 * t * half + f] = c * a.factor;
        table[(2 * t + 1) * half + f] = s * a.factor * a.sign;
    }
}

// The lane's part of a token's table
template <int VEC, int L, int NS>
__device__ __forceinline__ void read_table(float (&cs)[NS][VEC], float (&sn)[NS][VEC], const float *table, const Args &a,
                                           uint32_t t, const Slots<VEC, L, NS> &s) {
    const float *c = table + 2 * t * (uint32_t)(a.d_rot / 2), *n = c + a.d_rot / 2;
#pragma unroll
    for (int k = 0; k < NS; ++k)
        if (s.rot[k]) {
            if (VEC % 4 == 0) {
#pragma unroll
                for (int i = 0; i < VEC; i += 4) {
                    *reinterpret_cast<float4 *>(&cs[k][i]) = *reinterpret_cast<const float4 *>(c + s.f0[k] + i);
                    *reinterpret_cast<float4 *>(&sn[k][i]) = *reinterpret_cast<const float4 *>(n + s.f0[k] + i);
                }
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    cs[k][i] = c[s.f0[k] + i];
                    sn[k][i] = n[s.f0[k] + i];
                }
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
        } else if constexpr (VEC > 1) {
#pragma unroll
            for (int i = 0; i < VEC; i += 2) {
                const uint64_t u = at2(e[n], i), v = at2(e[n], VEC + i), c = at2(cs[n], i), z = at2(sn[n], i);
                unf2(sub2(mul2(u, c), mul2(v, z)), e[n][i], e[n][i + 1]);
                unf2(fma2(u, z, mul2(v, c)), e[n][VEC + i], e[n][VEC + i + 1]);
            }
        } else {
            const float u = e[n][0], v = e[n][1];
            e[n][0] = u * cs[n][0] - v * sn[n][0];
            e[n][1] = u * sn[n][0] + v * cs[n][0];
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
__device__ __forceinline__ void load_weight(float (&w)[NS][2 * VEC], const void *weight, const Slots<VEC, L, NS> &s) {
    const T *p = static_cast<const T *>(weight);
#pragma unroll
    for (int n = 0; n < NS; ++n) {
#pragma unroll
        for (int i = 0; i < 2 * VEC; ++i) w[n][i] = 1.f;
        Pack<T, VEC> a;
        if (p != nullptr && s.has0[n]) {
            a.load(p + s.o0[n]);
            a.widen(w[n]);
        }
        if (p != nullptr && s.has1[n]) {
            a.load(p + s.o1[n]);
            a.widen(w[n] + VEC);
        }
    }
}

// A lane's weights in shared memory, four of a slot beside the next lane's four
// (single elements: one), which the warp's groups read at once
template <int VEC, int L, int NS> struct Weights {
    static constexpr int W = VEC > 1 ? 4 : 1, N = NS * 2 * VEC * L;
    static __device__ __forceinline__ float *at(float *p, int sub, int n, int i) {
        return p + ((n * 2 * VEC + i) / W * L + sub) * W;
    }
    static __device__ __forceinline__ void put(float *p, int sub, const float (&w)[NS][2 * VEC]) {
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < 2 * VEC; i += W)
                if constexpr (W == 4) *reinterpret_cast<float4 *>(at(p, sub, n, i)) = make_float4(w[n][i], w[n][i + 1], w[n][i + 2], w[n][i + 3]);
                else *at(p, sub, n, i) = w[n][i];
    }
    static __device__ __forceinline__ void get(float (&w)[NS][2 * VEC], float *p, int sub) {
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < 2 * VEC; i += W)
                if constexpr (W == 4) *reinterpret_cast<float4 *>(&w[n][i]) = *reinterpret_cast<float4 *>(at(p, sub, n, i));
                else w[n][i] = *at(p, sub, n, i);
    }
};

// sum of squares of the lane's elements (an even number)
template <int NS, int E> __device__ __forceinline__ float squares(const float (&e)[NS][E]) {
    uint64_t q = f2(0.f, 0.f);
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int i = 0; i < E; i += 2) q = fma2(at2(e[n], i), at2(e[n], i), q);
    float a, b;
    unf2(q, a, b);
    return a + b;
}

// Shared memory for the gradient's staged rows, or its sums where they are more
template <typename T, int VEC, int NS, int U> __host__ __device__ constexpr int grad_stage_bytes() {
    const int rows = 2 * U * 2 * 2 * NS * kGradThreads * (int)sizeof(Pack<T, VEC>), sums = kGradThreads * NS * 2 * VEC * 4;
    return ((rows > sums ? rows : sums) + 15) / 16 * 16;
}

// The forward of both operators (and, with sign -1, the gradient of the
// rotation): a block takes a.tokens_of tokens and walks their heads, those of
// all tensors of a token one after another.  U: rows of a group that are under
// way together, each lane's in its own slots of shared memory, so that they
// cost no registers.  Each lane computes the place of one of its warp's rows.
template <typename T, int VEC, int L, int NS, int U, bool NORM>
__global__ void __launch_bounds__(kThreads, NORM ? kNormBlocksPerSm : 5) rope_kernel(const __grid_constant__ Args a) {
    constexpr uint32_t G = kThreads / L, GW = 32 / L;
    static_assert(GW * U <= 32, "a lane computes one row's place");
    __shared__ Pack<T, VEC> staged[U][2 * NS * kThreads];
    // weights: widened into shared memory where a lane has many rows (60.4 against
    // 62.7 us at 16384 tokens), read as they are for one
    constexpr bool kShared = NORM && U > 1;
    __shared__ __align__(16) float weights[kShared ? 3 : 1][kShared ? Weights<VEC, L, NS>::N : 1];
    static_assert(sizeof(staged) + sizeof(weights) + kTableBytes <= 48 * 1024, "what a launch may use unasked");
    extern __shared__ __align__(16) float table[];
    const int sub = (int)threadIdx.x % L;
    const uint32_t mask = L == 32 ? 0xffffffffu : ((1u << L) - 1u) << ((threadIdx.x & 31u) & ~(uint32_t)(L - 1));
    const uint32_t lane = threadIdx.x & 31u, in_warp = lane / L;  // the group's place in its warp
    const uint32_t tok0 = blockIdx.x * a.tokens_of, n_tok = min(a.tokens_of, a.n_tokens - tok0);
    const uint32_t rows = n_tok * a.heads, h0 = (uint32_t)a.t[0].heads, h1 = h0 + (uint32_t)a.t[1].heads;
    // (a copied row's elements go the same ways as a rotated one's)
    Slots<VEC, L, NS> s;
    s.init(a, sub);
#pragma unroll
    for (int u = 0; u < U; ++u) clear_rest<kThreads>(staged[u], s);
    // rows, positions, slots and weights may be the previous kernel's, and so may
    // readers of the rows written here
    ptx::grid_wait();
    for (uint32_t r0 = 0; r0 < rows; r0 += G * U) {
        const uint32_t mine = r0 + lane / GW * G + threadIdx.x / 32 * GW + lane % GW;
        const bool real = lane < GW * U && mine < rows;
        const uint32_t my_tok = real ? divide(mine, a.magic, a.shift) : 0u;
        uint32_t my_head = real ? mine - my_tok * a.heads : 0u;
        const uint32_t my_x = (my_head >= h0) + (my_head >= h1);
        my_head -= my_x == 0 ? 0 : my_x == 1 ? h0 : h1;
        const Tensor &my = a.t[my_x];
        int64_t my_to = (int64_t)tok0 + my_tok;
        const T *my_src = static_cast<const T *>(my.x) + my_to * my.xt + (int64_t)my_head * my.xh;
        const bool scatter = my.scatter;
        if (scatter && real) my_to = a.slots[my_to];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const T *src = reinterpret_cast<const T *>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(my_src), u * GW + in_warp));
            if (r0 + u * G + threadIdx.x / L < rows) stage_row<kThreads>(staged[u], src, s);
        }
        stage_commit();
        if (r0 == 0) {
            fill_table<kThreads>(table, a, tok0, n_tok);
            const uint32_t grp = threadIdx.x / L;  // (a group a tensor: kThreads / L >= 8 of them)
            if (kShared && grp < (uint32_t)a.n_tensors && a.t[grp].norm) {
                float w[NS][2 * VEC];
                load_weight<T>(w, a.t[grp].w, s);
                Weights<VEC, L, NS>::put(weights[grp], sub, w);
            }
            __syncthreads();
        }
        const bool kept = real && (!scatter || (my_to >= 0 && my_to < a.n_slots));
        T *my_dst = static_cast<T *>(my.y) + my_to * my.yt + (int64_t)my_head * my.yh;
        const uint32_t my_row = kept ? my_tok << 2 | my_x : ~0u;
        stage_wait<0>();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t row = __shfl_sync(0xffffffffu, my_row, u * GW + in_warp);
            T *dst = reinterpret_cast<T *>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(my_dst), u * GW + in_warp));
            if (row == ~0u) continue;
            const Tensor &t = a.t[row & 3u];
            float e[NS][2 * VEC];
            widen<kThreads>(e, staged[u], s);
            if (NORM && t.norm) {
                const float inv = rsqrtf(group_sum<L>(squares(e), mask) * a.inv_d + a.eps);
                float w[NS][2 * VEC];  // (read for each row: kept, it costs a block an SM)
                if constexpr (kShared) Weights<VEC, L, NS>::get(w, weights[row & 3u], sub);
                else load_weight<T>(w, t.w, s);
#pragma unroll
                for (int n = 0; n < NS; ++n)
#pragma unroll
                    for (int i = 0; i < 2 * VEC; i += 2)
                        unf2(mul2(mul2(at2(e[n], i), f2(inv, inv)), at2(w[n], i)), e[n][i], e[n][i + 1]);
            }
            if (!t.copy) {
                float cs[NS][VEC], sn[NS][VEC];
                read_table(cs, sn, table, a, row >> 2, s);
                turn(e, cs, sn, a, s);
            }
            store_row(dst, e, s);
        }
    }
}

// The gradient of norm and rotation.  With g = R^T dy, r = rsqrt(mean x^2 + eps):
// dx = r (g w - x r mean(g w x r)), dw = sum over rows of g x r.  A lane sums
// its elements' dw over all its rows in registers, a block its groups' sums in
// shared memory, and norm_dw_kernel the blocks' -- each in a fixed order.  The
// blocks are persistent, so that there are few partial sums, and each step's
// rows are staged while the step before is computed.
template <typename T, int VEC, int L, int NS, int U>
__global__ void __launch_bounds__(kGradThreads, kGradBlocksPerSm) norm_grad_kernel(const __grid_constant__ Args a) {
    constexpr int G = kGradThreads / L;
    constexpr int kSlots = 2 * NS * kGradThreads;
    extern __shared__ __align__(16) uint8_t sm[];
    Pack<T, VEC> *staged = reinterpret_cast<Pack<T, VEC> *>(sm);               // [2][U][x, dy][slots]
    float *sums = reinterpret_cast<float *>(sm);                               // [group][element], at the end
    float *table = reinterpret_cast<float *>(sm + grad_stage_bytes<T, VEC, NS, U>());  // [2][token][2][d_rot / 2]
    const int sub = (int)threadIdx.x % L;
    const uint32_t grp = threadIdx.x / L;
    const uint32_t mask = L == 32 ? 0xffffffffu : ((1u << L) - 1u) << ((threadIdx.x & 31u) & ~(uint32_t)(L - 1));
    Slots<VEC, L, NS> s;
    s.init(a, sub);
    ptx::grid_wait();
    for (int x = 0; x < a.n_tensors; ++x) {
        const Tensor &t = a.t[x];
        const uint32_t heads = (uint32_t)t.heads, magic = t.magic, shift = t.shift;
        // a step: up to G * U consecutive rows of the tensor whose tokens' angles fit the table
        const uint32_t rows = a.n_tokens * heads, per = min((uint32_t)(G * U), (a.table_tokens - 1) * heads);
        const int64_t xt = t.xt, xh = t.xh, gt = t.gt, gh = t.gh, yt = t.yt, yh = t.yh;
        const T *src = static_cast<const T *>(t.x), *grd = static_cast<const T *>(t.dy);
        T *dst = static_cast<T *>(t.y);
        float w[NS][2 * VEC], acc[NS][2 * VEC];
        load_weight<T>(w, t.w, s);
#pragma unroll
        for (int k = 0; k < 4 * U; ++k) clear_rest<kGradThreads>(staged + k * kSlots, s);
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < 2 * VEC; ++i) acc[n][i] = 0.f;
        auto issue = [&](uint32_t r0, uint32_t half) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t r = r0 + (uint32_t)(u * G) + grp;
                if ((uint32_t)(u * G) + grp < per && r < rows) {
                    const uint32_t tok = divide(r, magic, shift);
                    const int64_t h = (int64_t)(r - tok * heads);
                    Pack<T, VEC> *st = staged + (half * U + u) * 2 * kSlots;
                    stage_row<kGradThreads>(st, src + (int64_t)tok * xt + h * xh, s);
                    stage_row<kGradThreads>(st + kSlots, grd + (int64_t)tok * gt + h * gh, s);
                }
            }
            stage_commit();
        };
        const uint32_t step = gridDim.x * per;
        uint32_t half = 0;
        issue(blockIdx.x * per, half);
        for (uint32_t r0 = blockIdx.x * per; r0 < rows; r0 += step, half ^= 1u) {
            const uint32_t r1 = min(r0 + per, rows), tok0 = divide(r0, magic, shift);
            issue(r0 + step < rows ? r0 + step : rows, half ^ 1u);
            float *tab = table + half * a.table_tokens * (uint32_t)a.d_rot;
            fill_table<kGradThreads>(tab, a, tok0, divide(r1 - 1, magic, shift) - tok0 + 1);
            __syncthreads();
            stage_wait<1>();
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t r = r0 + (uint32_t)(u * G) + grp;
                if (r >= r1) break;
                const uint32_t tok = divide(r, magic, shift);
                const Pack<T, VEC> *st = staged + (half * U + u) * 2 * kSlots;
                float e[NS][2 * VEC], g[NS][2 * VEC];
                {
                    float cs[NS][VEC], sn[NS][VEC];
                    widen<kGradThreads>(g, st + kSlots, s);
                    read_table(cs, sn, tab, a, tok - tok0, s);
                    turn(g, cs, sn, a, s);
                }
                widen<kGradThreads>(e, st, s);
                float gw[NS][2 * VEC];
                uint64_t m2 = f2(0.f, 0.f);  // sums of g w x
#pragma unroll
                for (int n = 0; n < NS; ++n)
#pragma unroll
                    for (int i = 0; i < 2 * VEC; i += 2) {
                        const uint64_t v = mul2(at2(g[n], i), at2(w[n], i));
                        unf2(v, gw[n][i], gw[n][i + 1]);
                        m2 = fma2(v, at2(e[n], i), m2);
                    }
                float m0, m1;
                unf2(m2, m0, m1);
                const float inv = rsqrtf(group_sum<L>(squares(e), mask) * a.inv_d + a.eps);
                const float mean = group_sum<L>(m0 + m1, mask) * inv * a.inv_d;
                const uint64_t inv2 = f2(inv, inv), k2 = f2(-inv * mean, -inv * mean);
#pragma unroll
                for (int n = 0; n < NS; ++n)
#pragma unroll
                    for (int i = 0; i < 2 * VEC; i += 2) {
                        const uint64_t h = mul2(at2(e[n], i), inv2);
                        unf2(fma2(at2(g[n], i), h, at2(acc[n], i)), acc[n][i], acc[n][i + 1]);
                        unf2(fma2(h, k2, mul2(at2(gw[n], i), inv2)), e[n][i], e[n][i + 1]);
                    }
                store_row(dst + (int64_t)tok * yt + (int64_t)(r - tok * heads) * yh, e, s);
            }
        }
        stage_wait<0>();
        __syncthreads();  // every lane has read its staged rows
        if (a.partial == nullptr) continue;
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                if (s.has0[n]) sums[grp * a.d + s.o0[n] + i] = acc[n][i];
                if (s.has1[n]) sums[grp * a.d + s.o1[n] + i] = acc[n][VEC + i];
            }
        __syncthreads();
        for (int j = (int)threadIdx.x; j < a.d; j += kGradThreads) {
            float v = 0.f;
            for (int k = 0; k < G; ++k) v += sums[k * a.d + j];
            a.partial[((int64_t)blockIdx.x * 2 + x) * kMaxD + j] = v;
        }
        __syncthreads();  // the sums have been read
    }
}

// dw[j] of tensor blockIdx.y: the blocks' partial sums, 32 interleaved chains
// joined in a fixed order.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float *partial, int n, int d, float *dw0, float *dw1) {
    __shared__ float sums[32][33];
    const int j = (int)(blockIdx.x * 32 + threadIdx.x);
    float *dw = blockIdx.y == 0 ? dw0 : dw1;
    ptx::grid_wait();
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

// Written rows may not overlap: heads, and tokens (or slots) where there are several
int check_written(const char *name, int64_t token, int64_t head, int heads, int64_t rows, int d) {
    if ((heads > 1 && std::abs(head) < d) || (heads > 0 && rows > 1 && std::abs(token) < d))
        return host_fail(SYN_ERR_INVALID, std::string(name) + ": output rows overlap");
    return SYN_OK;
}

enum Kind { kTurn, kNorm, kNormGrad };

// Tokens whose rows of `heads` heads fill a block that walks `rows` rows, as
// far as their angles (d_rot floats a token) fit `bytes`; at least one.
uint32_t tokens_for(int64_t rows, int64_t heads, int d_rot, int bytes) {
    return (uint32_t)std::max<int64_t>(1, std::min<int64_t>(rows / heads, bytes / (4 * std::max(d_rot, 1))));
}

template <typename T, int VEC, int L, int NS, int U, bool NORM> int launch_forward(Args &a, int num_sms, cudaStream_t st) {
    constexpr int kPass = kThreads / L * U;  // rows of a block's pass
    a.tokens_of = U > 1 ? tokens_for(kPass * (NORM ? kNormPasses : 1), a.heads, a.d_rot, kTableBytes) : 1;
    // With the norm a pass costs its instructions too: as many tokens as give the
    // fewest rounds of resident blocks, a round costing its passes and half a one
    // (one pass always 65.2 us, up to five 60.4 at 16384 tokens; without the norm
    // one pass 101.4, three 104.0 us at 32768).
    if (NORM && U > 1) {
        const uint64_t slots = (uint64_t)num_sms * kNormBlocksPerSm;
        uint64_t least = ~0ull;
        for (uint32_t t = a.tokens_of, best = t; t >= 1; a.tokens_of = best, --t) {
            const uint64_t rounds = ((a.n_tokens + t - 1) / t + slots - 1) / slots, passes = ((uint64_t)t * a.heads + kPass - 1) / kPass;
            if (rounds * (2 * passes + 1) < least) {
                least = rounds * (2 * passes + 1);
                best = t;
            }
        }
    }
    const unsigned grid = (a.n_tokens + a.tokens_of - 1) / a.tokens_of;
    ROPE_CK((window::launch_early(rope_kernel<T, VEC, L, NS, U, NORM>, grid, kThreads,
                                  (size_t)a.tokens_of * (size_t)a.d_rot * 4, st, a)));
    return SYN_OK;
}

template <typename T, int VEC, int L, int NS> int launch(syn_rope_plan_s *pl, Args &a, Kind kind, cudaStream_t st, int &grid) {
    constexpr int G = kThreads / L, kMany = VEC == 1 ? 1 : kRowsPerLane;
    if (kind == kNormGrad) {
        constexpr int U = VEC == 1 ? 1 : kGradRowsPerLane, G = kGradThreads / L;
        a.table_tokens = 1;
        int64_t blocks = 1;
        for (int x = 0; x < a.n_tensors; ++x) {
            const int64_t heads = a.t[x].heads, most = kTableBytes / (4 * std::max(a.d_rot, 1));
            a.table_tokens = std::max<uint32_t>(a.table_tokens, (uint32_t)std::min<int64_t>(most, (G * U - 1) / heads + 2));
            blocks = std::max<int64_t>(blocks, ((int64_t)a.n_tokens * heads + G * U - 1) / (G * U));
        }
        grid = (int)std::min<int64_t>(blocks, (int64_t)pl->num_sms * kGradBlocksPerSm);
        const size_t smem = (size_t)grad_stage_bytes<T, VEC, NS, U>() + (size_t)a.table_tokens * (size_t)a.d_rot * 8;
        ROPE_CK((window::launch_early(norm_grad_kernel<T, VEC, L, NS, U>, grid, kGradThreads, smem, st, a)));
        return SYN_OK;
    }
    // several rows a lane once that still leaves every SM a few blocks
    int64_t rows = 0;
    for (int x = 0; x < a.n_tensors; ++x) rows += (int64_t)a.n_tokens * a.t[x].heads;
    const bool many = rows >= (int64_t)pl->num_sms * 4 * G * kMany;
    if (kind == kTurn)
        return many ? launch_forward<T, VEC, L, NS, kMany, false>(a, pl->num_sms, st) : launch_forward<T, VEC, L, NS, 1, false>(a, pl->num_sms, st);
    return many ? launch_forward<T, VEC, L, NS, kMany, true>(a, pl->num_sms, st) : launch_forward<T, VEC, L, NS, 1, true>(a, pl->num_sms, st);
}

// The gradient kernels may use as much shared memory as any call needs: set once
// here, since the limit is the context's, and a call that set its own need could
// lower it under another host thread's launch.
template <typename T, int VEC, int L, int NS> cudaError_t prepare() {
    constexpr int U = VEC == 1 ? 1 : kGradRowsPerLane;
    return cudaFuncSetAttribute(norm_grad_kernel<T, VEC, L, NS, U>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                grad_stage_bytes<T, VEC, NS, U>() + 2 * kTableBytes);
}
template <typename T> cudaError_t prepare_all() {
    constexpr int V = 16 / (int)sizeof(T);
    cudaError_t e = prepare<T, 1, 32, 4>();
    if (e == cudaSuccess) e = prepare<T, V, 4, 1>();
    if (e == cudaSuccess) e = prepare<T, V, 8, 1>();
    if (e == cudaSuccess) e = prepare<T, V, 16, 1>();
    if constexpr (sizeof(T) == 4)
        if (e == cudaSuccess) e = prepare<T, V, 32, 1>();
    return e;
}

// A lane's slot is two 16-byte vectors where every row, stride and both parts
// of the head allow it, else single elements.
template <typename T> int dispatch(syn_rope_plan_s *pl, Args &a, Kind kind, bool vec, cudaStream_t st, int &grid) {
    constexpr int V = 16 / (int)sizeof(T);
    if (!vec) return launch<T, 1, 32, 4>(pl, a, kind, st, grid);
    const int slots = a.d / (2 * V);
    if (slots <= 4) return launch<T, V, 4, 1>(pl, a, kind, st, grid);
    if (slots <= 8) return launch<T, V, 8, 1>(pl, a, kind, st, grid);
    if constexpr (sizeof(T) == 4)
        if (slots > 16) return launch<T, V, 32, 1>(pl, a, kind, st, grid);
    return launch<T, V, 16, 1>(pl, a, kind, st, grid);
}

// r / n for r < 2^31 as r * magic >> shift
void divisor(int n, uint32_t &magic, uint32_t &shift) {
    uint32_t bits = 0;
    while (((int64_t)1 << bits) < n) ++bits;
    shift = 31 + bits;
    magic = (uint32_t)((((uint64_t)1 << shift) + (uint64_t)n - 1) / (uint64_t)n);
}

int run(syn_rope_plan_s *pl, Args &a, Kind kind, cudaStream_t st, int &grid) {
    const syn_rope_cfg_t &c = pl->cfg;
    grid = 0;
    a.heads = 0;
    a.d = c.d;
    a.d_rot = c.d_rot;
    a.interleaved = c.layout == SYN_ROPE_INTERLEAVED;
    a.step = pl->d_step;
    a.factor = (float)pl->factor;
    a.inv_d = 1.f / (float)c.d;
    const int size = elem_size(c.dtype);
    bool vec = c.d % (32 / size) == 0 && c.d_rot % (32 / size) == 0;
    int64_t rows = 0;
    for (int x = 0; x < a.n_tensors; ++x) {
        const Tensor &t = a.t[x];
        vec = vec && vector_rows(t.w, 0, 0, size) && vector_rows(t.x, t.xt, t.xh, size) && vector_rows(t.y, t.yt, t.yh, size) &&
              (t.dy == nullptr || vector_rows(t.dy, t.gt, t.gh, size));
        rows += (int64_t)a.n_tokens * t.heads;
    }
    if (rows == 0) return SYN_OK;
    if (rows >= (int64_t)1 << 31) return host_fail(SYN_ERR_UNSUPPORTED, "2^31 or more rows in one call");
    for (int x = 0; x < a.n_tensors; ++x) {
        divisor(a.t[x].heads, a.t[x].magic, a.t[x].shift);
        a.heads += (uint32_t)a.t[x].heads;
    }
    divisor((int)a.heads, a.magic, a.shift);
    if (c.dtype == SYN_DTYPE_BF16) return dispatch<__nv_bfloat16>(pl, a, kind, vec, st, grid);
    if (c.dtype == SYN_DTYPE_F16) return dispatch<__half>(pl, a, kind, vec, st, grid);
    return dispatch<float>(pl, a, kind, vec, st, grid);
}

int add(const syn_rope_cfg_t &c, Args &a, const char *name, const syn_rope_rows_t *r, const void *w, bool copy, bool scatter, bool norm) {
    if (r == nullptr) return SYN_OK;
    const int size = elem_size(c.dtype);
    int rc;
    if ((rc = check_rows(name, r->x, size, r->heads, a.n_tokens > 0)) != SYN_OK || (rc = check_rows(name, r->y, size, r->heads, a.n_tokens > 0)) != SYN_OK ||
        (rc = check_rows(name, w, size, 0, false)) != SYN_OK ||
        (rc = check_written(name, r->y_token, r->y_head, r->heads, scatter ? a.n_slots : a.n_tokens, c.d)) != SYN_OK)
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
    const bool norm = kind == kNorm, scatter = slots != nullptr;
    a.slots = slots;
    a.n_slots = n_slots;
    a.eps = eps;
    if ((rc = add(pl->cfg, a, "q", q, wq, false, false, norm)) != SYN_OK || (rc = add(pl->cfg, a, "k", k, wk, false, scatter, norm)) != SYN_OK ||
        (rc = add(pl->cfg, a, "v", v, nullptr, true, scatter, false)) != SYN_OK)
        return rc;
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
    if (e == cudaSuccess)
        e = c.dtype == SYN_DTYPE_BF16 ? prepare_all<__nv_bfloat16>() : c.dtype == SYN_DTYPE_F16 ? prepare_all<__half>() : prepare_all<float>();
    if (e == cudaSuccess) e = cudaMalloc(&pl->d_step, std::max<size_t>(step.size(), 1) * sizeof(uint64_t));
    if (e == cudaSuccess)
        e = cudaMalloc(&pl->d_partial, (size_t)pl->num_sms * kGradBlocksPerSm * 2 * kMaxD * sizeof(float));
    if (e == cudaSuccess && !step.empty())
        e = cudaMemcpy(pl->d_step, step.data(), step.size() * sizeof(uint64_t), cudaMemcpyHostToDevice);
    // (the copy may return before it has reached the device, which other streams would not wait for)
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
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
    if ((rc = add(pl->cfg, a, "dq", dq, nullptr, false, false, false)) != SYN_OK ||
        (rc = add(pl->cfg, a, "dk", dk, nullptr, false, false, false)) != SYN_OK)
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
            (rc = check_rows(name, g->dw, 4, 0, false)) != SYN_OK ||
            (rc = check_written(name, g->dx_token, g->dx_head, g->heads, n_tokens, pl->cfg.d)) != SYN_OK)
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
    // the plan's workspace belongs to the one call that wants weight gradients
    const bool sums = dw[0] != nullptr || dw[1] != nullptr;
    a.partial = sums ? pl->d_partial : nullptr;
    int grid = 0;
    rc = run(pl, a, kNormGrad, st, grid);
    if (rc != SYN_OK || a.n_tensors == 0 || !sums) return rc;
    ROPE_CK((window::launch_early(norm_dw_kernel, dim3((unsigned)(pl->cfg.d + 31) / 32, (unsigned)a.n_tensors), dim3(32, 32), 0,
                                  st, pl->d_partial, grid, pl->cfg.d, dw[0], dw[1])));
    return SYN_OK;
}

}  // extern "C"
