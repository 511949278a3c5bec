// norm.cu -- layer norm of rows and its gradient (C ABI: include/syn_norm.h).
//
// Both operators read each element once and write one (the gradient reads x and
// dy), so HBM bounds them at long inputs and the launch at a few rows.  A row
// belongs to L lanes: a power of two up to 32, else a number of warps; a lane
// keeps its part of the row, NV vectors of 16 bytes (single elements where the
// tensors' rows lie differently to 16-byte boundaries), so that the mean comes
// first and the squares are those of the deviations from it.
//
// Measured on one GB300 (back-to-back calls): 16384 rows of 4096 bf16 43.8-45.6 us,
// 6.0 TB/s of the measured copy rate's 6.8 (its 24 warps an SM wait for a row's one
// reduction and barrier); the gradient 74.9-77.8 us, 5.3 TB/s (16 warps an SM: 128
// registers, half of the issue slots).  Without the reduction the forward takes 39.7 us,
// HBM's time.  Four rows take 3.0 us in a graph and 5.3-6.4 with the host side.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <initializer_list>
#include <new>
#include <string>

#include "elements.cuh"
#include "host_util.h"
#include "syn.h"
#include "syn_norm.h"
#include "window.cuh"

namespace syn {
namespace norm {

using elem::Num;
using elem::Pack;
using window::add2;
using window::f2;
using window::fma2;
using window::mul2;
using window::unf2;

constexpr int kMaxD = 16384;
constexpr int kMaxGroups = 12;  // groups of several warps (64 lanes or more) in a block: barriers 1..12

struct Args {
    const void *x, *dy;
    void *y;               // the gradient: dx
    const void *w, *b;
    int64_t xs, gs, ys;    // elements from row to row
    int64_t rows;
    int32_t d, lanes;
    int32_t off0, off1;    // elements from a 16-byte boundary to row 0, and from a row to the next (EDGE)
    float eps, inv_d;
    float *partial;        // [grid][2][d] sums of dw and db (nullptr: not wanted)
};

template <int N> __device__ __forceinline__ uint64_t at2(const float (&e)[N], int i) { return f2(e[i], e[i + 1]); }

// Elements as pairs, two fp32 operations an instruction (the odd one out of an odd
// vector goes alone)
__device__ __forceinline__ uint64_t twice(float v) { return f2(v, v); }
// s += sum of e
template <int E> __device__ __forceinline__ void add_all(const float (&e)[E], uint64_t &s) {
    if constexpr (E == 1) {
        s = add2(s, f2(e[0], 0.f));
    } else {
#pragma unroll
        for (int i = 0; i < E; i += 2) s = add2(s, at2(e, i));
    }
}
// s += sum of a * b
template <int E> __device__ __forceinline__ void add_products(const float (&a)[E], const float (&b)[E], uint64_t &s) {
    if constexpr (E == 1) {
        s = fma2(f2(a[0], 0.f), f2(b[0], 0.f), s);
    } else {
#pragma unroll
        for (int i = 0; i < E; i += 2) s = fma2(at2(a, i), at2(b, i), s);
    }
}
// o = a * b
template <int E> __device__ __forceinline__ void multiply(const float (&a)[E], const float (&b)[E], float (&o)[E]) {
    if constexpr (E == 1) {
        o[0] = a[0] * b[0];
    } else {
#pragma unroll
        for (int i = 0; i < E; i += 2) unf2(mul2(at2(a, i), at2(b, i)), o[i], o[i + 1]);
    }
}
// o = a * k + c
template <int E> __device__ __forceinline__ void scale_add(const float (&a)[E], float k, float c, float (&o)[E]) {
    if constexpr (E == 1) {
        o[0] = fmaf(a[0], k, c);
    } else {
#pragma unroll
        for (int i = 0; i < E; i += 2) unf2(fma2(at2(a, i), twice(k), twice(c)), o[i], o[i + 1]);
    }
}
// o = a - m
template <int E> __device__ __forceinline__ void subtract(const float (&a)[E], float m, float (&o)[E]) {
    if constexpr (E == 1) {
        o[0] = a[0] - m;
    } else {
#pragma unroll
        for (int i = 0; i < E; i += 2) unf2(add2(at2(a, i), twice(-m)), o[i], o[i + 1]);
    }
}
// o = a * b + o, b a factor for all or each its own
template <int E> __device__ __forceinline__ void accumulate(const float (&a)[E], const float (&b)[E], float *o) {
    if constexpr (E == 1) {
        o[0] = fmaf(a[0], b[0], o[0]);
    } else {
#pragma unroll
        for (int i = 0; i < E; i += 2) unf2(fma2(at2(a, i), at2(b, i), f2(o[i], o[i + 1])), o[i], o[i + 1]);
    }
}
template <int E> __device__ __forceinline__ void accumulate(const float (&a)[E], float b, float *o) {
    if constexpr (E == 1) {
        o[0] = fmaf(a[0], b, o[0]);
    } else {
#pragma unroll
        for (int i = 0; i < E; i += 2) unf2(fma2(at2(a, i), twice(b), f2(o[i], o[i + 1])), o[i], o[i + 1]);
    }
}
__device__ __forceinline__ float both(uint64_t s) {
    float a, b;
    unf2(s, a, b);
    return a + b;
}

// A vector's elements as pairs in 64-bit registers from load to store
template <typename T, int VEC> __device__ __forceinline__ void widen(const Pack<T, VEC> &p, uint64_t (&e)[VEC / 2]) {
    const uint32_t w[4] = {p.v.x, p.v.y, p.v.z, p.v.w};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) e[i] = f2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            float a, b;
            Num<T>::get2(w[i], a, b);
            e[i] = f2(a, b);
        }
    }
}
template <typename T, int VEC> __device__ __forceinline__ void narrow(Pack<T, VEC> &p, const uint64_t (&e)[VEC / 2]) {
    float f[VEC];
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) unf2(e[i], f[2 * i], f[2 * i + 1]);
    p.narrow(f);
}

// Where a lane's vectors lie in its row.  Vectors begin at 16-byte boundaries of
// memory; with EDGE a row begins `off` elements behind one, so that its first and
// last vector may be parts, whose elements are stored one by one.
template <int VEC, int NV, bool EDGE> struct Place {
    int col0, step, d;  // column of the lane's first vector; columns from one to the next
    __device__ __forceinline__ Place(const Args &a, int64_t row, int sub) {
        const int off = EDGE ? (int)((a.off0 + (row & (VEC - 1)) * a.off1) & (VEC - 1)) : 0;
        col0 = sub * VEC - off;
        step = a.lanes * VEC;
        d = a.d;
    }
    __device__ __forceinline__ int col(int i) const { return col0 + i * step; }
    __device__ __forceinline__ bool whole(int i) const { return (!EDGE || col(i) >= 0) && col(i) + VEC <= d; }
    __device__ __forceinline__ bool part(int i) const { return EDGE && !whole(i) && col(i) + VEC > 0 && col(i) < d; }
    __device__ __forceinline__ bool has(int i, int k) const { return col(i) + k >= 0 && col(i) + k < d; }
    // e's elements outside the row to zero
    __device__ __forceinline__ void mask(int i, float (&e)[VEC]) const {
        if (whole(i)) return;
#pragma unroll
        for (int k = 0; k < VEC; ++k)
            if (!has(i, k)) e[k] = 0.f;
    }
    template <typename T> __device__ __forceinline__ void load(Pack<T, VEC> &p, const T *row, int i) const {
        if constexpr (!EDGE && VEC > 1) {
            p.v = whole(i) ? *reinterpret_cast<const uint4 *>(row + col(i)) : make_uint4(0, 0, 0, 0);
            return;
        }
        float e[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) e[k] = 0.f;
        p.narrow(e);
        if (whole(i)) {
            p.load(row + col(i));
        } else if (part(i)) {
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                if (has(i, k)) e[k] = Num<T>::get(row[col(i) + k]);
            p.narrow(e);
        }
    }
    template <typename T> __device__ __forceinline__ void store(T *row, int i, const float (&e)[VEC]) const {
        if (whole(i)) {
            Pack<T, VEC> p;
            p.narrow(e);
            p.store(row + col(i));
        } else if (part(i)) {
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                if (has(i, k)) row[col(i) + k] = Num<T>::put(e[k]);
        }
    }
    __device__ __forceinline__ void mask(int i, uint64_t (&e)[VEC / 2 + (VEC == 1)]) const {
        if (whole(i)) return;
#pragma unroll
        for (int k = 0; k < VEC / 2; ++k) {
            float a, b;
            unf2(e[k], a, b);
            e[k] = f2(has(i, 2 * k) ? a : 0.f, has(i, 2 * k + 1) ? b : 0.f);
        }
    }
    template <typename T> __device__ __forceinline__ void store(T *row, int i, const uint64_t (&e)[VEC / 2 + (VEC == 1)]) const {
        if (whole(i)) {
            Pack<T, VEC> p;
            narrow(p, e);
            p.store(row + col(i));
        } else if (part(i)) {
#pragma unroll
            for (int k = 0; k < VEC / 2; ++k) {
                float a, b;
                unf2(e[k], a, b);
                if (has(i, 2 * k)) row[col(i) + 2 * k] = Num<T>::put(a);
                if (has(i, 2 * k + 1)) row[col(i) + 2 * k + 1] = Num<T>::put(b);
            }
        }
    }
    // a weight's elements (with EDGE they begin at no boundary of their own)
    template <typename T> __device__ __forceinline__ void weight(float (&e)[VEC], const T *w, int i) const {
        if (EDGE) {
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                if (has(i, k)) e[k] = Num<T>::get(w[col(i) + k]);
        } else if (whole(i)) {
            Pack<T, VEC> p;
            p.load(w + col(i));
            p.widen(e);
        }
    }
};

// A row whose first and last vectors, with what lies beside the row in them, are within
// its tensor: neither the first nor the last one, and not on top of each other.  They
// are brought as they are and masked when they are read (element by element a warp
// waited for them in each row).
template <int VEC> __device__ __forceinline__ bool inner(const Args &a, int64_t row, int64_t stride) {
    return row > 0 && row < a.rows - 1 && (stride >= VEC || stride <= -VEC);
}

// The lanes of a row: a power of two of a warp's, or several warps, whose sums meet
// in shared memory at barrier `bar` of the row's lanes.  Sums of N values take N x 32
// floats there, not in use by a sum that some lane has yet to leave, zero where no
// warp writes.  (Bounds and places are worked out once: with loops and remainders in
// them the sums were 126 of a row's 316 instructions.)
constexpr int kPlace = 4 * 32;  // floats of a place for sums
struct Row {
    int lanes, warps, bar, threads, lane;
    float *out[3], *in[3];  // this lane's, of one, two and four values
    __device__ __forceinline__ Row(int L, int sub, int bar_, int threads_, float *red) {
        lanes = L;
        warps = (L + 31) / 32;
        bar = bar_;
        threads = threads_;
        lane = (int)threadIdx.x & 31;
        const int half = (lane >> 4) * 32, quarter = ((lane >> 3) & 1) * 64 + half, warp = sub >> 5;
        out[0] = red + warp;
        out[1] = red + half + warp;
        out[2] = red + quarter + warp;
        in[0] = red + (lane & 7);
        in[1] = red + half + (lane & 7);
        in[2] = red + quarter + (lane & 7);
    }
    __device__ __forceinline__ static float over(float v, int from) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            if (o <= from) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
    // the warps' sums, of value k of kind `kind`, eight lanes taking them (and the lanes
    // beside them the same)
    __device__ __forceinline__ float join(float v, int kind, int lanes_each, int place) const {
        if ((lane & (lanes_each - 1)) == 0) out[kind][place] = v;
        asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(threads) : "memory");
        const float *p = in[kind] + place;
        v = p[0];
        if (warps > 8) v += p[8];
        if (warps > 16) v += p[16];
        if (warps > 24) v += p[24];
        return over(v, 4);
    }
    // Sum over the row's lanes, in each of them
    __device__ __forceinline__ float sum(float v, int place) const {
        if (lanes < 32) {
            for (int o = lanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            return v;
        }
        v = over(v, 16);
        return warps == 1 ? v : join(v, 0, 32, place);
    }
    // Two sums at once: half of a warp's lanes go on with each
    __device__ __forceinline__ void sum2(float &s0, float &s1, int place) const {
        if (lanes < 32) {
            for (int o = lanes / 2; o > 0; o >>= 1) {
                s0 += __shfl_xor_sync(0xffffffffu, s0, o);
                s1 += __shfl_xor_sync(0xffffffffu, s1, o);
            }
            return;
        }
        const bool odd = (lane & 16) != 0;
        float v = over((odd ? s1 : s0) + __shfl_xor_sync(0xffffffffu, odd ? s0 : s1, 16), 8);
        if (warps > 1) v = join(v, 1, 16, place);
        s0 = __shfl_sync(0xffffffffu, v, 0);
        s1 = __shfl_sync(0xffffffffu, v, 16);
    }
    // Four sums at once.  Half of the lanes go on with one of two sums, half with the
    // other; then halves of these with sums of both pairs: 6 exchanges for 20.
    __device__ __forceinline__ void sum4(float &s0, float &s1, float &s2, float &s3, int place) const {
        if (lanes < 32) {
            for (int o = lanes / 2; o > 0; o >>= 1) {
                s0 += __shfl_xor_sync(0xffffffffu, s0, o);
                s1 += __shfl_xor_sync(0xffffffffu, s1, o);
                s2 += __shfl_xor_sync(0xffffffffu, s2, o);
                s3 += __shfl_xor_sync(0xffffffffu, s3, o);
            }
            return;
        }
        const bool odd = (lane & 16) != 0, upper = (lane & 8) != 0;
        const float v = (odd ? s1 : s0) + __shfl_xor_sync(0xffffffffu, odd ? s0 : s1, 16);
        const float u = (odd ? s3 : s2) + __shfl_xor_sync(0xffffffffu, odd ? s2 : s3, 16);
        float w = over((upper ? u : v) + __shfl_xor_sync(0xffffffffu, upper ? v : u, 8), 4);
        if (warps > 1) w = join(w, 2, 8, place);
        s0 = __shfl_sync(0xffffffffu, w, 0);
        s1 = __shfl_sync(0xffffffffu, w, 16);
        s2 = __shfl_sync(0xffffffffu, w, 8);
        s3 = __shfl_sync(0xffffffffu, w, 24);
    }
};
// (before a barrier of all)
__device__ __forceinline__ void clear_places(float *red, int n) {
    for (int i = (int)threadIdx.x; i < n; i += (int)blockDim.x) red[i] = 0.f;
}

// The forward: a block of blockDim.x / L rows.
template <typename T, int VEC, int NV, bool EDGE>
__global__ void __launch_bounds__(NV == 8 ? 544 : 1024) layer_norm_kernel(const __grid_constant__ Args a) {
    __shared__ float red[2 * 32];
    const int L = a.lanes, sub = (int)threadIdx.x % L;
    const Row r(L, sub, 0, (int)blockDim.x, red);
    if (L > 32) {
        clear_places(red, 2 * 32);
        __syncthreads();
    }
    const int64_t row = (int64_t)blockIdx.x * ((int)blockDim.x / L) + (int)threadIdx.x / L;
    const bool real = row < a.rows;
    const Place<VEC, NV, EDGE> at(a, row, sub);
    ptx::grid_wait();
    // (a lane group without a row takes the last one and stores nothing)
    const T *x = static_cast<const T *>(a.x) + (real ? row : a.rows - 1) * a.xs;
    Pack<T, VEC> v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (!EDGE || real) {
            at.load(v[i], x, i);
        } else {
            float zero[VEC];
#pragma unroll
            for (int k = 0; k < VEC; ++k) zero[k] = 0.f;
            v[i].narrow(zero);
        }
    }
    uint64_t sum = twice(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float e[VEC];
        v[i].widen(e);
        add_all(e, sum);
    }
    const float mean = r.sum(both(sum), 0) * a.inv_d;
    sum = twice(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float e[VEC];
        v[i].widen(e);
        // what no row fills stays zero
        subtract(e, EDGE || at.whole(i) ? mean : 0.f, e);
        if (EDGE) at.mask(i, e);
        add_products(e, e, sum);
    }
    const float inv = rsqrtf(r.sum(both(sum), 32) * a.inv_d + a.eps);
    if (!real) return;
    T *y = static_cast<T *>(a.y) + row * a.ys;
    const T *w = static_cast<const T *>(a.w), *b = static_cast<const T *>(a.b);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float e[VEC], f[VEC];
        v[i].widen(e);
        subtract(e, mean, e);
        scale_add(e, inv, 0.f, e);
        if (w != nullptr) {
#pragma unroll
            for (int k = 0; k < VEC; ++k) f[k] = 0.f;
            at.weight(f, w, i);
            multiply(e, f, e);
        }
        if (b != nullptr) {
#pragma unroll
            for (int k = 0; k < VEC; ++k) f[k] = 0.f;
            at.weight(f, b, i);
            accumulate(f, 1.f, e);
        }
        at.store(y, i, e);
    }
}

// 16 bytes (4 bytes; an element of 2 bytes as it is) of global memory into this
// thread's own place in shared memory, asynchronously
template <typename T, int VEC> __device__ __forceinline__ void stage(Pack<T, VEC> *dst, const T *src) {
    if constexpr (sizeof(Pack<T, VEC>) == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
    else if constexpr (sizeof(Pack<T, VEC>) == 4)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
    else
        dst->load(src);
}

// The forward of many rows: persistent blocks as the gradient's below (rows staged ahead,
// weight and bias widened once), and one reduction a row, of its squares and the next
// row's sum.
constexpr int kRowThreads = 768, kRowElems = 16, kRowStages = 4;
static_assert(kRowThreads / 64 <= kMaxGroups, "places and barriers of a block's groups");
template <typename T, int VEC, bool EDGE>
__global__ void __launch_bounds__(kRowThreads, 1) layer_norm_rows_kernel(const __grid_constant__ Args a) {
    constexpr int E = kRowElems, NV = E / VEC, TH = kRowThreads, S = kRowStages;
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ float red[kMaxGroups][2][kPlace];
    Pack<T, VEC> *staged = reinterpret_cast<Pack<T, VEC> *>(sm) + threadIdx.x;  // [S][NV][TH]
    const int L = a.lanes, groups = (int)blockDim.x / L, grp = (int)threadIdx.x / L, sub = (int)threadIdx.x % L;
    const Row r(L, sub, 1 + grp, L, L > 32 ? red[grp][0] : nullptr);
    clear_places(red[0][0], kMaxGroups * 2 * kPlace);
    __syncthreads();
    const int64_t step = (int64_t)gridDim.x * groups, first = (int64_t)blockIdx.x * groups;
    const Place<VEC, NV, EDGE> at(a, first + grp, sub);
    const T *px = static_cast<const T *>(a.x), *pw = static_cast<const T *>(a.w), *pb = static_cast<const T *>(a.b);
    T *py = static_cast<T *>(a.y);
    {  // what no row fills reads as zero
        float zero[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) zero[k] = 0.f;
        for (int i = 0; i < S * NV; ++i) staged[i * TH].narrow(zero);
    }
    ptx::grid_wait();
    // rows of the group: this step's, and the one that is to be brought next
    int64_t row = first + grp, coming = row;
    const T *x_next = px + coming * a.xs;
    auto issue = [&](int slot) {
        if (coming < a.rows) {
            Pack<T, VEC> *st = staged + slot * NV * TH;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (at.whole(i) || (at.part(i) && inner<VEC>(a, coming, a.xs))) {
                    stage(st + i * TH, x_next + at.col(i));
                } else if (at.part(i)) {
                    T *sx = reinterpret_cast<T *>(st + i * TH);
#pragma unroll
                    for (int k = 0; k < VEC; ++k)
                        if (at.has(i, k)) sx[k] = x_next[at.col(i) + k];
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        coming += step;
        x_next += step * a.xs;
    };
    constexpr int H = VEC / 2;
    uint64_t kept_w[NV][H], kept_b[NV][H];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float w[VEC], b[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            w[k] = 1.f;
            b[k] = 0.f;
        }
        if (pw != nullptr) at.weight(w, pw, i);
        if (pb != nullptr) at.weight(b, pb, i);
#pragma unroll
        for (int k = 0; k < H; ++k) {
            kept_w[i][k] = at2(w, 2 * k);
            kept_b[i][k] = at2(b, 2 * k);
        }
    }
    auto part_sum = [&](int slot) {
        uint64_t sum = twice(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            uint64_t x[H];
            widen(staged[(slot * NV + i) * TH], x);
            if (EDGE) at.mask(i, x);
#pragma unroll
            for (int k = 0; k < H; ++k) sum = add2(sum, x[k]);
        }
        return both(sum);
    };
#pragma unroll
    for (int k = 0; k < S - 1; ++k) issue(k);
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
    float mean = r.sum(part_sum(0), kPlace) * a.inv_d;
    T *y = py + row * a.ys;
    // (every group takes the block's steps, one without a row in them with what its
    // places hold, and stores nothing: the shuffles need whole warps)
    int64_t at0 = first;
    auto take = [&](int slot) {
        const Pack<T, VEC> *st = staged + slot * NV * TH;
        issue((slot + S - 1) % S);
        uint64_t p = twice(0.f);
        uint64_t kept[NV][H];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            uint64_t(&x)[H] = kept[i];
            widen(st[i * TH], x);
            // what no row fills stays zero
            const uint64_t m = twice(EDGE || at.whole(i) ? -mean : 0.f);
#pragma unroll
            for (int k = 0; k < H; ++k) x[k] = add2(x[k], m);
            if (EDGE) at.mask(i, x);
#pragma unroll
            for (int k = 0; k < H; ++k) p = fma2(x[k], x[k], p);
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
        float squares = both(p), next = part_sum((slot + 1) % S);
        // (two places in turn: a warp may be a row ahead of another)
        r.sum2(squares, next, (slot & 1) * kPlace);
        mean = next * a.inv_d;
        if (row < a.rows) {
            const uint64_t by = twice(rsqrtf(squares * a.inv_d + a.eps));
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                uint64_t o[H];
#pragma unroll
                for (int k = 0; k < H; ++k) o[k] = fma2(mul2(kept[i][k], by), kept_w[i][k], kept_b[i][k]);
                at.store(y, i, o);
            }
        }
        row += step;
        y += step * a.ys;
        at0 += step;
    };
    while (at0 < a.rows) {
#pragma unroll
        for (int slot = 0; slot < S; ++slot)
            if (at0 < a.rows) take(slot);
    }
}

// Shared memory of the gradient kernel: the staged rows, or its sums at the end
template <typename T, int VEC, int NV, int TH> struct GradLay {
    static constexpr int STAGE = 2 * NV * TH * (int)sizeof(Pack<T, VEC>);
    static constexpr int S = 4 * STAGE <= 210 * 1024 ? 4 : 3 * STAGE <= 210 * 1024 ? 3 : 2 * STAGE <= 210 * 1024 ? 2 : 1;
    static constexpr int SUMS = TH * NV * VEC * 4;
    static constexpr int BYTES = S * STAGE > SUMS ? S * STAGE : SUMS;
};

// The gradient: persistent blocks that take several rows at a time, each group
// of lanes its own, and bring the rows of the steps ahead into shared memory
// meanwhile (a lane its own part, so that no barrier is needed).  A lane keeps the
// sums of its columns' dw and db in registers over all its rows, a block joins its
// groups' and layer_norm_sums_kernel the blocks', each in a fixed order.  With EDGE a group's
// rows all begin at the same distance from a 16-byte boundary (the host makes the
// steps a multiple of the distances' period), so that a lane's columns stay its own.
template <typename T, int VEC, int NV, int TH, bool EDGE>
__global__ void __launch_bounds__(TH, 1) layer_norm_grad_kernel(const __grid_constant__ Args a) {
    constexpr int E = NV * VEC;
    using Lay = GradLay<T, VEC, NV, TH>;
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ float red[kMaxGroups][2][kPlace];
    Pack<T, VEC> *staged = reinterpret_cast<Pack<T, VEC> *>(sm) + threadIdx.x;  // [S][x, dy][NV][TH]
    float *sums = reinterpret_cast<float *>(sm);                                // [group][d], at the end
    const int L = a.lanes, groups = (int)blockDim.x / L, grp = (int)threadIdx.x / L, sub = (int)threadIdx.x % L;
    const Row r(L, sub, 1 + grp, L, L > 32 ? red[grp][0] : nullptr);
    clear_places(red[0][0], kMaxGroups * 2 * kPlace);
    __syncthreads();
    const int64_t step = (int64_t)gridDim.x * groups, first = (int64_t)blockIdx.x * groups;
    const Place<VEC, NV, EDGE> at(a, first + grp, sub);
    const T *px = static_cast<const T *>(a.x), *pg = static_cast<const T *>(a.dy), *pw = static_cast<const T *>(a.w);
    T *py = static_cast<T *>(a.y);
    float dw[E], db[E];
#pragma unroll
    for (int i = 0; i < E; ++i) dw[i] = db[i] = 0.f;
    uint64_t dw2[NV][VEC > 1 ? VEC / 2 : 1], db2[NV][VEC > 1 ? VEC / 2 : 1];  // (as pairs, where a lane has few elements)
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < (VEC > 1 ? VEC / 2 : 1); ++k) dw2[i][k] = db2[i][k] = twice(0.f);
    {  // what no row fills reads as zero
        float zero[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) zero[k] = 0.f;
        for (int i = 0; i < Lay::S * 2 * NV; ++i) staged[i * TH].narrow(zero);
    }
    ptx::grid_wait();
    // rows of the group: this step's, and the one that is to be brought next
    int64_t row = first + grp, coming = row;
    const T *x_next = px + coming * a.xs, *g_next = pg + coming * a.gs;
    auto issue = [&](int slot) {
        if (coming < a.rows) {
            Pack<T, VEC> *st = staged + slot * 2 * NV * TH;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (at.whole(i) || (at.part(i) && inner<VEC>(a, coming, a.xs) && inner<VEC>(a, coming, a.gs))) {
                    stage(st + i * TH, x_next + at.col(i));
                    stage(st + (NV + i) * TH, g_next + at.col(i));
                } else if (at.part(i)) {
                    T *sx = reinterpret_cast<T *>(st + i * TH), *sg = reinterpret_cast<T *>(st + (NV + i) * TH);
#pragma unroll
                    for (int k = 0; k < VEC; ++k)
                        if (at.has(i, k)) {
                            sx[k] = x_next[at.col(i) + k];
                            sg[k] = g_next[at.col(i) + k];
                        }
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        coming += step;
        x_next += step * a.xs;
        g_next += step * a.gs;
    };
    // a lane of few elements keeps its weights widened
    constexpr bool FEW = E <= 16 && VEC > 1 && Lay::S >= 3;
    constexpr int H = VEC > 1 ? VEC / 2 : 1;
    uint64_t kept_w[FEW ? NV : 1][H];
    Pack<T, VEC> weight[FEW ? 1 : NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float w[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) w[k] = 1.f;
        if (pw != nullptr) at.weight(w, pw, i);
        if constexpr (FEW) {
#pragma unroll
            for (int k = 0; k < H; ++k) kept_w[i][k] = at2(w, 2 * k);
        } else {
            weight[i].narrow(w);
        }
    }
    auto landed = [&](int slot) { return staged + slot * 2 * NV * TH; };
    // a vector's deviations from the mean (zero where no row fills it)
    auto deviations = [&](const Pack<T, VEC> *st, int i, float mean, float (&x)[VEC]) {
        st[i * TH].widen(x);
        subtract(x, EDGE || at.whole(i) ? mean : 0.f, x);
        if (EDGE) at.mask(i, x);
    };
    // the lane's part of a row's sum
    auto part_sum = [&](const Pack<T, VEC> *st) {
        uint64_t sum = twice(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float x[VEC];
            st[i * TH].widen(x);
            if (EDGE) at.mask(i, x);
            add_all(x, sum);
        }
        return both(sum);
    };
    // a vector's results, with dx = inv g + h (-inv mean(g h)) - inv mean(g)
    auto results = [&](T *y, int i, float inv, float mg, float mh, float (&x)[VEC], float (&g)[VEC], const float (&w)[VEC]) {
        scale_add(x, inv, 0.f, x);
        accumulate(g, x, dw + i * VEC);
        accumulate(g, 1.f, db + i * VEC);
        multiply(g, w, g);
        scale_add(g, inv, mg, g);
        accumulate(x, mh, g);
        at.store(y, i, g);
    };
    // (every group takes the block's steps, one without a row in them with what its
    // places hold, and stores nothing: the shuffles need whole warps)
    int64_t at0 = first;
    T *y = py + row * a.ys;
    if constexpr (FEW) {
        // the next row's sum is taken beside this row's three, so that a row has one
        // reduction and one barrier
        constexpr int S = Lay::S;
        auto row_part = [&](const Pack<T, VEC> *st) {
            uint64_t sum = twice(0.f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                uint64_t x[H];
                widen(st[i * TH], x);
                if (EDGE) at.mask(i, x);
#pragma unroll
                for (int k = 0; k < H; ++k) sum = add2(sum, x[k]);
            }
            return both(sum);
        };
#pragma unroll
        for (int k = 0; k < S - 1; ++k) issue(k);
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
        float mean = r.sum(row_part(landed(0)), kPlace) * a.inv_d;
        auto take = [&](int slot, int place) {
            const Pack<T, VEC> *st = landed(slot);
            issue((slot + S - 1) % S);
            uint64_t p0 = twice(0.f), p1 = p0, p2 = p0;
            uint64_t x[NV][H], g[NV][H];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                widen(st[i * TH], x[i]);
                widen(st[(NV + i) * TH], g[i]);
                const uint64_t m = twice(EDGE || at.whole(i) ? -mean : 0.f);
#pragma unroll
                for (int k = 0; k < H; ++k) x[i][k] = add2(x[i][k], m);
                if (EDGE) {
                    at.mask(i, x[i]);
                    at.mask(i, g[i]);
                }
#pragma unroll
                for (int k = 0; k < H; ++k) {
                    const uint64_t gw = mul2(g[i][k], kept_w[i][k]);
                    p0 = fma2(x[i][k], x[i][k], p0);
                    p1 = add2(p1, gw);
                    p2 = fma2(gw, x[i][k], p2);
                }
            }
            asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
            float s0 = both(p0), s1 = both(p1), s2 = both(p2), next = row_part(landed((slot + 1) % S));
            r.sum4(s0, s1, s2, next, place);
            mean = next * a.inv_d;
            if (row < a.rows) {
                const float inv = rsqrtf(s0 * a.inv_d + a.eps);
                const uint64_t by = twice(inv), mg = twice(-inv * s1 * a.inv_d), mh = twice(-inv * inv * s2 * a.inv_d);
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    uint64_t o[H];
#pragma unroll
                    for (int k = 0; k < H; ++k) {
                        const uint64_t h = mul2(x[i][k], by);
                        dw2[i][k] = fma2(g[i][k], h, dw2[i][k]);
                        db2[i][k] = add2(db2[i][k], g[i][k]);
                        o[k] = fma2(h, mh, fma2(mul2(g[i][k], kept_w[i][k]), by, mg));
                    }
                    at.store(y, i, o);
                }
            }
            row += step;
            y += step * a.ys;
            at0 += step;
        };
        // (two places in turn: a warp may be a row ahead of another)
        while (at0 < a.rows) {
#pragma unroll
            for (int k = 0; k < (S % 2 == 0 ? S : 2 * S); ++k)
                if (at0 < a.rows) take(k % S, (k & 1) * kPlace);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < H; ++k) {
                unf2(dw2[i][k], dw[i * VEC + 2 * k], dw[i * VEC + 2 * k + 1]);
                unf2(db2[i][k], db[i * VEC + 2 * k], db[i * VEC + 2 * k + 1]);
            }
    } else {
        // (where there is room for them, the row that comes next has landed too, as above)
        constexpr bool AHEAD = Lay::S >= 3;
        int slot = 0, place = 0;
        float mean = 0.f;
#pragma unroll
        for (int k = 0; k < Lay::S - 1; ++k) issue(k);
        if constexpr (AHEAD) {
            asm volatile("cp.async.wait_group %0;" ::"n"(Lay::S - 2) : "memory");
            mean = r.sum(part_sum(landed(0)), kPlace) * a.inv_d;
        }
        for (; at0 < a.rows; at0 += step, row += step, y += step * a.ys) {
            issue(slot == 0 ? Lay::S - 1 : slot - 1);
            const Pack<T, VEC> *st = landed(slot);
            slot = slot + 1 == Lay::S ? 0 : slot + 1;
            if constexpr (!AHEAD) {
                asm volatile("cp.async.wait_group %0;" ::"n"(Lay::S - 1) : "memory");
                mean = r.sum(part_sum(st), 0) * a.inv_d;
                place = kPlace;
            }
            uint64_t p0 = twice(0.f), p1 = p0, p2 = p0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float x[VEC], g[VEC], w[VEC];
                deviations(st, i, mean, x);
                st[(NV + i) * TH].widen(g);
                if (EDGE) at.mask(i, g);
                weight[i].widen(w);
                add_products(x, x, p0);
                multiply(g, w, g);
                add_all(g, p1);
                add_products(g, x, p2);
            }
            float s0 = both(p0), s1 = both(p1), s2 = both(p2), next = 0.f;
            const float m = mean;
            if constexpr (AHEAD) {
                asm volatile("cp.async.wait_group %0;" ::"n"(Lay::S - 2) : "memory");
                next = part_sum(landed(slot));
            }
            r.sum4(s0, s1, s2, next, place);
            if constexpr (AHEAD) {
                mean = next * a.inv_d;
                place ^= kPlace;
            }
            if (row >= a.rows) continue;
            const float inv = rsqrtf(s0 * a.inv_d + a.eps);
            const float mg = -inv * s1 * a.inv_d, mh = -inv * inv * s2 * a.inv_d;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float x[VEC], g[VEC], w[VEC];
                deviations(st, i, m, x);
                st[(NV + i) * TH].widen(g);
                if (EDGE) at.mask(i, g);
                weight[i].widen(w);
                results(y, i, inv, mg, mh, x, g, w);
            }
        }
    }
    if (a.partial == nullptr) return;
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    for (int t = 0; t < 2; ++t) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                if (at.has(i, k)) sums[grp * a.d + at.col(i) + k] = t == 0 ? dw[i * VEC + k] : db[i * VEC + k];
        __syncthreads();
        float *out = a.partial + ((int64_t)blockIdx.x * 2 + t) * a.d;
        for (int j = (int)threadIdx.x; j < a.d; j += (int)blockDim.x) {
            float s = 0.f;
            for (int k = 0; k < groups; ++k) s += sums[k * a.d + j];
            out[j] = s;
        }
    }
}

// dw (blockIdx.y 0) and db: the blocks' sums, 32 interleaved chains joined in a
// fixed order.
__global__ void __launch_bounds__(1024) layer_norm_sums_kernel(const float *partial, int n, int d, float *dw, float *db) {
    __shared__ float sums[32][33];
    const int j = (int)(blockIdx.x * 32 + threadIdx.x);
    float *out = blockIdx.y == 0 ? dw : db;
    ptx::grid_wait();
    if (out == nullptr) return;
    float v = 0.f;
    if (j < d)
        for (int k = (int)threadIdx.y; k < n; k += 32) v += partial[((int64_t)k * 2 + blockIdx.y) * d + j];
    sums[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y == 0 && j < d) {
        v = 0.f;
        for (int k = 0; k < 32; ++k) v += sums[k][threadIdx.x];
        out[j] = v;
    }
}

}  // namespace norm
}  // namespace syn

using namespace syn;
using namespace syn::norm;

struct syn_norm_plan_s {
    syn_norm_cfg_t cfg;
    int device = 0, num_sms = 0;
    float *d_partial = nullptr;
};

namespace {

#define NORM_CK(call)                                                                                 \
    do {                                                                                              \
        cudaError_t e__ = (call);                                                                     \
        if (e__ != cudaSuccess) return host_fail(SYN_ERR_CUDA, std::string(#call) + ": " + cudaGetErrorString(e__)); \
    } while (0)

constexpr int kGradThreads = 512;
static_assert(kGradThreads <= kRowThreads, "places and barriers of a block's groups");
constexpr int kRowSteps = 3;  // rows of a group at least, for the persistent forward
constexpr int kGradElems = 16, kWideGradElems = 32;  // elements of a lane

int elem_size(int dtype) { return dtype == SYN_DTYPE_F32 ? 4 : 2; }

// How a call's rows may be read: 16-byte vectors from the row's first element, from
// the 16-byte boundary at or before it (where all its tensors' rows lie alike to
// these), or single elements.
enum Access { kVectors, kEdges, kElements };

// Elements from a 16-byte boundary to a row and from row to row
struct Lie {
    int off0, off1;
};
Lie lie_of(const void *p, int64_t row, int size) {
    const int64_t n = 16 / size;
    return {(int)((reinterpret_cast<uintptr_t>(p) & 15u) / (uintptr_t)size), (int)(((row % n) + n) % n)};
}

// Lanes of a row of n vectors with at most nv a lane
int lanes_for(int n, int nv) {
    const int l = (n + nv - 1) / nv;
    if (l > 32) return (l + 31) / 32 * 32;
    int p = 1;
    while (p < l) p *= 2;
    return p;
}

// Vectors of a row, the most that it may have
int vectors_of(int d, int vec, Access x) { return x == kEdges ? (d + 2 * vec - 2) / vec : (d + vec - 1) / vec; }

template <typename T, int VEC, int NV, bool EDGE> int launch_forward(Args &a, int n, cudaStream_t st) {
    a.lanes = lanes_for(n, NV);
    const int threads = a.lanes > 32 ? a.lanes : 128, per = threads / a.lanes;
    const int64_t grid = (a.rows + per - 1) / per;
    if (grid >= (int64_t)1 << 31) return host_fail(SYN_ERR_UNSUPPORTED, "too many rows in one call");
    NORM_CK((window::launch_early(layer_norm_kernel<T, VEC, NV, EDGE>, (unsigned)grid, (unsigned)threads, 0, st, a)));
    return SYN_OK;
}

int gcd(int a, int b) { return b == 0 ? a : gcd(b, a % b); }

// Blocks of `groups` rows each for all rows, at most one an SM.  With `edge`, rows of a
// group are to be a multiple of the period of their places apart.
int blocks_for(const syn_norm_plan_s *pl, const Args &a, int groups, bool edge, int vec) {
    int grid = (int)std::min<int64_t>((a.rows + groups - 1) / groups, pl->num_sms);
    if (edge) {
        const int period = vec / gcd(vec, a.off1), q = period / gcd(period, groups);
        grid = grid + q - 1 <= pl->num_sms ? (grid + q - 1) / q * q : std::max(pl->num_sms / q * q, q);
    }
    return grid;
}

template <typename T, int VEC, bool EDGE> int launch_rows(const syn_norm_plan_s *pl, Args &a, int n, cudaStream_t st) {
    a.lanes = lanes_for(n, kRowElems / VEC);
    const int groups = kRowThreads / a.lanes;
    NORM_CK((window::launch_early(layer_norm_rows_kernel<T, VEC, EDGE>, (unsigned)blocks_for(pl, a, groups, EDGE, VEC),
                                  (unsigned)(groups * a.lanes), (size_t)(kRowStages * kRowElems * kRowThreads * (int)sizeof(T)), st, a)));
    return SYN_OK;
}

template <typename T, int VEC, bool EDGE> int forward_of(const syn_norm_plan_s *pl, Args &a, cudaStream_t st) {
    // persistent blocks once a group of lanes has a few rows (a row a group instead: 55.4
    // against 45.6 us at 16384 rows of 4096, 17.2 against 16.8 at 5003 of 3584); else one
    // vector a lane while all rows together do not fill the SMs, then four (eight: 52.3
    // against 51.6 us at 16384 rows of 4096, 18.9 against 17.8 at 5003 of 3584)
    const int n = vectors_of(a.d, VEC, EDGE ? kEdges : kVectors), most = lanes_for(n, 1);
    if constexpr (VEC > 1)
        if (lanes_for(n, kRowElems / VEC) <= kRowThreads && a.rows * a.d >= (int64_t)pl->num_sms * kRowThreads * kRowElems * kRowSteps)
            return launch_rows<T, VEC, EDGE>(pl, a, n, st);
    if (a.rows * most <= (int64_t)pl->num_sms * 1024 && most <= 1024) return launch_forward<T, VEC, 1, EDGE>(a, n, st);
    if constexpr (VEC == 8) return launch_forward<T, VEC, 4, EDGE>(a, n, st);  // (2049 vectors at most)
    else if (n <= 4096) return launch_forward<T, VEC, 4, EDGE>(a, n, st);
    else return launch_forward<T, VEC, (VEC > 1 ? 8 : 16), EDGE>(a, n, st);
}

template <typename T> int forward_any(const syn_norm_plan_s *pl, Args &a, Access x, cudaStream_t st) {
    constexpr int V = 16 / (int)sizeof(T);
    return x == kVectors ? forward_of<T, V, false>(pl, a, st) : x == kEdges ? forward_of<T, V, true>(pl, a, st) : forward_of<T, 1, false>(pl, a, st);
}

template <typename T, int VEC, int E, int TH, bool EDGE>
int launch_grad(const syn_norm_plan_s *pl, Args &a, int n, cudaStream_t st, int &grid) {
    constexpr int NV = E / VEC;
    a.lanes = lanes_for(n, NV);
    const int groups = TH / a.lanes;
    grid = blocks_for(pl, a, groups, EDGE, VEC);
    NORM_CK((window::launch_early(layer_norm_grad_kernel<T, VEC, NV, TH, EDGE>, (unsigned)grid, (unsigned)(groups * a.lanes),
                                  (size_t)GradLay<T, VEC, NV, TH>::BYTES, st, a)));
    return SYN_OK;
}

template <typename T, int VEC, bool EDGE> int grad_of(const syn_norm_plan_s *pl, Args &a, cudaStream_t st, int &grid) {
    const int n = vectors_of(a.d, VEC, EDGE ? kEdges : kVectors);
    if (lanes_for(n, kGradElems / VEC) <= kGradThreads)
        return launch_grad<T, VEC, kGradElems, kGradThreads, EDGE>(pl, a, n, st, grid);
    return launch_grad<T, VEC, kWideGradElems, kGradThreads, EDGE>(pl, a, n, st, grid);
}

template <typename T> int grad_any(const syn_norm_plan_s *pl, Args &a, Access x, cudaStream_t st, int &grid) {
    constexpr int V = 16 / (int)sizeof(T);
    // (the widest rows may have a vector more than the lanes hold)
    if (x == kEdges && lanes_for(vectors_of(a.d, V, x), kWideGradElems / V) > kGradThreads) x = kElements;
    return x == kVectors ? grad_of<T, V, false>(pl, a, st, grid) : x == kEdges ? grad_of<T, V, true>(pl, a, st, grid)
                                                                               : grad_of<T, 1, false>(pl, a, st, grid);
}

// Shared memory that any call may need: set once, since the limit is the context's
template <typename T, int VEC, int E, int TH, bool EDGE> cudaError_t grad_prepare() {
    return cudaFuncSetAttribute(layer_norm_grad_kernel<T, VEC, E / VEC, TH, EDGE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                GradLay<T, VEC, E / VEC, TH>::BYTES);
}
template <typename T, int VEC, bool EDGE> cudaError_t both_prepare() {
    const cudaError_t e = grad_prepare<T, VEC, kGradElems, kGradThreads, EDGE>();
    return e != cudaSuccess ? e : grad_prepare<T, VEC, kWideGradElems, kGradThreads, EDGE>();
}
template <typename T> cudaError_t all_prepare() {
    constexpr int V = 16 / (int)sizeof(T);
    cudaError_t e = both_prepare<T, V, false>();
    if (e == cudaSuccess) e = both_prepare<T, V, true>();
    constexpr int bytes = kRowStages * kRowElems * kRowThreads * (int)sizeof(T);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(layer_norm_rows_kernel<T, V, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(layer_norm_rows_kernel<T, V, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    return e == cudaSuccess ? both_prepare<T, 1, false>() : e;
}

int check_rows(const char *name, const syn_norm_rows_t *r, int size, int64_t rows, int d, bool written) {
    if (r == nullptr || (rows > 0 && r->p == nullptr)) return host_fail(SYN_ERR_INVALID, std::string(name) + ": null operand");
    if (reinterpret_cast<uintptr_t>(r->p) % (uintptr_t)size != 0)
        return host_fail(SYN_ERR_INVALID, std::string(name) + ": operand not aligned to its element");
    if (rows > 1 && (r->row >= (int64_t)1 << 38 || r->row <= -((int64_t)1 << 38)))
        return host_fail(SYN_ERR_UNSUPPORTED, std::string(name) + ": stride of 2^38 elements or more");
    if (written && rows > 1 && std::abs(r->row) < d) return host_fail(SYN_ERR_INVALID, std::string(name) + ": output rows overlap");
    return SYN_OK;
}

// An output in the place of an input: a row's elements are written where they were read
int check_place(const char *name, const syn_norm_rows_t *in, const syn_norm_rows_t *out, int64_t rows) {
    if (rows > 1 && in->p == out->p && in->row != out->row)
        return host_fail(SYN_ERR_INVALID, std::string("in the place of ") + name + ": another row stride");
    return SYN_OK;
}

int check_vector(const char *name, const void *p, int size) {
    if (reinterpret_cast<uintptr_t>(p) % (uintptr_t)size != 0)
        return host_fail(SYN_ERR_INVALID, std::string(name) + ": operand not aligned to its element");
    return SYN_OK;
}

int check_call(const syn_norm_plan_s *pl, float eps, int64_t n_rows) {
    if (pl == nullptr) return host_fail(SYN_ERR_INVALID, "null plan");
    int device = -1;
    NORM_CK(cudaGetDevice(&device));
    if (device != pl->device) return host_fail(SYN_ERR_INVALID, "the plan belongs to another device than the current one");
    if (n_rows < 0) return host_fail(SYN_ERR_INVALID, "negative row count");
    if (n_rows >= (int64_t)1 << 31) return host_fail(SYN_ERR_UNSUPPORTED, "2^31 or more rows in one call");
    if (!(eps >= 0.f) || !std::isfinite(eps)) return host_fail(SYN_ERR_INVALID, "eps must be finite and not negative");
    return SYN_OK;
}

Args args_of(const syn_norm_plan_s *pl, float eps, int64_t n_rows) {
    Args a;
    std::memset(&a, 0, sizeof(a));
    a.rows = n_rows;
    a.d = pl->cfg.d;
    a.eps = eps;
    a.inv_d = 1.f / (float)a.d;
    return a;
}

// Access to the rows of up to three tensors, and the weights'; sets where they lie
Access access_of(Args &a, int size, std::initializer_list<Lie> rows, std::initializer_list<const void *> weights) {
    const Lie first = *rows.begin();
    for (const Lie &l : rows)
        if (l.off0 != first.off0 || l.off1 != first.off1) return kElements;
    a.off0 = first.off0;
    a.off1 = first.off1;
    bool whole = a.d % (16 / size) == 0 && first.off0 == 0 && first.off1 == 0;
    for (const void *w : weights) whole = whole && (reinterpret_cast<uintptr_t>(w) & 15u) == 0;
    return whole ? kVectors : kEdges;
}

}  // namespace

extern "C" {

int syn_norm_cfg_default(syn_norm_cfg_t *c) {
    if (c == nullptr) return host_fail(SYN_ERR_INVALID, "null cfg");
    std::memset(c, 0, sizeof(*c));
    c->dtype = SYN_DTYPE_BF16;
    c->d = 4096;
    return SYN_OK;
}

int syn_norm_plan_create(syn_norm_plan_t *out, const syn_norm_cfg_t *cfg) {
    if (out == nullptr || cfg == nullptr) return host_fail(SYN_ERR_INVALID, "null argument");
    *out = nullptr;
    if (cfg->dtype < SYN_DTYPE_BF16 || cfg->dtype > SYN_DTYPE_F32) return host_fail(SYN_ERR_INVALID, "unknown dtype");
    if (cfg->d < 1) return host_fail(SYN_ERR_INVALID, "d must be positive");
    if (cfg->d > kMaxD) return host_fail(SYN_ERR_UNSUPPORTED, "d > 16384");
    syn_norm_plan_s *pl = new (std::nothrow) syn_norm_plan_s();
    if (pl == nullptr) return host_fail(SYN_ERR_UNSUPPORTED, "not enough host memory");
    pl->cfg = *cfg;
    cudaError_t e = cudaGetDevice(&pl->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&pl->num_sms, cudaDevAttrMultiProcessorCount, pl->device);
    if (e == cudaSuccess)
        e = cfg->dtype == SYN_DTYPE_BF16 ? all_prepare<__nv_bfloat16>()
            : cfg->dtype == SYN_DTYPE_F16 ? all_prepare<__half>() : all_prepare<float>();
    if (e == cudaSuccess) e = cudaMalloc(&pl->d_partial, (size_t)pl->num_sms * 2 * (size_t)cfg->d * sizeof(float));
    if (e != cudaSuccess) {
        syn_norm_plan_destroy(pl);
        return host_fail(SYN_ERR_CUDA, std::string("norm plan: ") + cudaGetErrorString(e));
    }
    *out = pl;
    return SYN_OK;
}

int syn_norm_plan_destroy(syn_norm_plan_t pl) {
    if (pl == nullptr) return SYN_OK;
    cudaFree(pl->d_partial);
    delete pl;
    return SYN_OK;
}

int syn_layer_norm(syn_norm_plan_t pl, const syn_norm_rows_t *x, const void *w, const void *b, float eps,
                   const syn_norm_rows_t *y, int64_t n_rows, void *stream) {
    int rc = check_call(pl, eps, n_rows);
    if (rc != SYN_OK) return rc;
    const int size = elem_size(pl->cfg.dtype), d = pl->cfg.d;
    if ((rc = check_rows("x", x, size, n_rows, d, false)) != SYN_OK || (rc = check_rows("y", y, size, n_rows, d, true)) != SYN_OK ||
        (rc = check_place("x", x, y, n_rows)) != SYN_OK || (rc = check_vector("w", w, size)) != SYN_OK ||
        (rc = check_vector("b", b, size)) != SYN_OK)
        return rc;
    if (n_rows == 0) return SYN_OK;
    const int64_t xs = n_rows > 1 ? x->row : 0, ys = n_rows > 1 ? y->row : 0;
    Args a = args_of(pl, eps, n_rows);
    const Access how = access_of(a, size, {lie_of(x->p, xs, size), lie_of(y->p, ys, size)}, {w, b});
    a.x = x->p;
    a.y = y->p;
    a.w = w;
    a.b = b;
    a.xs = xs;
    a.ys = ys;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (pl->cfg.dtype == SYN_DTYPE_BF16) return forward_any<__nv_bfloat16>(pl, a, how, st);
    if (pl->cfg.dtype == SYN_DTYPE_F16) return forward_any<__half>(pl, a, how, st);
    return forward_any<float>(pl, a, how, st);
}

int syn_layer_norm_backward(syn_norm_plan_t pl, const syn_norm_rows_t *x, const syn_norm_rows_t *dy, const void *w,
                            float eps, const syn_norm_rows_t *dx, float *dw, float *db, int64_t n_rows, void *stream) {
    int rc = check_call(pl, eps, n_rows);
    if (rc != SYN_OK) return rc;
    const int size = elem_size(pl->cfg.dtype), d = pl->cfg.d;
    if ((rc = check_rows("x", x, size, n_rows, d, false)) != SYN_OK || (rc = check_rows("dy", dy, size, n_rows, d, false)) != SYN_OK ||
        (rc = check_rows("dx", dx, size, n_rows, d, true)) != SYN_OK || (rc = check_place("x", x, dx, n_rows)) != SYN_OK ||
        (rc = check_place("dy", dy, dx, n_rows)) != SYN_OK || (rc = check_vector("w", w, size)) != SYN_OK ||
        (rc = check_vector("dw", dw, 4)) != SYN_OK || (rc = check_vector("db", db, 4)) != SYN_OK)
        return rc;
    if (dw != nullptr && dw == db) return host_fail(SYN_ERR_INVALID, "dw and db are the same memory");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (n_rows == 0) {
        for (float *p : {dw, db})
            if (p != nullptr) NORM_CK(cudaMemsetAsync(p, 0, (size_t)d * sizeof(float), st));
        return SYN_OK;
    }
    const int64_t xs = n_rows > 1 ? x->row : 0, gs = n_rows > 1 ? dy->row : 0, ys = n_rows > 1 ? dx->row : 0;
    Args a = args_of(pl, eps, n_rows);
    const Access how = access_of(a, size, {lie_of(x->p, xs, size), lie_of(dy->p, gs, size), lie_of(dx->p, ys, size)}, {w});
    a.x = x->p;
    a.dy = dy->p;
    a.y = dx->p;
    a.w = w;
    a.xs = xs;
    a.gs = gs;
    a.ys = ys;
    // the plan's workspace belongs to the one call that wants weight gradients
    const bool want = dw != nullptr || db != nullptr;
    a.partial = want ? pl->d_partial : nullptr;
    int grid = 0;
    rc = pl->cfg.dtype == SYN_DTYPE_BF16 ? grad_any<__nv_bfloat16>(pl, a, how, st, grid)
         : pl->cfg.dtype == SYN_DTYPE_F16 ? grad_any<__half>(pl, a, how, st, grid)
                                          : grad_any<float>(pl, a, how, st, grid);
    if (rc != SYN_OK || !want) return rc;
    NORM_CK((window::launch_early(layer_norm_sums_kernel, dim3((unsigned)(d + 31) / 32, 2), dim3(32, 32), 0, st, pl->d_partial,
                                  grid, d, dw, db)));
    return SYN_OK;
}

}  // extern "C"
