// clip.cu -- the global 2-norm of many tensors and clipping by it (C ABI:
// include/syn_clip.h).
//
// The list of tensors travels in a launch's arguments, so that a call copies
// nothing to the device and can be captured; up to kMany tensors a launch.  The
// tensors are cut into chunks of kVecs vectors and dealt out to persistent
// blocks in turn.  One pass reads every element for the norm; the block that ends
// last joins the blocks' sums in their order.  A second pass, from the last chunk
// to the first so that what the first read last still comes from L2, reads and
// writes every element.
//
// Measured on one GB300: nine fp32 tensors, 872 MB, 411-420 us (norm 150, products 264),
// 6.3 TB/s of the three passes' bytes: HBM bounds both.  24 tensors of 0.4 MB in all
// take 10.4 us in a graph, two launches' time, and 24.5-27 with the host side.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <new>
#include <string>
#include <utility>
#include <vector>

#include "elements.cuh"
#include "host_util.h"
#include "syn.h"
#include "syn_clip.h"
#include "window.cuh"

namespace syn {
namespace clip {

using elem::Num;
using elem::Pack;

constexpr int kThreads = 256, kUnroll = 4;       // vectors that a thread has under way
constexpr int kVecs = 2 * kThreads * kUnroll;    // vectors of 16 bytes of a chunk
constexpr int kBlocksPerSm = 4, kNormBlocksPerSm = 6;
constexpr int kFew = 32, kMany = 1024;           // tensors of a launch (1 and 28 KB of arguments)
constexpr int kMaxLaunches = 64;

struct Sums {                    // a plan's workspace
    double total;                // sum of squares of all tensors
    uint32_t arrived, pad;
};

template <int N> struct Args {
    const void *x[N];
    void *y[N];
    int64_t n[N];
    uint32_t chunk0[N + 1];      // first chunk of each tensor
    uint8_t dtype[N];
    int32_t n_tensors, n_before; // partial sums of the launches before
    double *partial;
    Sums *sums;
    float *norm;                 // the last launch of the first pass: nullable
    float max_norm, eps;
    int32_t last;
};

// The tensor that chunk c lies in
template <int N> __device__ __forceinline__ int tensor_of(const Args<N> &a, uint32_t c) {
    int lo = 0, hi = a.n_tensors - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (a.chunk0[mid] <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Where a tensor's 16-byte vectors begin: elements before the first one, vectors,
// elements behind the last
struct Split {
    int64_t head, vecs, tail;
    __device__ __forceinline__ Split(const void *p, int64_t n, int size) {
        const int64_t want = (int64_t)((16 - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / size;
        head = want < n ? want : n;
        vecs = (n - head) / (16 / size);
        tail = n - head - vecs * (16 / size);
    }
};

template <typename T> struct Vec {
    static constexpr int N = 16 / (int)sizeof(T);
    static __device__ __forceinline__ void widen(const uint4 &v, float (&e)[N]) {
        Pack<T, N> p;
        p.v = v;
        p.widen(e);
    }
};

// Sum of squares of a thread's vectors from `at` on, where they leave fp32's range:
// the elements are scaled by a power of two that brings the largest to about one.
// (Out of line: inline its registers cost the loop's blocks.  Vectors of zeros come here
// too and are read a second time: the norm of 176 million takes 113 us in fp32 for 104 of
// other values, 64 for 56 in bf16.)
template <typename T> __device__ __noinline__ double scaled_squares(const uint4 *q, int at, int end) {
    constexpr int N = Vec<T>::N;
    float top = 0.f;
    for (int u = 0; u < kUnroll && at + u * kThreads < end; ++u) {
        float e[N];
        Vec<T>::widen(q[at + u * kThreads], e);
        for (int i = 0; i < N; ++i) top = fmaxf(top, fabsf(e[i]));
    }
    if (top == 0.f) return 0.0;
    if (isinf(top)) return (double)top;
    const int k = ilogbf(top);
    float s = 0.f;
    for (int u = 0; u < kUnroll && at + u * kThreads < end; ++u) {
        float e[N];
        Vec<T>::widen(q[at + u * kThreads], e);
        for (int i = 0; i < N; ++i) {
            const float x = scalbnf(e[i], -k);
            s = fmaf(x, x, s);
        }
    }
    return scalbn((double)s, 2 * k);
}

template <typename T> __device__ __forceinline__ double chunk_squares(const void *x, int64_t n, uint32_t chunk) {
    constexpr int N = Vec<T>::N;
    const Split sp(x, n, (int)sizeof(T));
    const T *p = static_cast<const T *>(x) + sp.head;
    const uint4 *q = reinterpret_cast<const uint4 *>(p) + (int64_t)chunk * kVecs;
    const int end = (int)min((int64_t)kVecs, sp.vecs - (int64_t)chunk * kVecs);
    double s = 0.0;
#pragma unroll 1
    for (int at = (int)threadIdx.x; at < end; at += kThreads * kUnroll) {
        uint4 v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) v[u] = at + u * kThreads < end ? q[at + u * kThreads] : make_uint4(0, 0, 0, 0);
        float f = 0.f;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            float e[N];
            Vec<T>::widen(v[u], e);
#pragma unroll
            for (int i = 0; i < N; ++i) f = fmaf(e[i], e[i], f);
        }
        // below 2^-80 a square that was lost to the subnormals would show (NaN stays)
        s += (f < 3.0e38f && f > 8.3e-25f) || f != f ? (double)f : scaled_squares<T>(q, at, end);
    }
    if (chunk == 0 && threadIdx.x < 2 * N) {  // the ends, an element a thread
        const int i = (int)threadIdx.x;
        const T *e = nullptr;
        if (i < N && i < sp.head) e = static_cast<const T *>(x) + i;
        if (i >= N && i - N < sp.tail) e = p + sp.vecs * N + (i - N);
        if (e != nullptr) {
            const double d = (double)Num<T>::get(*e);
            s += d * d;
        }
    }
    return s;
}

template <int N> __global__ void __launch_bounds__(kThreads, kNormBlocksPerSm) grad_norm_kernel(const __grid_constant__ Args<N> a) {
    __shared__ double part[kThreads / 32];
    __shared__ bool last;
    ptx::grid_wait();
    double s = 0.0;
    const uint32_t chunks = a.chunk0[a.n_tensors];
    for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int t = tensor_of(a, c);
        const uint32_t at = c - a.chunk0[t];
        if (a.dtype[t] == SYN_DTYPE_F32) s += chunk_squares<float>(a.x[t], a.n[t], at);
        else if (a.dtype[t] == SYN_DTYPE_BF16) s += chunk_squares<__nv_bfloat16>(a.x[t], a.n[t], at);
        else s += chunk_squares<__half>(a.x[t], a.n[t], at);
    }
    auto block_sum = [&](double v) {  // in thread 0
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if ((threadIdx.x & 31u) == 0) part[threadIdx.x / 32] = v;
        __syncthreads();
        v = 0.0;
        for (int i = 0; i < kThreads / 32; ++i) v += part[i];
        return v;
    };
    s = block_sum(s);
    const int n = a.n_before + (int)gridDim.x;
    if (threadIdx.x == 0) {
        __stcg(a.partial + a.n_before + blockIdx.x, s);
        __threadfence();
        last = ptx::atom_add_acq_rel_gpu(&a.sums->arrived, 1u) == gridDim.x - 1u;
        if (last) a.sums->arrived = 0u;  // for the next launch
        __threadfence();
    }
    __syncthreads();
    if (!last || !a.last) return;
    s = 0.0;
    for (int i = (int)threadIdx.x; i < n; i += kThreads) s += __ldcg(a.partial + i);
    __syncthreads();  // (part has been read)
    s = block_sum(s);
    if (threadIdx.x == 0) {
        a.sums->total = s;
        if (a.norm != nullptr) *a.norm = (float)sqrt(s);
    }
}

// The factor c, as c * back where fp32 would hold it as a subnormal (a norm above
// 2^126 max_norm): back is a power of two, so its product is exact.
struct Factor {
    float c, back;
    __device__ __forceinline__ float operator()(float x) const { return x * c * back; }
};

// A chunk's products where the two pointers lie differently to 16-byte boundaries:
// element by element, the ends in the first and the last chunk
template <typename T> __device__ __noinline__ void scale_apart(const T *x, T *y, int64_t n, uint32_t chunk, Factor c) {
    constexpr int N = Vec<T>::N;
    const Split sp(x, n, (int)sizeof(T));
    const int64_t per = (int64_t)kVecs * N, stop = sp.head + ((int64_t)chunk + 1) * per;
    const int64_t hi = stop >= sp.head + sp.vecs * N ? n : stop;
    for (int64_t i = (chunk == 0 ? 0 : sp.head + chunk * per) + threadIdx.x; i < hi; i += kThreads) y[i] = Num<T>::put(c(Num<T>::get(x[i])));
}

// A chunk's products
template <typename T> __device__ __forceinline__ void scale_chunk(const void *x, void *y, int64_t n, uint32_t chunk, const Factor &c) {
    constexpr int N = Vec<T>::N;
    const T *px = static_cast<const T *>(x);
    T *py = static_cast<T *>(y);
    if (((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(y)) & 15u) != 0) {
        scale_apart(px, py, n, chunk, c);
        return;
    }
    const Split sp(x, n, (int)sizeof(T));
    const uint4 *q = reinterpret_cast<const uint4 *>(px + sp.head) + (int64_t)chunk * kVecs;
    uint4 *o = reinterpret_cast<uint4 *>(py + sp.head) + (int64_t)chunk * kVecs;
    const int end = (int)min((int64_t)kVecs, sp.vecs - (int64_t)chunk * kVecs);
#pragma unroll 1
    for (int at = (int)threadIdx.x; at < end; at += kThreads * kUnroll) {
        uint4 v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (at + u * kThreads < end) v[u] = __ldcs(q + at + u * kThreads);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (at + u * kThreads >= end) continue;
            float e[N];
            Vec<T>::widen(v[u], e);
#pragma unroll
            for (int i = 0; i < N; ++i) e[i] = c(e[i]);
            Pack<T, N> p;
            p.narrow(e);
            __stcs(o + at + u * kThreads, p.v);
        }
    }
    if (chunk == 0 && threadIdx.x < 2 * N) {
        const int i = (int)threadIdx.x;
        int64_t j = -1;
        if (i < N && i < sp.head) j = i;
        if (i >= N && i - N < sp.tail) j = sp.head + sp.vecs * N + (i - N);
        if (j >= 0) py[j] = Num<T>::put(c(Num<T>::get(px[j])));
    }
}

template <int N> __global__ void __launch_bounds__(kThreads, kBlocksPerSm) grad_scale_kernel(const __grid_constant__ Args<N> a) {
    __shared__ Factor factor;
    ptx::grid_wait();
    if (threadIdx.x == 0) {
        const double total = a.sums->total, q = (double)a.max_norm / (sqrt(total) + (double)a.eps);
        const bool tiny = q < 1.2e-38;
        factor.c = total == 0.0 || q >= 1.0 ? 1.f : tiny ? (float)(q * 0x1p64) : (float)q;  // (NaN stays)
        factor.back = tiny && total != 0.0 ? 0x1p-64f : 1.f;
    }
    __syncthreads();
    const Factor c = factor;
    const uint32_t chunks = a.chunk0[a.n_tensors];
    for (uint32_t i = blockIdx.x; i < chunks; i += gridDim.x) {
        const uint32_t k = chunks - 1u - i;
        const int t = tensor_of(a, k);
        const uint32_t at = k - a.chunk0[t];
        if (c.c == 1.f && a.x[t] == a.y[t]) continue;  // every element keeps its bits
        if (a.dtype[t] == SYN_DTYPE_F32) scale_chunk<float>(a.x[t], a.y[t], a.n[t], at, c);
        else if (a.dtype[t] == SYN_DTYPE_BF16) scale_chunk<__nv_bfloat16>(a.x[t], a.y[t], a.n[t], at, c);
        else scale_chunk<__half>(a.x[t], a.y[t], a.n[t], at, c);
    }
}

}  // namespace clip
}  // namespace syn

using namespace syn;
using namespace syn::clip;

struct syn_clip_plan_s {
    int device = 0, num_sms = 0;
    Sums *d_sums = nullptr;
    double *d_partial = nullptr;
};

namespace {

#define CLIP_CK(call)                                                                                 \
    do {                                                                                              \
        cudaError_t e__ = (call);                                                                     \
        if (e__ != cudaSuccess) return host_fail(SYN_ERR_CUDA, std::string(#call) + ": " + cudaGetErrorString(e__)); \
    } while (0)

int elem_size(int dtype) { return dtype == SYN_DTYPE_F32 ? 4 : 2; }

// Chunks of a tensor (one at least, which does its ends)
int64_t chunks_of(const syn_clip_tensor_t &t) {
    const int size = elem_size(t.dtype);
    const int64_t head = std::min<int64_t>(t.n, (int64_t)((16 - (reinterpret_cast<uintptr_t>(t.x) & 15u)) & 15u) / size);
    const int64_t vecs = (t.n - head) / (16 / size), per = kVecs;
    return std::max<int64_t>((vecs + per - 1) / per, 1);
}

struct Span {
    uintptr_t lo, hi;
    bool written;
    bool operator<(const Span &o) const { return lo < o.lo; }
};

// Memory that is written may meet no other of the call
int check_overlap(const syn_clip_tensor_t *t, int n, const float *norm) {
    std::vector<Span> s;
    s.reserve((size_t)2 * (size_t)n + 1);
    bool sorted = true;
    auto add = [&](const void *p, int64_t bytes, bool written) {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        sorted = sorted && (s.empty() || s.back().lo <= lo);
        s.push_back({lo, lo + (uintptr_t)bytes, written});
    };
    for (int i = 0; i < n; ++i) {
        if (t[i].n == 0) continue;
        const int64_t bytes = t[i].n * elem_size(t[i].dtype);
        if (t[i].x != t[i].y) add(t[i].x, bytes, false);
        add(t[i].y, bytes, true);
    }
    if (norm != nullptr) add(norm, 4, true);
    if (!sorted) std::sort(s.begin(), s.end());
    uintptr_t any = 0, wrote = 0;  // the furthest ends so far, of all and of what is written
    for (const Span &x : s) {
        if (x.lo < wrote || (x.written && x.lo < any)) return host_fail(SYN_ERR_INVALID, "written memory overlaps other tensors of the call");
        any = std::max(any, x.hi);
        if (x.written) wrote = std::max(wrote, x.hi);
    }
    return SYN_OK;
}

int check_call(const syn_clip_plan_s *pl, const syn_clip_tensor_t *t, int n, bool clip, const float *norm) {
    if (pl == nullptr) return host_fail(SYN_ERR_INVALID, "null plan");
    int device = -1;
    CLIP_CK(cudaGetDevice(&device));
    if (device != pl->device) return host_fail(SYN_ERR_INVALID, "the plan belongs to another device than the current one");
    if (n < 0 || (n > 0 && t == nullptr)) return host_fail(SYN_ERR_INVALID, "need a list of n_tensors >= 0 tensors");
    if (n > kMany * kMaxLaunches) return host_fail(SYN_ERR_UNSUPPORTED, "more than 65536 tensors");
    if (reinterpret_cast<uintptr_t>(norm) % 4 != 0) return host_fail(SYN_ERR_INVALID, "norm: not aligned");
    for (int i = 0; i < n; ++i) {
        const syn_clip_tensor_t &x = t[i];
        if (x.dtype < SYN_DTYPE_BF16 || x.dtype > SYN_DTYPE_F32) return host_fail(SYN_ERR_INVALID, "unknown dtype of tensor " + std::to_string(i));
        if (x.n < 0) return host_fail(SYN_ERR_INVALID, "negative size of tensor " + std::to_string(i));
        if (x.n >= (int64_t)1 << 40) return host_fail(SYN_ERR_UNSUPPORTED, "2^40 or more elements in tensor " + std::to_string(i));
        if (x.n == 0) continue;
        const uintptr_t off = reinterpret_cast<uintptr_t>(x.x) | (clip ? reinterpret_cast<uintptr_t>(x.y) : 0);
        if (x.x == nullptr || (clip && x.y == nullptr)) return host_fail(SYN_ERR_INVALID, "null tensor " + std::to_string(i));
        if (off % (uintptr_t)elem_size(x.dtype) != 0) return host_fail(SYN_ERR_INVALID, "tensor " + std::to_string(i) + " not aligned to its element");
    }
    return clip ? check_overlap(t, n, norm) : SYN_OK;
}

// Launches over tensors [i0, i1), which do not have more than N
template <int N>
int launch(syn_clip_plan_s *pl, const syn_clip_tensor_t *t, int i0, int i1, bool scale, int &n_before, bool last, float *norm,
           float max_norm, float eps, cudaStream_t st) {
    Args<N> a;
    int k = 0;
    int64_t chunks = 0;
    for (int i = i0; i < i1; ++i) {
        if (t[i].n == 0) continue;
        a.x[k] = t[i].x;
        a.y[k] = t[i].y;
        a.n[k] = t[i].n;
        a.dtype[k] = (uint8_t)t[i].dtype;
        a.chunk0[k++] = (uint32_t)chunks;
        chunks += chunks_of(t[i]);
        if (chunks >= (int64_t)1 << 31) return host_fail(SYN_ERR_UNSUPPORTED, "2^31 or more chunks in one call");
    }
    a.chunk0[k] = (uint32_t)chunks;
    a.n_tensors = k;
    a.n_before = n_before;
    a.partial = pl->d_partial;
    a.sums = pl->d_sums;
    a.norm = norm;
    a.max_norm = max_norm;
    a.eps = eps;
    a.last = last;
    if (scale && k == 0) return SYN_OK;
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(chunks, (int64_t)pl->num_sms * (scale ? kBlocksPerSm : kNormBlocksPerSm)));
    n_before += grid;
    if (scale)
        CLIP_CK((window::launch_early(grad_scale_kernel<N>, (unsigned)grid, kThreads, 0, st, a)));
    else
        CLIP_CK((window::launch_early(grad_norm_kernel<N>, (unsigned)grid, kThreads, 0, st, a)));
    return SYN_OK;
}

int run(syn_clip_plan_s *pl, const syn_clip_tensor_t *t, int n, bool clip, float max_norm, float eps, float *norm, cudaStream_t st) {
    int before = 0, rc = SYN_OK;
    for (int i = 0; rc == SYN_OK && (i == 0 || i < n); i += kMany) {
        const int end = std::min(n, i + kMany);
        const bool last = end >= n;
        rc = end - i <= kFew ? launch<kFew>(pl, t, i, end, false, before, last, norm, max_norm, eps, st)
                             : launch<kMany>(pl, t, i, end, false, before, last, norm, max_norm, eps, st);
    }
    // (the last tensors first, which the norm read last)
    for (int i = (n - 1) / kMany * kMany; clip && rc == SYN_OK && i >= 0 && n > 0; i -= kMany) {
        const int end = std::min(n, i + kMany);
        rc = end - i <= kFew ? launch<kFew>(pl, t, i, end, true, before, true, norm, max_norm, eps, st)
                             : launch<kMany>(pl, t, i, end, true, before, true, norm, max_norm, eps, st);
    }
    return rc;
}

}  // namespace

extern "C" {

int syn_clip_plan_create(syn_clip_plan_t *out) {
    if (out == nullptr) return host_fail(SYN_ERR_INVALID, "null argument");
    *out = nullptr;
    syn_clip_plan_s *pl = new (std::nothrow) syn_clip_plan_s();
    if (pl == nullptr) return host_fail(SYN_ERR_UNSUPPORTED, "not enough host memory");
    cudaError_t e = cudaGetDevice(&pl->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&pl->num_sms, cudaDevAttrMultiProcessorCount, pl->device);
    if (e == cudaSuccess) e = cudaMalloc(&pl->d_sums, sizeof(Sums));
    if (e == cudaSuccess)
        e = cudaMalloc(&pl->d_partial, (size_t)pl->num_sms * kNormBlocksPerSm * kMaxLaunches * sizeof(double));
    if (e == cudaSuccess) e = cudaMemset(pl->d_sums, 0, sizeof(Sums));
    // (the clearing may return before it has reached the device, which other streams would not wait for)
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) {
        syn_clip_plan_destroy(pl);
        return host_fail(SYN_ERR_CUDA, std::string("clip plan: ") + cudaGetErrorString(e));
    }
    *out = pl;
    return SYN_OK;
}

int syn_clip_plan_destroy(syn_clip_plan_t pl) {
    if (pl == nullptr) return SYN_OK;
    cudaFree(pl->d_sums);
    cudaFree(pl->d_partial);
    delete pl;
    return SYN_OK;
}

int syn_grad_norm(syn_clip_plan_t pl, const syn_clip_tensor_t *tensors, int n, float *norm, void *stream) {
    const int rc = check_call(pl, tensors, n, false, norm);
    if (rc != SYN_OK) return rc;
    if (norm == nullptr) return host_fail(SYN_ERR_INVALID, "null norm");
    return run(pl, tensors, n, false, 0.f, 0.f, norm, static_cast<cudaStream_t>(stream));
}

int syn_grad_clip(syn_clip_plan_t pl, const syn_clip_tensor_t *tensors, int n, float max_norm, float eps, float *norm,
                  void *stream) try {
    if (!(max_norm >= 0.f)) return host_fail(SYN_ERR_INVALID, "max_norm must not be negative or NaN");
    if (!(eps >= 0.f) || !std::isfinite(eps)) return host_fail(SYN_ERR_INVALID, "eps must be finite and not negative");
    const int rc = check_call(pl, tensors, n, true, norm);
    if (rc != SYN_OK) return rc;
    return run(pl, tensors, n, true, max_norm, eps, norm, static_cast<cudaStream_t>(stream));
} catch (const std::bad_alloc &) {  // (the list of overlaps grows with the tensors)
    return host_fail(SYN_ERR_UNSUPPORTED, "not enough host memory for the list of tensors");
}

}  // extern "C"
