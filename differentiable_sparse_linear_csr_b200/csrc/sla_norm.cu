// Global norm of many tensors (the gradients of a training step) and their
// scaling to a bound:
//   norm = sqrt(sum g^2) or max |g|;   dst = src * min(1, max_norm / (norm + 1e-6)).
// Bound by memory: the norm reads every element once, the scaling reads and
// writes them once more.  The tensors' addresses travel in the kernel
// arguments, so a call needs no copy and can be captured.  Pass 1 leaves one
// partial result a block in the workspace; every block of pass 2 adds them up
// in the same fixed order, so equal calls give equal bits without atomics.
// 200 M float32 elements: norm 117 us (6.8 TB/s), scaling 264 us (6.1 TB/s); 62
// tensors of odd sizes, 12 M elements: 10 and 13 us.  Pass 2 walks the chunks
// backwards: what pass 1 read last is still in L2.
// Squares are summed in 64 bits whatever the type: the square of a 32-bit or
// bfloat16 number need not be one.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <new>
#include <vector>

#include "sla_common.cuh"

namespace sla {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormLoads = 4;                                    // 16-byte loads of a thread in flight
constexpr int kChunkBytes = kNormThreads * kNormLoads * 16;      // what a block takes at a time
constexpr int kMaxPartials = 2048;

enum { kNormL2 = 0, kNormMax = 1 };

// What one launch takes (its arguments: a call with two tensors pays nothing for the
// unused ones).
constexpr int kTable = 256;
struct Table {
    int n;
    unsigned chunk0[kTable + 1];    // first chunk of each tensor
    const void *src[kTable];
    void *dst[kTable];
    int64_t count[kTable];
    uint8_t dtype[kTable];
};

template <typename T> __device__ __forceinline__ double wide(T x) {
    if constexpr (std::is_same_v<T, __nv_bfloat16>) return (double)__bfloat162float(x);
    else if constexpr (std::is_same_v<T, __half>) return (double)__half2float(x);
    else return (double)x;
}

template <typename T, int KIND>
__device__ __forceinline__ void take(double &s, T x) {
    const double v = wide(x);
    if constexpr (KIND == kNormL2) s = fma(v, v, s);
    else s = (fabs(v) > s || v != v) ? fabs(v) : s;    // a NaN stays
}

template <int KIND>
__device__ __forceinline__ double join(double a, double b) {
    if constexpr (KIND == kNormL2) return a + b;
    else return a != a ? a : (b != b ? b : fmax(a, b));
}

template <typename T, int KIND>
__device__ __forceinline__ double chunk_norm(const T *p, int64_t count, int64_t e0, bool vec) {
    constexpr int V = 16 / sizeof(T), E = kChunkBytes / sizeof(T);
    double s = 0.0;
    if (vec && e0 + E <= count) {
        uint4 r[kNormLoads];
#pragma unroll
        for (int i = 0; i < kNormLoads; ++i)
            r[i] = *reinterpret_cast<const uint4 *>(p + e0 + (int64_t)(i * kNormThreads + threadIdx.x) * V);
#pragma unroll
        for (int i = 0; i < kNormLoads; ++i) {
            const T *x = reinterpret_cast<const T *>(&r[i]);
#pragma unroll
            for (int e = 0; e < V; ++e) take<T, KIND>(s, x[e]);
        }
        return s;
    }
    const int64_t end = e0 + E < count ? e0 + E : count;
    int64_t from = e0;
    if (vec) {                       // a tensor's last chunk: whole vectors, then what is left
        from = e0 + (end - e0) / V * V;
#pragma unroll
        for (int i = 0; i < kNormLoads; ++i) {
            const int64_t at = e0 + (int64_t)(i * kNormThreads + threadIdx.x) * V;
            if (at < from) {
                const uint4 r = *reinterpret_cast<const uint4 *>(p + at);
                const T *x = reinterpret_cast<const T *>(&r);
#pragma unroll
                for (int e = 0; e < V; ++e) take<T, KIND>(s, x[e]);
            }
        }
    }
#pragma unroll 4
    for (int64_t i = from + threadIdx.x; i < end; i += kNormThreads) take<T, KIND>(s, p[i]);
    return s;
}

template <int KIND>
__device__ __forceinline__ double block_join(double v, double *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = join<KIND>(v, __shfl_xor_sync(0xffffffffu, v, o));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
    if (lane == 0) red[warp] = v;
    __syncthreads();
    double s = red[0];
#pragma unroll
    for (int w = 1; w < kNormThreads / 32; ++w) s = join<KIND>(s, red[w]);
    return s;
}

__device__ __forceinline__ int tensor_of(const Table &t, unsigned chunk) {
    int lo = 0, hi = t.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.chunk0[mid] <= chunk) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <int KIND>
__device__ __forceinline__ double table_norm(const Table &t, unsigned first, unsigned stride) {
    double s = 0.0;
    for (unsigned c = first; c < t.chunk0[t.n]; c += stride) {
        const int k = tensor_of(t, c);
        const int64_t at = (int64_t)(c - t.chunk0[k]) * kChunkBytes;
        const bool vec = ((uintptr_t)t.src[k] & 15) == 0;
        double v;
        switch (t.dtype[k]) {
            case SLA_F64: v = chunk_norm<double, KIND>((const double *)t.src[k], t.count[k], at / 8, vec); break;
            case SLA_F32: v = chunk_norm<float, KIND>((const float *)t.src[k], t.count[k], at / 4, vec); break;
            case SLA_BF16: v = chunk_norm<__nv_bfloat16, KIND>((const __nv_bfloat16 *)t.src[k], t.count[k], at / 2, vec); break;
            default: v = chunk_norm<__half, KIND>((const __half *)t.src[k], t.count[k], at / 2, vec); break;
        }
        s = join<KIND>(s, v);
    }
    return s;
}

template <int KIND>
__global__ void __launch_bounds__(kNormThreads) norm_partial_kernel(const __grid_constant__ Table t, double *part) {
    __shared__ double red[kNormThreads / 32];
    const double s = block_join<KIND>(table_norm<KIND>(t, blockIdx.x, gridDim.x), red);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// The norm from the partial results, the same in every block.
template <int KIND>
__device__ __forceinline__ double total_norm(const double *part, int n_part, double *red) {
    double s = 0.0;
    for (int i = threadIdx.x; i < n_part; i += kNormThreads) s = join<KIND>(s, part[i]);
    s = block_join<KIND>(s, red);
    return KIND == kNormL2 ? sqrt(s) : s;
}

__device__ __forceinline__ void store_norm(void *norm, int f64, double v) {
    if (f64) *static_cast<double *>(norm) = v;
    else *static_cast<float *>(norm) = (float)v;
}

template <int KIND>
__global__ void __launch_bounds__(kNormThreads) norm_finish_kernel(const double *part, int n_part, void *norm, int f64) {
    __shared__ double red[kNormThreads / 32];
    const double v = total_norm<KIND>(part, n_part, red);
    if (threadIdx.x == 0) store_norm(norm, f64, v);
}

// src * factor, in 64 bits for 64-bit tensors, else in 32.
template <typename T> __device__ __forceinline__ T scaled(T x, double f, float ff) {
    if constexpr (std::is_same_v<T, double>) return x * f;
    else if constexpr (std::is_same_v<T, float>) return x * ff;
    else if constexpr (std::is_same_v<T, __nv_bfloat16>) return __float2bfloat16_rn(__bfloat162float(x) * ff);
    else return __float2half_rn(__half2float(x) * ff);
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const T *p, T *q, int64_t count, int64_t e0, bool vec, double f) {
    constexpr int V = 16 / sizeof(T), E = kChunkBytes / sizeof(T);
    const float ff = (float)f;
    if (vec && e0 + E <= count) {
        uint4 r[kNormLoads];
#pragma unroll
        for (int i = 0; i < kNormLoads; ++i)
            r[i] = __ldcs(reinterpret_cast<const uint4 *>(p + e0 + (int64_t)(i * kNormThreads + threadIdx.x) * V));
#pragma unroll
        for (int i = 0; i < kNormLoads; ++i) {
            T *x = reinterpret_cast<T *>(&r[i]);
#pragma unroll
            for (int e = 0; e < V; ++e) x[e] = scaled<T>(x[e], f, ff);
            __stcs(reinterpret_cast<uint4 *>(q + e0 + (int64_t)(i * kNormThreads + threadIdx.x) * V), r[i]);
        }
        return;
    }
    const int64_t end = e0 + E < count ? e0 + E : count;
    int64_t from = e0;
    if (vec) {
        from = e0 + (end - e0) / V * V;
#pragma unroll
        for (int i = 0; i < kNormLoads; ++i) {
            const int64_t at = e0 + (int64_t)(i * kNormThreads + threadIdx.x) * V;
            if (at < from) {
                uint4 r = *reinterpret_cast<const uint4 *>(p + at);
                T *x = reinterpret_cast<T *>(&r);
#pragma unroll
                for (int e = 0; e < V; ++e) x[e] = scaled<T>(x[e], f, ff);
                *reinterpret_cast<uint4 *>(q + at) = r;
            }
        }
    }
#pragma unroll 4
    for (int64_t i = from + threadIdx.x; i < end; i += kNormThreads) q[i] = scaled<T>(p[i], f, ff);
}

// The chunks in the reverse of pass 1's order: the last ones read are the ones
// still in L2.
__device__ __forceinline__ void table_scale(const Table &t, unsigned first, unsigned stride, double f) {
    const unsigned n = t.chunk0[t.n];
    for (unsigned i = first; i < n; i += stride) {
        const unsigned c = n - 1 - i;
        const int k = tensor_of(t, c);
        if (f == 1.0 && t.src[k] == t.dst[k]) continue;
        const int64_t at = (int64_t)(c - t.chunk0[k]) * kChunkBytes;
        const bool vec = (((uintptr_t)t.src[k] | (uintptr_t)t.dst[k]) & 15) == 0;
        switch (t.dtype[k]) {
            case SLA_F64: chunk_scale<double>((const double *)t.src[k], (double *)t.dst[k], t.count[k], at / 8, vec, f); break;
            case SLA_F32: chunk_scale<float>((const float *)t.src[k], (float *)t.dst[k], t.count[k], at / 4, vec, f); break;
            case SLA_BF16: chunk_scale<__nv_bfloat16>((const __nv_bfloat16 *)t.src[k], (__nv_bfloat16 *)t.dst[k], t.count[k], at / 2, vec, f); break;
            default: chunk_scale<__half>((const __half *)t.src[k], (__half *)t.dst[k], t.count[k], at / 2, vec, f); break;
        }
    }
}

__device__ __forceinline__ double clip_factor(double norm, double max_norm) {
    const double f = max_norm / (norm + 1e-6);
    return f > 1.0 ? 1.0 : f;                       // a NaN norm gives a NaN factor
}

template <int KIND>
__global__ void __launch_bounds__(kNormThreads)
clip_scale_kernel(const __grid_constant__ Table t, const double *part, int n_part, double max_norm, void *norm,
                  int f64) {
    __shared__ double red[kNormThreads / 32];
    const double v = total_norm<KIND>(part, n_part, red);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) store_norm(norm, f64, v);
    table_scale(t, blockIdx.x, gridDim.x, clip_factor(v, max_norm));
}

// Both passes of a short list in one block: one launch, nothing to join.
template <int KIND>
__global__ void __launch_bounds__(kNormThreads)
clip_small_kernel(const __grid_constant__ Table t, double max_norm, void *norm, int f64) {
    __shared__ double red[kNormThreads / 32];
    double v = block_join<KIND>(table_norm<KIND>(t, 0, 1), red);
    if (KIND == kNormL2) v = sqrt(v);
    if (threadIdx.x == 0) store_norm(norm, f64, v);
    if (max_norm >= 0.0) table_scale(t, 0, 1, clip_factor(v, max_norm));
}

int fill(Table &t, const sla_tensor *list, int from, int n) {
    t.n = 0;
    t.chunk0[0] = 0;
    int i = from;
    for (; i < n && t.n < kTable; ++i) {
        if (list[i].count == 0) continue;
        const int64_t size = list[i].dtype == SLA_F64 ? 8 : (list[i].dtype == SLA_F32 ? 4 : 2);
        const int64_t chunks = (list[i].count * size + kChunkBytes - 1) / kChunkBytes;
        if ((int64_t)t.chunk0[t.n] + chunks > INT_MAX) break;
        t.src[t.n] = list[i].src;
        t.dst[t.n] = list[i].dst;
        t.count[t.n] = list[i].count;
        t.dtype[t.n] = (uint8_t)list[i].dtype;
        t.chunk0[t.n + 1] = t.chunk0[t.n] + (unsigned)chunks;
        ++t.n;
    }
    return i;
}

int num_sms() {
    int dev = 0, n = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n;
}

// Chunks that one block takes alone.  Clipping 1, 2, 4 and 8 chunks of float32: 2.2, 2.9,
// 4.6 and 7.3 us against 4.0 to 4.4 for two launches.  At 4 chunks the device loses 0.2
// to 0.6 us, and the host saves a launch of about 4.
constexpr int kSmallChunks = 4;

// Pass 1 over the list, tables of kTable tensors at a time; then the norm alone, or
// pass 2.  Partial results: at most kMaxPartials a table.
template <int KIND>
sla_status run_norm(const sla_tensor *list, int n, bool clip, double max_norm, void *norm, int f64, double *part,
                    cudaStream_t s) {
    Table t;
    if (fill(t, list, 0, n) == n && t.chunk0[t.n] <= (unsigned)kSmallChunks) {
        clip_small_kernel<KIND><<<1, kNormThreads, 0, s>>>(t, clip ? max_norm : -1.0, norm, f64);
        SLA_CHECK_LAUNCH();
        return SLA_OK;
    }
    const unsigned most = std::min(kMaxPartials, num_sms() * 8);
    int n_part = 0;
    for (int i = 0; i < n;) {
        i = fill(t, list, i, n);
        if (t.n == 0) break;
        const unsigned grid = std::min(t.chunk0[t.n], most);
        norm_partial_kernel<KIND><<<grid, kNormThreads, 0, s>>>(t, part + n_part);
        SLA_CHECK_LAUNCH();
        n_part += (int)grid;
    }
    if (!clip) {
        norm_finish_kernel<KIND><<<1, kNormThreads, 0, s>>>(part, n_part, norm, f64);
        SLA_CHECK_LAUNCH();
        return SLA_OK;
    }
    bool first = true;
    for (int i = 0; i < n;) {
        i = fill(t, list, i, n);
        if (t.n == 0) break;
        const unsigned grid = std::min(t.chunk0[t.n], most);
        clip_scale_kernel<KIND><<<grid, kNormThreads, 0, s>>>(t, part, n_part, max_norm, first ? norm : nullptr, f64);
        SLA_CHECK_LAUNCH();
        first = false;
    }
    return SLA_OK;
}

size_t norm_ws(int64_t n) { return align_up((size_t)(n / kTable + 1) * kMaxPartials * sizeof(double)); }

int64_t bytes_of(const sla_tensor &t) {
    return t.count * (t.dtype == SLA_F64 ? 8 : (t.dtype == SLA_F32 ? 4 : 2));
}

// No two outputs may share memory, nor an output and another tensor's input
// (an output may be its own input).  Returns the first offending index or -1.
int find_overlap(const sla_tensor *list, int n, std::vector<int> &order) {
    order.clear();
    for (int i = 0; i < n; ++i)
        if (list[i].count > 0) order.push_back(i);
    auto begin = [&](int i) { return (uintptr_t)list[i].dst; };
    auto end = [&](int i) { return (uintptr_t)list[i].dst + (uintptr_t)bytes_of(list[i]); };
    std::sort(order.begin(), order.end(), [&](int a, int b) { return begin(a) < begin(b); });
    for (size_t k = 1; k < order.size(); ++k)
        if (begin(order[k]) < end(order[k - 1])) return order[k];
    for (int i : order) {
        const uintptr_t s0 = (uintptr_t)list[i].src, s1 = s0 + (uintptr_t)bytes_of(list[i]);
        // the outputs are disjoint, so their ends are sorted too
        auto it = std::upper_bound(order.begin(), order.end(), s0, [&](uintptr_t x, int j) { return x < end(j); });
        for (; it != order.end() && begin(*it) < s1; ++it)
            if (*it != i || begin(i) != s0) return i;
    }
    return -1;
}

sla_status check_list(const char *fn, int32_t n, const sla_tensor *list, int32_t kind, int32_t norm_dtype, void *norm,
                      const void *ws, size_t ws_bytes, bool clip) {
    SLA_REQUIRE(n >= 0, "%s: negative count %d", fn, n);
    SLA_REQUIRE(n == 0 || list, "%s: NULL list", fn);
    SLA_REQUIRE(kind == SLA_NORM_L2 || kind == SLA_NORM_MAX, "%s: unknown norm %d", fn, kind);
    SLA_REQUIRE(norm_dtype == SLA_F64 || norm_dtype == SLA_F32, "%s: the norm is SLA_F64 or SLA_F32 (got %d)", fn,
                norm_dtype);
    SLA_REQUIRE(norm != nullptr, "%s: NULL norm", fn);
    for (int i = 0; i < n; ++i) {
        SLA_REQUIRE(list[i].dtype >= SLA_F64 && list[i].dtype <= SLA_F16, "%s: bad dtype %lld of tensor %d", fn,
                    (long long)list[i].dtype, i);
        SLA_REQUIRE(list[i].count >= 0 && list[i].count < (int64_t)1 << 45, "%s: bad count %lld of tensor %d", fn,
                    (long long)list[i].count, i);
        SLA_REQUIRE(list[i].count == 0 || (list[i].src && (!clip || list[i].dst)), "%s: NULL pointer of tensor %d", fn, i);
        const uintptr_t size = list[i].dtype == SLA_F64 ? 8 : (list[i].dtype == SLA_F32 ? 4 : 2);
        SLA_REQUIRE((uintptr_t)list[i].src % size == 0 && (!clip || (uintptr_t)list[i].dst % size == 0),
                    "%s: tensor %d is not aligned to its elements", fn, i);
    }
    SLA_REQUIRE(ws && ws_bytes >= norm_ws(n), "%s: workspace too small (%zu < %zu)", fn, ws_bytes, norm_ws(n));
    SLA_REQUIRE(((uintptr_t)ws & 255) == 0, "%s: workspace must be 256-byte aligned", fn);
    return SLA_OK;
}

}  // namespace
}  // namespace sla

using namespace sla;

extern "C" size_t sla_norm_workspace_bytes(int32_t n) { return n < 0 ? 0 : norm_ws(n); }

extern "C" sla_status sla_global_norm(int32_t n, const sla_tensor *list, int32_t kind, void *norm, int32_t norm_dtype,
                                      void *ws, size_t ws_bytes, void *stream) {
    SLA_RANGE("sla_global_norm");
    clear_error();
    sla_status st = check_list("sla_global_norm", n, list, kind, norm_dtype, norm, ws, ws_bytes, false);
    if (st != SLA_OK) return st;
    double *part = static_cast<double *>(ws);
    const int f64 = norm_dtype == SLA_F64;
    if (kind == SLA_NORM_L2) return run_norm<kNormL2>(list, n, false, 0.0, norm, f64, part, as_stream(stream));
    return run_norm<kNormMax>(list, n, false, 0.0, norm, f64, part, as_stream(stream));
}

extern "C" sla_status sla_clip_norm(int32_t n, const sla_tensor *list, int32_t kind, double max_norm, void *norm,
                                    int32_t norm_dtype, void *ws, size_t ws_bytes, void *stream) {
    SLA_RANGE("sla_clip_norm");
    clear_error();
    SLA_REQUIRE(max_norm >= 0.0 && max_norm <= DBL_MAX, "sla_clip_norm: max_norm must be finite and not negative");
    sla_status st = check_list("sla_clip_norm", n, list, kind, norm_dtype, norm, ws, ws_bytes, true);
    if (st != SLA_OK) return st;
    int bad = -1;
    try {
        std::vector<int> order;
        bad = find_overlap(list, n, order);
    } catch (const std::bad_alloc &) {
        set_error("sla_clip_norm: out of host memory");
        return SLA_ERR_OOM;
    }
    SLA_REQUIRE(bad < 0, "sla_clip_norm: the output of tensor %d shares memory with another tensor", bad);
    double *part = static_cast<double *>(ws);
    const int f64 = norm_dtype == SLA_F64;
    if (kind == SLA_NORM_L2) return run_norm<kNormL2>(list, n, true, max_norm, norm, f64, part, as_stream(stream));
    return run_norm<kNormMax>(list, n, true, max_norm, norm, f64, part, as_stream(stream));
}
