// Internals shared by the attention kernels: parameters, the plan that splits a
// pattern's rows into work items, element loads and the partial results of
// split rows.
//
//   s_t = scale * q_i . k_j + vals_t      for entry t = (i, j) of row i
//   p_t = exp(s_t - m_i) / l_i,  l_i = sum_t exp(s_t - m_i),  o_i = sum_t p_t v_j
// with a reference m_i near the row's maximum (lse_i = m_i + log l_i).  The backward
// needs m and l apart: beside a large m their sum holds little or nothing of log l.
// Backwards, with D_i = do_i . o_i:
//   ds_t = p_t (do_i . v_j - D_i),  dq_i = scale sum_t ds_t k_j,
//   dk_j = scale sum_t ds_t q_i,    dv_j = sum_t p_t do_i,  dvals_t = sum_heads ds_t.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <vector>

#include "sla_common.cuh"

namespace sla {

// Work items of one direction of a pattern: a unit is `rows` consecutive rows;
// a unit longer than seg_len (entries of its row; chunks of its tile) is split
// into several items (segments), whose partial results a second kernel joins.
// Null item arrays: item == unit, one segment each.
struct AttnPlan {
    bool built = false;
    int32_t rows = 1, n_units = 0, n_items = 0, n_slots = 0, n_multi = 0, seg_len = 0, most_segs = 1;
    int32_t *item_unit = nullptr, *item_seg = nullptr, *item_slot = nullptr;   // [n_items]
    int2 *item_chunks = nullptr;       // tiles: [n_items] first and last (excluded) chunk
    int32_t *multi_unit = nullptr;                                             // [n_multi]
    int32_t *multi_slot = nullptr;                                             // [n_multi + 1]
};

// The tiles of one direction: the columns that any row of a tile stores, in
// increasing order, 16 to a chunk.  A tile is the left side of a 16-row matrix
// product: 16 rows, or fewer rows with several of the query heads that share a key
// head (A: 16 / 2^k rows with 2^k heads).  A^T's tiles have 16 rows always, and every
// column 2^k times in a row, once for each of those heads.
struct AttnTiles {
    bool built = false;
    int32_t *chunk0 = nullptr;         // [n_units + 1]: first chunk of each tile
    struct TileChunk *chunks = nullptr;
};
struct TileChunk {
    int32_t col[16];                   // a tile's last chunk is padded with valid columns
    uint16_t bits[16];                 // row r of the tile: the columns it stores
    int32_t start[16];                 // row r: its first entry in this chunk
};

constexpr int kTileRows = 16;
// How finely long rows are split depends on how many systems and heads share
// the GPU: a plan for few, some and many of them.
constexpr int kAttnLevels = 3;

constexpr int kTileKinds = 5;          // k = 0 to 4

struct AttnPlans {
    AttnPlan row[2][kAttnLevels];      // one row a unit: A, A^T
    AttnPlan tile[2][kTileKinds][kAttnLevels];
    AttnTiles tiles[2][kTileKinds];
};

// The kind k of tiles with 2^k query heads together: the largest power of two that
// divides the heads sharing a key head.
inline int attn_tile_kind(const sla_attn_opts *o) {
    const int share = o->heads / o->kv_heads;
    int k = 0;
    while (k < kTileKinds - 1 && share % (2 << k) == 0) ++k;
    return k;
}

// 16-bit heads of whole 16-element steps go through the tensor cores.
inline bool attn_tiled(const sla_attn_opts *o) {
    return (o->dtype == SLA_BF16 || o->dtype == SLA_F16) && o->dim % 16 == 0 && o->dim <= 128;
}

inline int attn_level(const Csr *h, const sla_attn_opts *o) {
    const int64_t share = (int64_t)h->batch * (attn_tiled(o) ? o->heads >> attn_tile_kind(o) : o->heads);
    return share >= 64 ? 2 : (share >= 8 ? 1 : 0);
}

// What every kernel gets (strides in elements, heads of `dim` consecutive elements).
struct AttnArgs {
    int32_t n_rows, n_cols, batch, heads, kv_heads, dim;
    int64_t nnz;
    double scale;
    const int32_t *rowptr, *colind, *perm;
    int32_t n_items, n_slots, seg_len;
    const int32_t *item_unit, *item_seg, *item_slot;
    int32_t rows_log;                      // tiles: rows of one of A's, as a power of two (4 - kind)
    const int32_t *chunk0;                 // chunks of each unit, and of each item of a split plan
    const int2 *item_chunks;
    const TileChunk *chunks;
    const void *q, *k, *v, *o, *dout;
    int64_t qs[3], ks[3], vs[3], ds[3];    // system, row, head
    const void *vals;
    int32_t vals_f64;
    void *out, *wide, *lse;                // forward (wide: out before its rounding, or null)
    int32_t lse_pairs;                     // lse holds pairs (m, l)
    void *dq, *dk, *dv, *dvals;            // backward
    void *pds;                             // row kernels: [B][nnz][heads] pairs (p, ds)
    float4 *stat;                          // tile kernels: [B][heads][n_rows] m, 1 / l, D / l, 0 (m / log 2 without values)
    float *ds_out;                         // tile kernels: [B][heads][nnz] ds, or null
    float *vals_w;                         // tile kernels: room for [B][nnz] 32-bit values
    const float *vals_f, *vals_t;          // and the values as they read them, in A's and A^T's order
    void *part;                            // partial sums of split rows (part_index)
    void *part_ml;                         // forward: their maximum and sum, pairs in the same order
};

// Accumulator type of a storage type: 32 bits for 16- and 32-bit types.
template <typename T> struct AccOf { using type = float; };
template <> struct AccOf<double> { using type = double; };

__device__ __forceinline__ double to_acc(double x) { return x; }
__device__ __forceinline__ float to_acc(float x) { return x; }
__device__ __forceinline__ float to_acc(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_acc(__half x) { return __half2float(x); }
template <typename T, typename A> __device__ __forceinline__ T from_acc(A x) {
    if constexpr (std::is_same_v<T, __nv_bfloat16>) return __float2bfloat16_rn(x);
    else if constexpr (std::is_same_v<T, __half>) return __float2half_rn(x);
    else return (T)x;
}

// N consecutive elements, by 16-byte loads when they fill one or two.
template <typename T, int N> struct alignas(sizeof(T) * N) Pack { T e[N]; };

template <typename T, int N>
__device__ __forceinline__ Pack<T, N> load_pack(const T *p) {
    Pack<T, N> r;
    if constexpr (sizeof(T) * N == 16) {
        *reinterpret_cast<uint4 *>(&r) = __ldg(reinterpret_cast<const uint4 *>(p));
    } else if constexpr (sizeof(T) * N == 32) {
        reinterpret_cast<uint4 *>(&r)[0] = __ldg(reinterpret_cast<const uint4 *>(p));
        reinterpret_cast<uint4 *>(&r)[1] = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) r.e[i] = p[i];
    }
    return r;
}

// Two 32-bit multiply-adds in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(*reinterpret_cast<unsigned long long *>(&a)), "l"(*reinterpret_cast<unsigned long long *>(&b)),
          "l"(*reinterpret_cast<unsigned long long *>(&c)));
    return *reinterpret_cast<float2 *>(&d);
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<unsigned long long *>(&a)), "l"(*reinterpret_cast<unsigned long long *>(&b)));
    return *reinterpret_cast<float2 *>(&d);
}

// The hardware's exponential (2 ulp; results below 2^-126 are zero, which a
// softmax does not notice).
__device__ __forceinline__ float exp2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float exp_acc(float x) { return exp2_of(x * 1.4426950408889634f); }
__device__ __forceinline__ double exp_acc(double x) { return exp(x); }
__device__ __forceinline__ float log_acc(float x) { return logf(x); }
__device__ __forceinline__ double log_acc(double x) { return log(x); }
template <typename A> __device__ __forceinline__ A neg_inf();
template <> __device__ __forceinline__ float neg_inf<float>() { return __int_as_float(0xff800000); }
template <> __device__ __forceinline__ double neg_inf<double>() { return __longlong_as_double(0xfff0000000000000ll); }

// A row's statistics: l == 0 (no weight) is lse = -inf.
template <typename A>
__device__ __forceinline__ void store_lse(const AttnArgs &a, int64_t at, A m, A l) {
    const A top = l == (A)0 ? neg_inf<A>() : m;
    A *p = static_cast<A *>(a.lse);
    if (a.lse_pairs) {
        p[2 * at] = top;
        p[2 * at + 1] = l;
    } else {
        p[at] = l == (A)0 ? top : m + log_acc(l);
    }
}

// A stored value as a score term.  A finite 64-bit value beyond the 32-bit
// range stays finite, so that only -inf removes an entry.
template <typename A>
__device__ __forceinline__ A load_value(const void *vals, int f64, int64_t t) {
    if (!vals) return (A)0;
    if (!f64) return (A)__ldg(static_cast<const float *>(vals) + t);
    const double x = __ldg(static_cast<const double *>(vals) + t);
    if constexpr (sizeof(A) == 8) {
        return x;
    } else {
        if (isinf(x)) return (float)x;
        return x > FLT_MAX ? FLT_MAX : (x < -FLT_MAX ? -FLT_MAX : (float)x);
    }
}

// Place of one segment's partial result: `dim` sums (forward; `dim` or twice as many
// backward).  Rows of a unit and heads are the fastest indices.
__host__ __device__ __forceinline__ int64_t part_index(int64_t slot, int32_t n_slots, int b, int rows, int r,
                                                       int heads, int h) {
    return (((int64_t)b * n_slots + slot) * rows + r) * heads + h;
}

void use_plan(AttnArgs &a, const AttnPlan &p);
void free_attn_plans(Csr *h);

// Joins of split rows (sla_attention.cu), shared by the row and tile kernels.
template <typename T>
sla_status attn_join(const AttnArgs &a, const AttnPlan &p, cudaStream_t s);
template <typename T>
sla_status attn_join_sums(const AttnArgs &a, const AttnPlan &p, int n_rows, int heads, int width, void *out0, void *out1,
                          cudaStream_t s);

// Tile kernels (sla_attention_tile.cu): plan arrays of a tile plan, and the calls.
sla_status build_tiles(AttnTiles *t, const AttnPlan &parts, int rows, int times, int n_rows, const int32_t *rowptr, const int32_t *colind,
                       cudaStream_t s);
template <typename T> sla_status attn_tile_forward(AttnArgs a, cudaStream_t s);
template <typename T> sla_status attn_tile_bwd_rows(AttnArgs a, cudaStream_t s);
template <typename T> sla_status attn_tile_bwd_cols(AttnArgs a, cudaStream_t s);

inline unsigned blocks_of(int64_t n, int t = 256) { return (unsigned)((n + t - 1) / t); }

// Device memory for the work queued on a stream, given back to the stream's pool
// when the scope ends.
struct DeviceScratch {
    cudaStream_t stream;
    std::vector<void *> held;
    explicit DeviceScratch(cudaStream_t s) : stream(s) {}
    ~DeviceScratch() {
        for (void *p : held) cudaFreeAsync(p, stream);
    }
    template <typename U>
    U *get(size_t count) {
        void *p = nullptr;
        if (cudaMallocAsync(&p, (count > 0 ? count : 1) * sizeof(U), stream) != cudaSuccess) {
            cudaGetLastError();
            return nullptr;
        }
        held.push_back(p);
        return static_cast<U *>(p);
    }
};

template <typename U>
bool alloc_array(U **p, size_t count) {
    if (cudaMalloc(p, (count > 0 ? count : 1) * sizeof(U)) == cudaSuccess) return true;
    cudaGetLastError();
    return false;
}

}  // namespace sla
