// Attention over a CSR pattern for 16-bit heads, on the tensor cores.
//
// A warp takes 16 consecutive rows of the pattern (a tile), one head and the
// columns that any of those rows stores, 16 at a time (a chunk).  Neighbouring
// rows of a mesh or graph share columns, so a k or v row is fetched once for the
// tile instead of once an entry, and the scores of all 16 x 16 pairs are a
// matrix product; pairs that are not stored are masked by the chunk's row bits.
// Most of that product is thrown away (a 5-point grid uses 5 of 34 columns a
// row), which costs nothing: the gathers bound the kernel.
//
// No shared memory: operands go from global memory to the registers the matrix
// instructions take.  A dot product does not depend on the order of its terms,
// so thread (g, c) of a quad layout (g = lane / 4, c = lane % 4) reads dim / 4
// consecutive elements of column g (16-byte loads) and feeds them as its four
// places of every k step, the tile's own rows in the same order.  For the
// products that sum over columns, thread (g, c) reads dim / 8 consecutive
// elements of the columns 2c and 2c + 1 and takes element nb of them as output
// block nb, so its outputs are consecutive too.
//
// Scores: 16-bit products, exact, summed in 32 bits.  Weights are not rounded to
// 16 bits: they multiply as tf32 (the 16-bit operand is exact in it), rounded to
// 11 bits for bfloat16 outputs (8 bits) and as a sum of two 11-bit parts for
// float16 outputs (11 bits), which keeps the outputs as good as 32-bit products.
//
// Masked pairs have weight 0, but 0 times an infinity or a NaN is a NaN.  A column
// that every row leaves out (values of -inf: padding, which may hold anything) is
// read as zeros.  If a sum ends as a NaN all the same, the warp redoes its rows
// entry by entry: a bad number of a column that some rows use would otherwise
// reach the tile's other rows.
#include <climits>

#include "sla_attention.cuh"

namespace sla {
namespace {

constexpr int kTileWarps = 4;
constexpr int kTileThreads = 32 * kTileWarps;
constexpr unsigned kAll = 0xffffffffu;

// ----------------------------------------------------------------- plan ----
// One warp a part of a tile: the columns from one entry of the tile's longest
// row to the entry seg_len further on.  Lane r < 16 walks row r's entries
// there, and the smallest column any row is at is the next one.  FILL == false
// counts the columns; FILL writes them, at[part] columns after the first part's.
template <bool FILL>
__global__ void __launch_bounds__(128)
tile_columns_kernel(int n_rows, const int32_t *__restrict__ rowptr, const int32_t *__restrict__ colind, int n_parts,
                    int seg_len, const int32_t *__restrict__ part_unit, const int32_t *__restrict__ part_seg,
                    unsigned *count, const unsigned *__restrict__ at, const int32_t *__restrict__ chunk0,
                    TileChunk *chunks) {
    const int part = (int)((blockIdx.x * (int64_t)128 + threadIdx.x) >> 5), lane = threadIdx.x & 31;
    if (part > n_parts) return;
    if (part == n_parts) {
        if (!FILL && lane == 0) count[part] = 0;
        return;
    }
    const int unit = part_unit ? part_unit[part] : part, seg = part_seg ? part_seg[part] : 0;
    const int64_t row = (int64_t)unit * kTileRows + lane;
    int t0 = 0, t1 = 0;
    if (lane < kTileRows && row < n_rows) {
        t0 = rowptr[row];
        t1 = rowptr[row + 1];
    }
    bool last = true;
    if (part_unit) {
        const int len = t1 - t0, most = __reduce_max_sync(kAll, len);
        const int who = __ffs(__ballot_sync(kAll, len == most)) - 1;
        const int b0 = __shfl_sync(kAll, t0, who);
        const int64_t e0 = (int64_t)seg * seg_len, e1 = e0 + seg_len;
        const int lo = seg == 0 ? 0 : colind[b0 + e0], hi = e1 < most ? colind[b0 + e1] : INT_MAX;
        last = hi == INT_MAX;
        auto first_at = [&](int c) {            // first entry of the row with a column >= c
            int a = t0, b = t1;
            while (a < b) {
                const int mid = a + ((b - a) >> 1);
                if (colind[mid] < c) a = mid + 1;
                else b = mid;
            }
            return a;
        };
        const int a = first_at(lo), b = first_at(hi);
        t0 = a;
        t1 = b;
    }
    int cur = t0 < t1 ? colind[t0] : INT_MAX, next = t0 + 1 < t1 ? colind[t0 + 1] : INT_MAX, t = t0;
    const unsigned n0 = FILL ? at[part] - at[part - seg] : 0;
    unsigned n = n0, row_bits = 0;
    int mine = 0, first = (int)(n0 & 15);       // places [first, n & 15) of the current chunk are this part's
    TileChunk *ck = FILL ? chunks + chunk0[unit] + (n0 >> 4) : nullptr;
    auto flush = [&](int end) {
        if (lane >= first && lane < end) ck->col[lane] = mine;
        // two rows a word; neighbouring parts may share a chunk
        if (lane < kTileRows && row_bits)
            atomicOr(reinterpret_cast<unsigned *>(ck->bits) + (lane >> 1), row_bits << (16 * (lane & 1)));
        row_bits = 0;
        first = 0;
        ++ck;
    };
    for (;;) {
        const int c = __reduce_min_sync(kAll, cur);
        if (c == INT_MAX) break;
        const int place = (int)(n & 15);
        if (FILL && place == 0 && lane < kTileRows) ck->start[lane] = t;
        if (cur == c) {
            row_bits |= 1u << place;
            cur = next;
            ++t;
            next = t + 1 < t1 ? colind[t + 1] : INT_MAX;
        }
        if (lane >= place) mine = c;            // later places hold the last column until they get theirs
        ++n;
        if (FILL && place == 15) flush(16);
    }
    if (FILL && (n & 15) && n > n0) flush(last ? 16 : (int)(n & 15));
    if (!FILL && lane == 0) count[part] = n;
}

// Chunks of each tile, from its parts' columns.
__global__ void tile_chunks_kernel(int n_units, int n_parts, const unsigned *__restrict__ at,
                                   const int32_t *__restrict__ part_unit, const int32_t *__restrict__ part_seg,
                                   unsigned *chunks) {
    const int part = blockIdx.x * blockDim.x + threadIdx.x;
    if (part == 0) chunks[n_units] = 0;
    if (part >= n_parts) return;
    const int unit = part_unit ? part_unit[part] : part, seg = part_seg ? part_seg[part] : 0;
    if (part + 1 < n_parts && part_seg && part_seg[part + 1] > seg) return;    // not the tile's last part
    chunks[unit] = (at[part + 1] - at[part - seg] + 15) / 16;
}

// ------------------------------------------------------------ operands ----
// W consecutive 32-bit words (W * 4 bytes apart for neighbouring threads).
template <int W>
__device__ __forceinline__ void load_words(uint32_t (&r)[W], const void *p) {
    if constexpr (W % 4 == 0) {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const uint4 x = __ldg(static_cast<const uint4 *>(p) + i);
            r[4 * i] = x.x;
            r[4 * i + 1] = x.y;
            r[4 * i + 2] = x.z;
            r[4 * i + 3] = x.w;
        }
    } else if constexpr (W % 2 == 0) {
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
            const uint2 x = __ldg(static_cast<const uint2 *>(p) + i);
            r[2 * i] = x.x;
            r[2 * i + 1] = x.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) r[i] = __ldg(static_cast<const uint32_t *>(p) + i);
    }
}

template <int W>
__device__ __forceinline__ void store_words(void *p, const uint32_t (&r)[W]) {
    if constexpr (W % 4 == 0) {
#pragma unroll
        for (int i = 0; i < W / 4; ++i)
            static_cast<uint4 *>(p)[i] = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
    } else if constexpr (W % 2 == 0) {
#pragma unroll
        for (int i = 0; i < W / 2; ++i) static_cast<uint2 *>(p)[i] = make_uint2(r[2 * i], r[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) static_cast<uint32_t *>(p)[i] = r[i];
    }
}

template <typename T>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same_v<T, __nv_bfloat16>)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The two 16-bit elements of a word as 32-bit numbers.
template <typename T>
__device__ __forceinline__ void widen(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if constexpr (std::is_same_v<T, __nv_bfloat16>) {
        lo = w << 16;
        hi = w & 0xffff0000u;
    } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        lo = __float_as_uint(f.x);
        hi = __float_as_uint(f.y);
    }
}

template <typename T>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
    uint32_t r;
    if constexpr (std::is_same_v<T, __nv_bfloat16>) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        r = *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __half2 v = __floats2half2_rn(lo, hi);
        r = *reinterpret_cast<const uint32_t *>(&v);
    }
    return r;
}

__device__ __forceinline__ float exp_of(float x) { return exp2f(x * 1.4426950408889634f); }

// The main loops hold scores in units of log 2, so that a weight is one
// exponential of a difference (the hardware's: 2 ulp, results below 2^-126 are
// zero, which a softmax does not notice).
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
__device__ __forceinline__ float exp2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// A stored value in those units; a finite one stays finite.
__device__ __forceinline__ float value_log2(float x) {
    constexpr float kMost = 2.3e38f;
    if (x > kMost && x <= FLT_MAX) x = kMost;
    if (x < -kMost && x >= -FLT_MAX) x = -kMost;
    return x * kLog2e;
}


// The tile's own 16 rows as the left operand of score products.
template <int D>
struct Own {
    uint32_t a[D / 16][4];
    template <typename T>
    __device__ __forceinline__ void load(const T *base, int64_t stride, int64_t row0, int n_rows, int g, int c) {
        uint32_t r[2][D / 8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (row0 + g + 8 * i < n_rows) load_words<D / 8>(r[i], base + (row0 + g + 8 * i) * stride + c * (D / 4));
            else {
#pragma unroll
                for (int w = 0; w < D / 8; ++w) r[i][w] = 0;
            }
        }
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
            a[s][0] = r[0][2 * s];
            a[s][1] = r[1][2 * s];
            a[s][2] = r[0][2 * s + 1];
            a[s][3] = r[1][2 * s + 1];
        }
    }
};

// s[2][4]: the products of the 16 own rows with the 16 columns of a chunk, the
// columns 8 blk + (2c, 2c + 1) of rows g and g + 8 in this thread.
template <typename T, int D>
__device__ __forceinline__ void score_products(float (&s)[2][4], const Own<D> &own, const uint32_t (&k)[2][D / 8]) {
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
        s[blk][0] = s[blk][1] = s[blk][2] = s[blk][3] = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) mma16<T>(s[blk], own.a[i], k[blk][2 * i], k[blk][2 * i + 1]);
    }
}

// Sums over a chunk's columns: o[nb] += w . x, with x the rows of the columns
// 8 blk + (2c, 2c + 1), elements g * (D / 8) + nb.
template <typename T, int D>
struct Sums {
    float o[D / 8][4];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int nb = 0; nb < D / 8; ++nb) o[nb][0] = o[nb][1] = o[nb][2] = o[nb][3] = 0.0f;
    }
    __device__ __forceinline__ void scale(float lo, float hi) {
#pragma unroll
        for (int nb = 0; nb < D / 8; ++nb) {
            o[nb][0] *= lo;
            o[nb][1] *= lo;
            o[nb][2] *= hi;
            o[nb][3] *= hi;
        }
    }
    __device__ __forceinline__ void add(const float (&w)[4], const uint32_t (&x0)[D / 16], const uint32_t (&x1)[D / 16]) {
        const float v[4] = {w[0], w[2], w[1], w[3]};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (std::is_same_v<T, __nv_bfloat16>) {
                asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi[i]) : "f"(v[i]));
            } else {
                hi[i] = __float_as_uint(v[i]) & 0xffffe000u;
                lo[i] = __float_as_uint(v[i] - __uint_as_float(hi[i]));
            }
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            uint32_t a0, a1, b0, b1;
            widen<T>(x0[i], a0, a1);
            widen<T>(x1[i], b0, b1);
            mma_tf32(o[2 * i], hi, a0, b0);
            mma_tf32(o[2 * i + 1], hi, a1, b1);
            if constexpr (!std::is_same_v<T, __nv_bfloat16>) {
                mma_tf32(o[2 * i], lo, a0, b0);
                mma_tf32(o[2 * i + 1], lo, a1, b1);
            }
        }
    }
    __device__ __forceinline__ bool bad() const {
        bool b = false;
#pragma unroll
        for (int nb = 0; nb < D / 8; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) b = b || o[nb][i] != o[nb][i];
        return __any_sync(kAll, b);
    }
    // Row g (i = 0) or g + 8 (i = 1): elements 2c (D / 8) and the next D / 4.
    __device__ __forceinline__ void store(T *p, int i, int c) const {
        uint32_t w[D / 8];
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            w[j] = narrow2<T>(o[2 * j][2 * i], o[2 * j + 1][2 * i]);
            w[D / 16 + j] = narrow2<T>(o[2 * j][2 * i + 1], o[2 * j + 1][2 * i + 1]);
        }
        store_words<D / 8>(p + c * (D / 4), w);
    }
    __device__ __forceinline__ void store(float *p, int i, int c) const {
        uint32_t w[D / 4];
#pragma unroll
        for (int nb = 0; nb < D / 8; ++nb) {
            w[nb] = __float_as_uint(o[nb][2 * i]);
            w[D / 8 + nb] = __float_as_uint(o[nb][2 * i + 1]);
        }
        store_words<D / 4>(p + c * (D / 4), w);
    }
};

// A warp's work: chunks [ch0, ch1) of a tile, one head of one system.
struct TileWork {
    int64_t row0;
    int b, h, kh, slot;
    const TileChunk *ch0, *ch1;
};

__device__ __forceinline__ bool tile_item(TileWork &w, const AttnArgs &a, unsigned x, unsigned y, unsigned share) {
    const unsigned it = x / share;
    if (it >= (unsigned)a.n_items) return false;
    w.b = (int)(y / (unsigned)a.kv_heads);
    w.kh = (int)(y - (unsigned)w.b * a.kv_heads);
    w.h = w.kh * (a.heads / a.kv_heads) + (int)(x - it * share);
    int unit = (int)it, seg = 0;
    w.slot = -1;
    if (a.item_unit) {
        unit = __ldg(a.item_unit + it);
        seg = __ldg(a.item_seg + it);
        w.slot = __ldg(a.item_slot + it);
    }
    w.row0 = (int64_t)unit * kTileRows;
    const int c0 = __ldg(a.chunk0 + unit), c1 = __ldg(a.chunk0 + unit + 1);
    const int64_t from = (int64_t)c0 + (int64_t)seg * a.seg_len, to = from + a.seg_len;
    w.ch0 = a.chunks + from;
    w.ch1 = a.chunks + (to < c1 ? to : (int64_t)c1);
    return true;
}

// What a thread needs of a chunk: the columns it reads for the scores (g and
// 8 + g) and for the sums (8 blk + 2c, + 1), rows g's and g + 8's bits, and
// with ENTRIES the first entry of those rows.
template <bool ENTRIES>
struct Chunk {
    unsigned kc[2], vc[4], bits[2];
    int at[2];
    __device__ __forceinline__ void load(const TileChunk *p, int g, int c, int n_cols) {
        kc[0] = (unsigned)__ldg(p->col + g);
        kc[1] = (unsigned)__ldg(p->col + 8 + g);
        const int2 x = __ldg(reinterpret_cast<const int2 *>(p->col) + c);
        const int2 y = __ldg(reinterpret_cast<const int2 *>(p->col) + 4 + c);
        vc[0] = (unsigned)x.x;
        vc[1] = (unsigned)x.y;
        vc[2] = (unsigned)y.x;
        vc[3] = (unsigned)y.y;
        bits[0] = __ldg(p->bits + g);
        bits[1] = __ldg(p->bits + 8 + g);
        if constexpr (ENTRIES) {
            at[0] = __ldg(p->start + g);
            at[1] = __ldg(p->start + 8 + g);
        }
#if SLA_DEBUG_BOUNDS
        for (int i = 0; i < 2; ++i) kc[i] = (unsigned)SLA_IDX((int)kc[i], n_cols, kBndColumn);
        for (int i = 0; i < 4; ++i) vc[i] = (unsigned)SLA_IDX((int)vc[i], n_cols, kBndColumn);
#else
        (void)n_cols;
#endif
    }
    // Entry of row g + 8 i at position pos (if the row stores it).
    __device__ __forceinline__ int entry(int i, int pos) const {
        return at[i] + __popc(bits[i] & ((1u << pos) - 1u));
    }
};

// Row `col` of a tensor with rows `bytes` apart (below 2^32: one multiply-add).
template <typename T>
__device__ __forceinline__ const void *row_at(const T *base, unsigned col, unsigned bytes) {
    return reinterpret_cast<const char *>(base) + (uint64_t)col * bytes;
}

// Zeros for the gathered rows of the columns that no row of the tile uses; used:
// bit j for this thread's column vc[j], from its own rows.
template <int W>
__device__ __forceinline__ void drop_unused(uint32_t (&x)[4][W], unsigned used) {
    used |= __shfl_xor_sync(kAll, used, 4);
    used |= __shfl_xor_sync(kAll, used, 8);
    used |= __shfl_xor_sync(kAll, used, 16);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (!(used >> j & 1))
#pragma unroll
            for (int i = 0; i < W; ++i) x[j][i] = 0;
}

// Entry range of row r of the tile in the item (every lane r < 16 its own row).
__device__ __forceinline__ void row_range(const TileWork &w, int lane, int &t0, int &t1) {
    t0 = t1 = 0;
    if (lane < kTileRows && w.ch0 < w.ch1) {
        t0 = t1 = __ldg(w.ch0->start + lane);
        for (const TileChunk *ch = w.ch0; ch < w.ch1; ++ch) t1 += __popc((unsigned)__ldg(ch->bits + lane));
    }
}

__device__ __forceinline__ float warp_sumf(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

constexpr int kSlowVec = 4;     // elements of a head a lane holds, 128 / 32

template <typename T>
__device__ __forceinline__ void slow_load(float (&x)[kSlowVec], const T *p, int dim, int lane) {
#pragma unroll
    for (int i = 0; i < kSlowVec; ++i) x[i] = i * 32 + lane < dim ? to_acc(p[i * 32 + lane]) : 0.0f;
}

__device__ __forceinline__ float slow_dot(const float (&x)[kSlowVec], const float (&y)[kSlowVec]) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kSlowVec; ++i) s = fmaf(x[i], y[i], s);
    return warp_sumf(s);
}

// --------------------------------------------------------------- forward ----
// The same rows entry by entry, for tiles that a number that is not finite reached.
template <typename T>
__device__ __noinline__ void slow_forward(const AttnArgs &a, const TileWork &w) {
    const int lane = threadIdx.x & 31;
    int s0, s1;
    row_range(w, lane, s0, s1);
    const T *qb = static_cast<const T *>(a.q) + w.b * a.qs[0] + w.h * a.qs[2];
    const T *kb = static_cast<const T *>(a.k) + w.b * a.ks[0] + w.kh * a.ks[2];
    const T *vb = static_cast<const T *>(a.v) + w.b * a.vs[0] + w.kh * a.vs[2];
    const float scale = (float)a.scale, none = neg_inf<float>();
    for (int r = 0; r < kTileRows && w.row0 + r < a.n_rows; ++r) {
        const int t0 = __shfl_sync(kAll, s0, r), t1 = __shfl_sync(kAll, s1, r);
        float q[kSlowVec], acc[kSlowVec] = {}, m = none, l = 0.0f;
        slow_load(q, qb + (w.row0 + r) * a.qs[1], a.dim, lane);
        for (int t = t0; t < t1; ++t) {
            const int64_t col = SLA_IDX((int64_t)__ldg(a.colind + t), a.n_cols, kBndColumn);
            const float x = load_value<float>(a.vals, a.vals_f64, w.b * a.nnz + t);
            if (x == none) continue;
            float k[kSlowVec], v[kSlowVec];
            slow_load(k, kb + col * a.ks[1], a.dim, lane);
            slow_load(v, vb + col * a.vs[1], a.dim, lane);
            const float s = fmaf(slow_dot(q, k), scale, x), top = fmaxf(m, s);
            const float ref = top == none ? 0.0f : top, fix = exp_of(m - ref), p = exp_of(s - ref);
            m = top;
            l = l * fix + p;
#pragma unroll
            for (int i = 0; i < kSlowVec; ++i) acc[i] = fmaf(p, v[i], acc[i] * fix);
        }
        if (w.slot < 0) {
            const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
            const int64_t at = ((int64_t)w.b * a.n_rows + w.row0 + r) * a.heads + w.h;
#pragma unroll
            for (int i = 0; i < kSlowVec; ++i)
                if (i * 32 + lane < a.dim) {
                    static_cast<T *>(a.out)[at * a.dim + i * 32 + lane] = from_acc<T>(acc[i] * inv);
                    if (a.wide) static_cast<float *>(a.wide)[at * a.dim + i * 32 + lane] = acc[i] * inv;
                }
            if (lane == 0) static_cast<float *>(a.lse)[at] = l == 0.0f ? none : m + logf(l);
        } else {
            float *p = static_cast<float *>(a.part) +
                       part_index(w.slot, a.n_slots, w.b, kTileRows, r, a.heads, w.h) * (a.dim + 2);
#pragma unroll
            for (int i = 0; i < kSlowVec; ++i)
                if (i * 32 + lane < a.dim) p[i * 32 + lane] = acc[i];
            if (lane == 0) {
                p[a.dim] = m;
                p[a.dim + 1] = l;
            }
        }
    }
}

template <typename T, int D, bool VALS>
__global__ void __launch_bounds__(kTileThreads) tile_forward_kernel(const __grid_constant__ AttnArgs a) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const unsigned share = (unsigned)(a.heads / a.kv_heads), n_y = (unsigned)a.batch * a.kv_heads;
    const unsigned kst = (unsigned)a.ks[1] * 2, vst = (unsigned)a.vs[1] * 2;
    const float scale = (float)(a.scale * 1.4426950408889634), none = neg_inf<float>();
    for (unsigned y = blockIdx.y; y < n_y; y += gridDim.y) {
        TileWork w;
        if (!tile_item(w, a, blockIdx.x * kTileWarps + (threadIdx.x >> 5), y, share)) return;
        Own<D> q;
        q.load(static_cast<const T *>(a.q) + w.b * a.qs[0] + w.h * a.qs[2], a.qs[1], w.row0, a.n_rows, g, c);
        const T *kb = static_cast<const T *>(a.k) + w.b * a.ks[0] + w.kh * a.ks[2] + c * (D / 4);
        const T *vb = static_cast<const T *>(a.v) + w.b * a.vs[0] + w.kh * a.vs[2] + g * (D / 8);
        Sums<T, D> acc;
        acc.zero();
        float m[2] = {none, none}, l[2] = {0.0f, 0.0f};
        Chunk<VALS> next;
        if (w.ch0 < w.ch1) next.load(w.ch0, g, c, a.n_cols);
        for (const TileChunk *ch = w.ch0; ch < w.ch1; ++ch) {
            const Chunk<VALS> cur = next;
            uint32_t k[2][D / 8], v[4][D / 16];
#pragma unroll
            for (int i = 0; i < 2; ++i) load_words<D / 8>(k[i], row_at(kb, cur.kc[i], kst));
#pragma unroll
            for (int i = 0; i < 4; ++i) load_words<D / 16>(v[i], row_at(vb, cur.vc[i], vst));
            if (ch + 1 < w.ch1) next.load(ch + 1, g, c, a.n_cols);
            float s[2][4];
            score_products<T, D>(s, q, k);
            float top[2] = {m[0], m[1]};
            unsigned used = 0;
            const unsigned mine[2] = {cur.bits[0] >> (2 * c), cur.bits[1] >> (2 * c)};
#pragma unroll
            for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                for (int e = 0; e < 4; ++e) {           // row g + 8 (e / 2), column 8 blk + 2c + e % 2
                    const int i = e >> 1;
                    bool on = mine[i] & (1u << (8 * blk + (e & 1)));
                    if constexpr (VALS) {
                        float x = 0.0f;
                        if (on)
                            x = load_value<float>(a.vals, a.vals_f64,
                                                  w.b * a.nnz + cur.entry(i, 8 * blk + 2 * c + (e & 1)));
                        on = on && x != none;
                        used |= (unsigned)on << (2 * blk + (e & 1));
                        s[blk][e] = fmaf(s[blk][e], scale, value_log2(x));
                    } else {
                        s[blk][e] *= scale;
                    }
                    s[blk][e] = on ? s[blk][e] : none;
                    top[i] = fmaxf(top[i], s[blk][e]);
                }
            if constexpr (VALS) drop_unused(v, used);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                top[i] = fmaxf(top[i], __shfl_xor_sync(kAll, top[i], 1));
                top[i] = fmaxf(top[i], __shfl_xor_sync(kAll, top[i], 2));
            }
            const float ref[2] = {top[0] == none ? 0.0f : top[0], top[1] == none ? 0.0f : top[1]};
            if (__any_sync(kAll, top[0] != m[0] || top[1] != m[1])) {
                const float f0 = exp2_of(m[0] - ref[0]), f1 = exp2_of(m[1] - ref[1]);
                acc.scale(f0, f1);
                l[0] *= f0;
                l[1] *= f1;
                m[0] = top[0];
                m[1] = top[1];
            }
#pragma unroll
            for (int blk = 0; blk < 2; ++blk) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[blk][e] = exp2_of(s[blk][e] - ref[e >> 1]);
                    l[e >> 1] += s[blk][e];
                }
                acc.add(s[blk], v[2 * blk], v[2 * blk + 1]);
            }
        }
        if (acc.bad()) {
            slow_forward<T>(a, w);
            continue;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(kAll, l[i], 1);
            l[i] += __shfl_xor_sync(kAll, l[i], 2);
            m[i] *= kLn2;
        }
        if (w.slot < 0) acc.scale(l[0] > 0.0f ? 1.0f / l[0] : 0.0f, l[1] > 0.0f ? 1.0f / l[1] : 0.0f);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = g + 8 * i;
            if (w.row0 + r >= a.n_rows) continue;
            if (w.slot < 0) {
                const int64_t o = ((int64_t)w.b * a.n_rows + w.row0 + r) * a.heads + w.h;
                acc.store(static_cast<T *>(a.out) + o * D, i, c);
                if (a.wide) acc.store(static_cast<float *>(a.wide) + o * D, i, c);
                if (c == 0) static_cast<float *>(a.lse)[o] = l[i] == 0.0f ? none : m[i] + logf(l[i]);
            } else {
                float *p = static_cast<float *>(a.part) +
                           part_index(w.slot, a.n_slots, w.b, kTileRows, r, a.heads, w.h) * (D + 2);
#pragma unroll
                for (int nb = 0; nb < D / 8; ++nb) {    // D + 2 numbers a partial: not on 16 bytes
                    p[c * (D / 4) + nb] = acc.o[nb][2 * i];
                    p[c * (D / 4) + D / 8 + nb] = acc.o[nb][2 * i + 1];
                }
                if (c == 0) {
                    p[D] = m[i];
                    p[D + 1] = l[i];
                }
            }
        }
    }
}

// -------------------------------------------------------------- backward ----
// dq of the tile's rows, entry by entry.
template <typename T>
__device__ __noinline__ void slow_bwd_rows(const AttnArgs &a, const TileWork &w) {
    const int lane = threadIdx.x & 31;
    int s0, s1;
    row_range(w, lane, s0, s1);
    const T *kb = static_cast<const T *>(a.k) + w.b * a.ks[0] + w.kh * a.ks[2];
    const T *vb = static_cast<const T *>(a.v) + w.b * a.vs[0] + w.kh * a.vs[2];
    const float scale = (float)a.scale, none = neg_inf<float>();
    for (int r = 0; r < kTileRows && w.row0 + r < a.n_rows; ++r) {
        const int t0 = __shfl_sync(kAll, s0, r), t1 = __shfl_sync(kAll, s1, r);
        const int64_t row = w.row0 + r, at = ((int64_t)w.b * a.n_rows + row) * a.heads + w.h;
        float q[kSlowVec], go[kSlowVec], o[kSlowVec], acc[kSlowVec] = {};
        slow_load(q, static_cast<const T *>(a.q) + w.b * a.qs[0] + row * a.qs[1] + w.h * a.qs[2], a.dim, lane);
        slow_load(go, static_cast<const T *>(a.dout) + w.b * a.ds[0] + row * a.ds[1] + w.h * a.ds[2], a.dim, lane);
        slow_load(o, static_cast<const float *>(a.o) + at * a.dim, a.dim, lane);
        const float delta = slow_dot(go, o), lse = static_cast<const float *>(a.lse)[at];
        for (int t = t0; t < t1 && lse != none; ++t) {
            const int64_t col = SLA_IDX((int64_t)__ldg(a.colind + t), a.n_cols, kBndColumn);
            const float x = load_value<float>(a.vals, a.vals_f64, w.b * a.nnz + t);
            if (x == none) continue;
            float k[kSlowVec], v[kSlowVec];
            slow_load(k, kb + col * a.ks[1], a.dim, lane);
            slow_load(v, vb + col * a.vs[1], a.dim, lane);
            const float p = exp_of(fmaf(slow_dot(q, k), scale, x) - lse);
            const float ds = p * (slow_dot(go, v) - delta);
#pragma unroll
            for (int i = 0; i < kSlowVec; ++i) acc[i] = fmaf(ds, k[i], acc[i]);
        }
#pragma unroll
        for (int i = 0; i < kSlowVec; ++i)
            if (i * 32 + lane < a.dim) {
                const int d = i * 32 + lane;
                if (w.slot < 0) static_cast<T *>(a.dq)[at * a.dim + d] = from_acc<T>(acc[i] * scale);
                else
                    static_cast<float *>(a.part)[part_index(w.slot, a.n_slots, w.b, kTileRows, r, a.heads, w.h) * a.dim + d] =
                        acc[i] * scale;
            }
    }
}

// By A's rows: (lse, D) of every row, dq, and ds of every entry if asked for.
template <typename T, int D, bool VALS>
__global__ void __launch_bounds__(kTileThreads) tile_bwd_rows_kernel(const __grid_constant__ AttnArgs a) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const unsigned share = (unsigned)(a.heads / a.kv_heads), n_y = (unsigned)a.batch * a.kv_heads;
    const unsigned kst = (unsigned)a.ks[1] * 2, vst = (unsigned)a.vs[1] * 2;
    const float scale = (float)(a.scale * 1.4426950408889634), none = neg_inf<float>();
    for (unsigned y = blockIdx.y; y < n_y; y += gridDim.y) {
        TileWork w;
        if (!tile_item(w, a, blockIdx.x * kTileWarps + (threadIdx.x >> 5), y, share)) return;
        Own<D> q, go;
        q.load(static_cast<const T *>(a.q) + w.b * a.qs[0] + w.h * a.qs[2], a.qs[1], w.row0, a.n_rows, g, c);
        go.load(static_cast<const T *>(a.dout) + w.b * a.ds[0] + w.h * a.ds[2], a.ds[1], w.row0, a.n_rows, g, c);
        float lse[2] = {none, none}, delta[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t row = w.row0 + g + 8 * i;
            if (row < a.n_rows) {
                const int64_t at = ((int64_t)w.b * a.n_rows + row) * a.heads + w.h;
                lse[i] = __ldg(static_cast<const float *>(a.lse) + at);
                uint32_t o[D / 4];
                load_words<D / 4>(o, static_cast<const float *>(a.o) + at * D + c * (D / 4));
#pragma unroll
                for (int s = 0; s < D / 16; ++s)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t lo, hi;
                        widen<T>(go.a[s][2 * e + i], lo, hi);
                        delta[i] = fmaf(__uint_as_float(lo), __uint_as_float(o[4 * s + 2 * e]), delta[i]);
                        delta[i] = fmaf(__uint_as_float(hi), __uint_as_float(o[4 * s + 2 * e + 1]), delta[i]);
                    }
            }
            delta[i] += __shfl_xor_sync(kAll, delta[i], 1);
            delta[i] += __shfl_xor_sync(kAll, delta[i], 2);
            if (row < a.n_rows && c == 0)
                a.stat[((int64_t)w.b * a.heads + w.h) * a.n_rows + row] = make_float2(lse[i] * kLog2e, delta[i]);
        }
        const bool dead[2] = {lse[0] == none, lse[1] == none};
        lse[0] *= kLog2e;
        lse[1] *= kLog2e;
        const T *kb = static_cast<const T *>(a.k) + w.b * a.ks[0] + w.kh * a.ks[2];
        const T *vb = static_cast<const T *>(a.v) + w.b * a.vs[0] + w.kh * a.vs[2] + c * (D / 4);
        float *ds_out = VALS && a.ds_out ? a.ds_out + ((int64_t)w.b * a.heads + w.h) * a.nnz : nullptr;
        Sums<T, D> acc;
        acc.zero();
        Chunk<VALS> next;
        if (w.ch0 < w.ch1) next.load(w.ch0, g, c, a.n_cols);
        for (const TileChunk *ch = w.ch0; ch < w.ch1; ++ch) {
            const Chunk<VALS> cur = next;
            float s[2][4], dp[2][4];
            uint32_t x[4][D / 16];
            {
                uint32_t k[2][D / 8], v[2][D / 8];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    load_words<D / 8>(k[i], row_at(kb + c * (D / 4), cur.kc[i], kst));
                    load_words<D / 8>(v[i], row_at(vb, cur.kc[i], vst));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) load_words<D / 16>(x[i], row_at(kb + g * (D / 8), cur.vc[i], kst));
                if (ch + 1 < w.ch1) next.load(ch + 1, g, c, a.n_cols);
                score_products<T, D>(s, q, k);
                score_products<T, D>(dp, go, v);
            }
            unsigned used = 0;
            const unsigned mine[2] = {cur.bits[0] >> (2 * c), cur.bits[1] >> (2 * c)};
#pragma unroll
            for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = e >> 1;
                    const bool there = mine[i] & (1u << (8 * blk + (e & 1)));
                    bool on = there && !dead[i];
                    if constexpr (VALS) {
                        float val = 0.0f;
                        const int t = cur.entry(i, 8 * blk + 2 * c + (e & 1));
                        if (there) val = load_value<float>(a.vals, a.vals_f64, w.b * a.nnz + t);
                        on = on && val != none;
                        used |= (unsigned)on << (2 * blk + (e & 1));
                        s[blk][e] = fmaf(s[blk][e], scale, value_log2(val)) - lse[i];
                        s[blk][e] = on ? exp2_of(s[blk][e]) * (dp[blk][e] - delta[i]) : 0.0f;
                        if (ds_out && there) ds_out[t] = s[blk][e];
                    } else {
                        s[blk][e] = on ? exp2_of(fmaf(s[blk][e], scale, -lse[i])) * (dp[blk][e] - delta[i]) : 0.0f;
                    }
                }
            if constexpr (VALS) drop_unused(x, used);
#pragma unroll
            for (int blk = 0; blk < 2; ++blk) acc.add(s[blk], x[2 * blk], x[2 * blk + 1]);
        }
        if (!a.dq) continue;
        if (acc.bad()) {
            slow_bwd_rows<T>(a, w);
            continue;
        }
        acc.scale((float)a.scale, (float)a.scale);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = g + 8 * i;
            if (w.row0 + r >= a.n_rows) continue;
            if (w.slot < 0)
                acc.store(static_cast<T *>(a.dq) + (((int64_t)w.b * a.n_rows + w.row0 + r) * a.heads + w.h) * D, i, c);
            else
                acc.store(static_cast<float *>(a.part) +
                              part_index(w.slot, a.n_slots, w.b, kTileRows, r, a.heads, w.h) * D, i, c);
        }
    }
}

// dk and dv of the tile's rows of A^T, entry by entry.
template <typename T>
__device__ __noinline__ void slow_bwd_cols(const AttnArgs &a, const TileWork &w, bool want_dk, bool want_dv) {
    const int lane = threadIdx.x & 31, share = a.heads / a.kv_heads;
    int s0, s1;
    row_range(w, lane, s0, s1);
    const float scale = (float)a.scale, none = neg_inf<float>();
    for (int r = 0; r < kTileRows && w.row0 + r < a.n_cols; ++r) {
        const int t0 = __shfl_sync(kAll, s0, r), t1 = __shfl_sync(kAll, s1, r);
        const int64_t row = w.row0 + r;
        float k[kSlowVec], v[kSlowVec], dk[kSlowVec] = {}, dv[kSlowVec] = {};
        slow_load(k, static_cast<const T *>(a.k) + w.b * a.ks[0] + row * a.ks[1] + w.kh * a.ks[2], a.dim, lane);
        slow_load(v, static_cast<const T *>(a.v) + w.b * a.vs[0] + row * a.vs[1] + w.kh * a.vs[2], a.dim, lane);
        for (int h = w.kh * share; h < (w.kh + 1) * share; ++h)
            for (int t = t0; t < t1; ++t) {
                const int64_t i = SLA_IDX((int64_t)__ldg(a.colind + t), a.n_rows, kBndColumn);
                const int64_t e = SLA_IDX((int64_t)__ldg(a.perm + t), a.nnz, kBndEntry);
                const float x = load_value<float>(a.vals, a.vals_f64, w.b * a.nnz + e);
                const float2 st = a.stat[((int64_t)w.b * a.heads + h) * a.n_rows + i];
                if (x == none || st.x == none) continue;
                float q[kSlowVec], go[kSlowVec];
                slow_load(q, static_cast<const T *>(a.q) + w.b * a.qs[0] + i * a.qs[1] + h * a.qs[2], a.dim, lane);
                slow_load(go, static_cast<const T *>(a.dout) + w.b * a.ds[0] + i * a.ds[1] + h * a.ds[2], a.dim, lane);
                const float p = exp2f(fmaf(fmaf(slow_dot(q, k), scale, x), kLog2e, -st.x));
                const float ds = p * (slow_dot(go, v) - st.y);
#pragma unroll
                for (int j = 0; j < kSlowVec; ++j) {
                    dk[j] = fmaf(ds, q[j], dk[j]);
                    dv[j] = fmaf(p, go[j], dv[j]);
                }
            }
        const int64_t at = (((int64_t)w.b * a.n_cols + row) * a.kv_heads + w.kh) * a.dim;
        float *part = static_cast<float *>(a.part) +
                      part_index(w.slot, a.n_slots, w.b, kTileRows, r, a.kv_heads, w.kh) * 2 * a.dim;
#pragma unroll
        for (int j = 0; j < kSlowVec; ++j) {
            const int d = j * 32 + lane;
            if (d >= a.dim) continue;
            if (w.slot < 0) {
                if (want_dk && a.dk) static_cast<T *>(a.dk)[at + d] = from_acc<T>(dk[j] * scale);
                if (want_dv && a.dv) static_cast<T *>(a.dv)[at + d] = from_acc<T>(dv[j]);
            } else {
                if (want_dk) part[d] = dk[j] * scale;
                if (want_dv) part[a.dim + d] = dv[j];
            }
        }
    }
}

// By A^T's rows: dk (DK) and dv (DV) of 16 columns of A, the shared heads one
// after the other.  Wide heads take two launches: both sums and both own
// operands would not fit the registers.
template <typename T, int D, bool DK, bool DV, bool VALS>
__global__ void __launch_bounds__(kTileThreads) tile_bwd_cols_kernel(const __grid_constant__ AttnArgs a) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, share = a.heads / a.kv_heads;
    const unsigned n_y = (unsigned)a.batch * a.kv_heads;
    const unsigned qst = (unsigned)a.qs[1] * 2, dst = (unsigned)a.ds[1] * 2;
    const float scale = (float)(a.scale * 1.4426950408889634), none = neg_inf<float>();
    for (unsigned y = blockIdx.y; y < n_y; y += gridDim.y) {
        TileWork w;
        if (!tile_item(w, a, blockIdx.x * kTileWarps + (threadIdx.x >> 5), y, 1)) return;
        Own<D> k, v;
        k.load(static_cast<const T *>(a.k) + w.b * a.ks[0] + w.kh * a.ks[2], a.ks[1], w.row0, a.n_cols, g, c);
        if constexpr (DK)
            v.load(static_cast<const T *>(a.v) + w.b * a.vs[0] + w.kh * a.vs[2], a.vs[1], w.row0, a.n_cols, g, c);
        Sums<T, D> dk, dv;
        if constexpr (DK) dk.zero();
        if constexpr (DV) dv.zero();
        for (int h = w.kh * share; h < (w.kh + 1) * share; ++h) {
            const T *qb = static_cast<const T *>(a.q) + w.b * a.qs[0] + h * a.qs[2];
            const T *gb = static_cast<const T *>(a.dout) + w.b * a.ds[0] + h * a.ds[2];
            const float2 *stat = a.stat + ((int64_t)w.b * a.heads + h) * a.n_rows;
            Chunk<VALS> next;
            if (w.ch0 < w.ch1) next.load(w.ch0, g, c, a.n_rows);
            for (const TileChunk *ch = w.ch0; ch < w.ch1; ++ch) {
                const Chunk<VALS> cur = next;
                float s[2][4], dp[2][4];
                float2 st[4];
                {
                    uint32_t x[2][D / 8], z[2][D / 8];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        load_words<D / 8>(x[i], row_at(qb + c * (D / 4), cur.kc[i], qst));
                        if constexpr (DK) load_words<D / 8>(z[i], row_at(gb + c * (D / 4), cur.kc[i], dst));
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) st[i] = stat[cur.vc[i]];
                    if (ch + 1 < w.ch1) next.load(ch + 1, g, c, a.n_rows);
                    score_products<T, D>(s, k, x);
                    if constexpr (DK) score_products<T, D>(dp, v, z);
                }
                unsigned used = 0;
                const unsigned mine[2] = {cur.bits[0] >> (2 * c), cur.bits[1] >> (2 * c)};
#pragma unroll
                for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = e >> 1, j = 2 * blk + (e & 1);
                        bool on = mine[i] & (1u << (8 * blk + (e & 1)));
                        float val = 0.0f;
                        if constexpr (VALS) {
                            if (on) {
                                const int64_t at = SLA_IDX((int64_t)__ldg(a.perm + cur.entry(i, 8 * blk + 2 * c + (e & 1))),
                                                           a.nnz, kBndEntry);
                                val = load_value<float>(a.vals, a.vals_f64, w.b * a.nnz + at);
                            }
                        }
                        on = on && val != none && st[j].x != none;
                        if constexpr (VALS) used |= (unsigned)on << j;
                        s[blk][e] = on ? exp2_of(fmaf(s[blk][e], scale, value_log2(val)) - st[j].x) : 0.0f;
                        if constexpr (DK) dp[blk][e] = on ? s[blk][e] * (dp[blk][e] - st[j].y) : 0.0f;
                    }
                uint32_t x[4][D / 16];
                if constexpr (DV) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) load_words<D / 16>(x[j], row_at(gb + g * (D / 8), cur.vc[j], dst));
                    if constexpr (VALS) drop_unused(x, used);
                    dv.add(s[0], x[0], x[1]);
                    dv.add(s[1], x[2], x[3]);
                }
                if constexpr (DK) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) load_words<D / 16>(x[j], row_at(qb + g * (D / 8), cur.vc[j], qst));
                    if constexpr (VALS) drop_unused(x, used);
                    dk.add(dp[0], x[0], x[1]);
                    dk.add(dp[1], x[2], x[3]);
                }
            }
        }
        bool bad = false;
        if constexpr (DK) bad = dk.bad();
        if constexpr (DV) bad = dv.bad() || bad;
        if (bad) {
            slow_bwd_cols<T>(a, w, DK, DV);
            continue;
        }
        if constexpr (DK) dk.scale((float)a.scale, (float)a.scale);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = g + 8 * i;
            if (w.row0 + r >= a.n_cols) continue;
            if (w.slot < 0) {
                const int64_t o = (((int64_t)w.b * a.n_cols + w.row0 + r) * a.kv_heads + w.kh) * D;
                if constexpr (DK)
                    if (a.dk) dk.store(static_cast<T *>(a.dk) + o, i, c);
                if constexpr (DV)
                    if (a.dv) dv.store(static_cast<T *>(a.dv) + o, i, c);
            } else {
                float *p = static_cast<float *>(a.part) +
                           part_index(w.slot, a.n_slots, w.b, kTileRows, r, a.kv_heads, w.kh) * 2 * D;
                if constexpr (DK) dk.store(p, i, c);
                if constexpr (DV) dv.store(p + D, i, c);
            }
        }
    }
}

// -------------------------------------------------------------- launches ----
enum { kTileFwd, kTileBwdRows, kTileBwdCols };

template <typename T, int D, bool VALS>
sla_status launch_tile(int what, const AttnArgs &a, cudaStream_t s) {
    const int64_t warps = (int64_t)a.n_items * (what == kTileBwdCols ? 1 : a.heads / a.kv_heads);
    const int64_t x = (warps + kTileWarps - 1) / kTileWarps, y = (int64_t)a.batch * a.kv_heads;
    SLA_REQUIRE(x < INT_MAX / kTileWarps && y < INT_MAX, "sla_attention: too many rows, systems and heads");
    if (x == 0) return SLA_OK;
    const dim3 grid((unsigned)x, (unsigned)(y < 65535 ? y : 65535));
    if (what == kTileFwd) {
        tile_forward_kernel<T, D, VALS><<<grid, kTileThreads, 0, s>>>(a);
    } else if (what == kTileBwdRows) {
        tile_bwd_rows_kernel<T, D, VALS><<<grid, kTileThreads, 0, s>>>(a);
    } else if constexpr (D <= 64) {
        tile_bwd_cols_kernel<T, D, true, true, VALS><<<grid, kTileThreads, 0, s>>>(a);
    } else {
        if (a.dv) tile_bwd_cols_kernel<T, D, false, true, VALS><<<grid, kTileThreads, 0, s>>>(a);
        if (a.dk) tile_bwd_cols_kernel<T, D, true, false, VALS><<<grid, kTileThreads, 0, s>>>(a);
    }
    SLA_CHECK_LAUNCH();
    return SLA_OK;
}

template <typename T, int D>
sla_status launch_tile(int what, const AttnArgs &a, cudaStream_t s) {
    return a.vals ? launch_tile<T, D, true>(what, a, s) : launch_tile<T, D, false>(what, a, s);
}

template <typename T>
sla_status launch_tile_of(int what, const AttnArgs &a, cudaStream_t s) {
    switch (a.dim) {
        case 16: return launch_tile<T, 16>(what, a, s);
        case 32: return launch_tile<T, 32>(what, a, s);
        case 48: return launch_tile<T, 48>(what, a, s);
        case 64: return launch_tile<T, 64>(what, a, s);
        case 80: return launch_tile<T, 80>(what, a, s);
        case 96: return launch_tile<T, 96>(what, a, s);
        case 112: return launch_tile<T, 112>(what, a, s);
        default: return launch_tile<T, 128>(what, a, s);
    }
}

}  // namespace

sla_status build_tiles(AttnTiles *t, const AttnPlan &parts, int n_rows, const int32_t *rowptr, const int32_t *colind,
                       cudaStream_t s) {
    const int n = parts.n_items, U = parts.n_units;
    DeviceScratch tmp;
    unsigned *count = tmp.get<unsigned>((size_t)n + 1), *chunks = tmp.get<unsigned>((size_t)U + 1);
    void *ws = tmp.get<char>(scan_ws_bytes((int64_t)n + 1));
    if (!count || !chunks || !ws || !alloc_array(&t->chunk0, (size_t)U + 1)) {
        set_error("attention plan: out of device memory");
        return SLA_ERR_OOM;
    }
    const unsigned grid = blocks_of(((int64_t)n + 1) * 32, 128);
    tile_columns_kernel<false><<<grid, 128, 0, s>>>(n_rows, rowptr, colind, n, parts.seg_len, parts.item_unit,
                                                    parts.item_seg, count, nullptr, nullptr, nullptr);
    SLA_CHECK_LAUNCH();
    sla_status st = exclusive_scan(count, count, (int64_t)n + 1, ws, s);
    if (st != SLA_OK) return st;
    tile_chunks_kernel<<<blocks_of(n), 256, 0, s>>>(U, n, count, parts.item_unit, parts.item_seg, chunks);
    SLA_CHECK_LAUNCH();
    st = exclusive_scan(chunks, reinterpret_cast<unsigned *>(t->chunk0), (int64_t)U + 1, ws, s);
    if (st != SLA_OK) return st;
    int32_t total = 0;
    SLA_CHECK_CUDA(cudaMemcpyAsync(&total, t->chunk0 + U, sizeof total, cudaMemcpyDeviceToHost, s));
    SLA_CHECK_CUDA(cudaStreamSynchronize(s));
    if (!alloc_array(&t->chunks, (size_t)total)) {
        set_error("attention plan: out of device memory");
        return SLA_ERR_OOM;
    }
    SLA_CHECK_CUDA(cudaMemsetAsync(t->chunks, 0, (size_t)total * sizeof(TileChunk), s));
    tile_columns_kernel<true><<<grid, 128, 0, s>>>(n_rows, rowptr, colind, n, parts.seg_len, parts.item_unit,
                                                   parts.item_seg, nullptr, count, t->chunk0, t->chunks);
    SLA_CHECK_LAUNCH();
    SLA_CHECK_CUDA(cudaStreamSynchronize(s));
    t->built = true;
    return SLA_OK;
}

template <typename T> sla_status attn_tile_forward(const AttnArgs &a, cudaStream_t s) {
    return launch_tile_of<T>(kTileFwd, a, s);
}
template <typename T> sla_status attn_tile_bwd_rows(const AttnArgs &a, cudaStream_t s) {
    return launch_tile_of<T>(kTileBwdRows, a, s);
}
template <typename T> sla_status attn_tile_bwd_cols(const AttnArgs &a, cudaStream_t s) {
    return launch_tile_of<T>(kTileBwdCols, a, s);
}
template sla_status attn_tile_forward<__nv_bfloat16>(const AttnArgs &, cudaStream_t);
template sla_status attn_tile_forward<__half>(const AttnArgs &, cudaStream_t);
template sla_status attn_tile_bwd_rows<__nv_bfloat16>(const AttnArgs &, cudaStream_t);
template sla_status attn_tile_bwd_rows<__half>(const AttnArgs &, cudaStream_t);
template sla_status attn_tile_bwd_cols<__nv_bfloat16>(const AttnArgs &, cudaStream_t);
template sla_status attn_tile_bwd_cols<__half>(const AttnArgs &, cudaStream_t);

}  // namespace sla
