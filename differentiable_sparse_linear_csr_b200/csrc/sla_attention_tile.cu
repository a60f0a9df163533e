// Attention over a CSR pattern for 16-bit heads, on the tensor cores.
//
// A warp takes 16 consecutive rows of the pattern (a tile), one head and the
// columns that any of those rows stores, 16 at a time (a chunk).  Neighbouring
// rows of a mesh or graph share columns, so a k or v row is fetched once for the
// tile instead of once an entry, and the scores of all 16 x 16 pairs are a
// matrix product; pairs that are not stored are masked by the chunk's row bits.
// Most of that product is thrown away (a 5-point grid uses 5 of 50 columns a row).
//
// Each warp copies the chunk's rows into its own ring of shared-memory stages
// (cp.async, a few chunks ahead: the loads' latency is what the kernels wait for)
// and reads them from there twice, as columns of the scores and as rows of the
// sums.  A dot product does not depend on the order of its terms, so thread (g, c)
// of a quad layout (g = lane / 4, c = lane % 4) takes the 16-byte pieces 8 i + 2c
// and 8 i + 2c + 1 of a column as its places of the k steps 4 i to 4 i + 3, and in
// the sums piece 8 i + g, element e, as output block 8 i + e: whole 16-byte reads.
// Rows lie an odd number of pieces apart (1 modulo 8), which keeps both reads free
// of bank conflicts and every address a constant away from one number a lane.
// Narrow heads go several to a warp, so that a gathered row is at least 128
// consecutive bytes and the chunk's bookkeeping is shared.  Query heads that share
// a key head are rows of one matrix product: 2^k of them with 16 / 2^k rows of the
// pattern, which store fewer different columns, and what is gathered serves all.
//
// Scores: 16-bit products, exact, summed in 32 bits.  Weights are not rounded to
// 16 bits: they multiply as tf32 (the 16-bit operand is exact in it), as a sum of
// two 11-bit parts, which hold a weight to 2^-20 of itself.  One part would show
// where terms cancel: the gradients' weights ds sum to zero over a row, so what its
// keys share must leave no trace in dq (keys with a common offset of 16: dq off by
// 5e-3 with one part), and D = dout . o is subtracted from numbers of its size.
//
// What bounds it is neither the memory (a quarter of the DRAM rate) nor the tensor
// pipe (23 to 36 % active) but chains of dependent instructions, the masked softmax
// of all 256 pairs between two products and reads of shared memory, with 8 to 12
// warps an SM to cover them: issue slots 45 to 53 % busy, most waits for results of
// a fixed latency, then for loads.  Measured: 1024 x 1024 grid, 4 heads of 32
// bfloat16 elements, forward 524 us (2.1 TB/s of the bytes that cannot be left out;
// the row kernels take 772); graph of 100 k rows and 1.2 M entries, 8 heads of 64:
// forward 202 us, dq and ds 208, dk and dv 246, 2.5 to 3.0 TB/s (row kernels 334,
// 458, 406).
//
// Masked pairs have weight 0, but 0 times an infinity or a NaN is a NaN.  A column
// that every row leaves out (values of -inf: padding, which may hold anything) is
// read as zeros.  If a sum ends as a NaN all the same, the warp redoes its rows
// entry by entry: a bad number of a column that some rows use would otherwise
// reach the tile's other rows.
#include <atomic>
#include <climits>

#include "sla_attention.cuh"

namespace sla {
namespace {

constexpr int kTileWarps = 4;
constexpr int kTileThreads = 32 * kTileWarps;
constexpr unsigned kAll = 0xffffffffu;

// ----------------------------------------------------------------- plan ----
// One warp a part of a tile: the columns from one entry of the tile's longest
// row to the entry seg_len further on.  Lane r < rows walks row r's entries
// there, and the smallest column any row is at is the next one.  FILL == false
// counts the columns, each `times` times (a power of two); FILL writes them, at[part]
// places after the first part's.
template <bool FILL>
__global__ void __launch_bounds__(128)
tile_columns_kernel(int rows, int times, int n_rows, const int32_t *__restrict__ rowptr, const int32_t *__restrict__ colind, int n_parts,
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
    const int64_t row = (int64_t)unit * rows + lane;
    int t0 = 0, t1 = 0;
    if (lane < rows && row < n_rows) {
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
            row_bits |= ((1u << times) - 1u) << place;
            cur = next;
            ++t;
            next = t + 1 < t1 ? colind[t + 1] : INT_MAX;
        }
        if (lane >= place) mine = c;            // later places hold the last column until they get theirs
        n += times;
        if (FILL && (n & 15) == 0) flush(16);
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
__device__ __forceinline__ uint4 lds16(unsigned p) {
    uint4 x;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(p));
    return x;
}
__device__ __forceinline__ uint2 lds8(unsigned p) {
    uint2 x;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(p));
    return x;
}
__device__ __forceinline__ uint32_t lds4(unsigned p) {
    uint32_t x;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(p));
    return x;
}

// One head's row: D elements in pieces of 8 (16 bytes).  What a thread takes of it:
//   scores: pieces 8 i + 2c, 8 i + 2c + 1 (i < D / 64), piece c of the next four,
//           8 bytes of the last two;  words 2 s, 2 s + 1 belong to k step s;
//   sums:   pieces 8 i + g (i < D / 64), 8 bytes of the next four, 4 bytes of the
//           last two;  word w holds output blocks 2 w, 2 w + 1.
// Addresses are shared-memory ones; `row` includes nothing of c or g.
template <int D>
__device__ __forceinline__ void read_score(uint32_t (&w)[D / 8], unsigned row, int c) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        const uint4 x = i < D / 64 * 2 ? lds16(row + c * 32 + (i >> 1) * 128 + (i & 1) * 16)
                                       : lds16(row + c * 16 + D / 64 * 128);
        w[4 * i] = x.x;
        w[4 * i + 1] = x.y;
        w[4 * i + 2] = x.z;
        w[4 * i + 3] = x.w;
    }
    if constexpr (D % 32 != 0) {
        const uint2 x = lds8(row + c * 8 + D / 32 * 64);
        w[D / 8 - 2] = x.x;
        w[D / 8 - 1] = x.y;
    }
}

template <int D>
__device__ __forceinline__ void read_sum(uint32_t (&w)[D / 16], unsigned row, int g) {
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        const uint4 x = lds16(row + g * 16 + i * 128);
        w[4 * i] = x.x;
        w[4 * i + 1] = x.y;
        w[4 * i + 2] = x.z;
        w[4 * i + 3] = x.w;
    }
    if constexpr (D % 64 >= 32) {
        const uint2 x = lds8(row + g * 8 + D / 64 * 128);
        w[D / 64 * 4] = x.x;
        w[D / 64 * 4 + 1] = x.y;
    }
    if constexpr (D % 32 != 0) w[D / 16 - 1] = lds4(row + g * 4 + D / 32 * 64);
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

// The same onto zeros.
__device__ __forceinline__ void mma_tf32_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
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

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// Scores less a reference (a number near the maximum), and their
// exponential.  Without values both are in units of log 2: the factor log2 e is
// part of `scale`, so that the difference is one multiply-add.  Values come in
// natural units, and the factor is applied to the difference, so that the lowest
// finite value does not overflow.
template <bool VALS>
__device__ __forceinline__ float relative(float dot, float scale, float val, float ref) {
    if constexpr (VALS) return fmaf(dot, scale, val) - ref;
    else return fmaf(dot, scale, -ref);
}
template <bool VALS>
__device__ __forceinline__ float weight(float t) { return exp2_of(VALS ? t * kLog2e : t); }
template <bool VALS>
__device__ __forceinline__ float score_scale(double scale) {
    return VALS ? (float)scale : (float)(scale * 1.4426950408889634);
}

// Bits of the pairs (row g + 8 (e / 2), column 8 blk + 2c + e % 2) in a row's
// bits shifted by 2c.
__device__ __forceinline__ unsigned pair_bit(int blk, int e) { return 1u << (8 * blk + (e & 1)); }


// The rows g and g + 8 of a tile's matrix product: row of the tile and query head
// (PACK: several heads; else row g + 8 i of head 0).
template <bool PACK>
struct TileRows {
    int r[2], h[2];
    __device__ __forceinline__ TileRows(int rows_log, int g) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            r[i] = PACK ? (g + 8 * i) & ((1 << rows_log) - 1) : g + 8 * i;
            h[i] = PACK ? (g + 8 * i) >> rows_log : 0;
        }
    }
};

// The tile's own 16 rows as the left operand of score products.
template <int D>
struct Own {
    uint32_t a[D / 16][4];
    // `stride`: bytes from row to row, below 2^32; `head`: elements between heads.
    template <typename T, bool PACK>
    __device__ __forceinline__ void load(const T *base, unsigned stride, int64_t head, const TileRows<PACK> &t, int row0, int n_rows,
                                         int c) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const bool on = row0 + t.r[i] < n_rows;
            const char *p = reinterpret_cast<const char *>(base + t.h[i] * head) + (uint64_t)(unsigned)(row0 + t.r[i]) * stride;
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                const int at = j < D / 64 * 2 ? c * 2 + (j >> 1) * 8 + (j & 1) : c + D / 64 * 8;
                const uint4 x = on ? __ldg(reinterpret_cast<const uint4 *>(p) + at) : make_uint4(0, 0, 0, 0);
                a[2 * j][i] = x.x;
                a[2 * j][2 + i] = x.y;
                a[2 * j + 1][i] = x.z;
                a[2 * j + 1][2 + i] = x.w;
            }
            if constexpr (D % 32 != 0) {
                const uint2 x = on ? __ldg(reinterpret_cast<const uint2 *>(p + D / 32 * 64) + c) : make_uint2(0, 0);
                a[D / 16 - 1][i] = x.x;
                a[D / 16 - 1][2 + i] = x.y;
            }
        }
    }
};

// s[2][4]: the products of the 16 own rows with the 16 staged columns of a chunk,
// the columns 8 blk + (2c, 2c + 1) of rows g and g + 8 in this thread.
template <typename T, int D, int PITCH>
__device__ __forceinline__ void score_products(float (&s)[2][4], const Own<D> &own, unsigned stage, int g, int c) {
    // the halves alternate, so that a product does not wait for the one before it
    uint32_t k[2][D / 8];
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
        read_score<D>(k[blk], stage + g * PITCH + 8 * blk * PITCH, c);
        s[blk][0] = s[blk][1] = s[blk][2] = s[blk][3] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) mma16<T>(s[blk], own.a[i], k[blk][2 * i], k[blk][2 * i + 1]);
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

// Sums over a chunk's columns: o[nb] += w . x, with x the rows of the columns
// 8 blk + (2c, 2c + 1).
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
    // The weights of one half of a chunk in two parts.
    static __device__ __forceinline__ void split(const float (&w)[4], uint32_t (&hi)[4], uint32_t (&lo)[4]) {
        const float v[4] = {w[0], w[2], w[1], w[3]};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            hi[i] = __float_as_uint(v[i]) & 0xffffe000u;
            lo[i] = __float_as_uint(v[i] - __uint_as_float(hi[i]));
        }
    }
    // The tensor core drops the bits that its 32-bit sums cannot hold, always towards
    // zero, so a sum that stayed in it over a long row would drift (1500 entries: by
    // 3.6e-6, a row of products in rounded sums 5e-7).  A chunk is summed from zero
    // there and added to the running sums with rounding to nearest.
    __device__ __forceinline__ void add(const float (&w)[2][4], const uint32_t (&x)[4][D / 16]) {
        uint32_t hi[2][4], lo[2][4];
        split(w[0], hi[0], lo[0]);
        split(w[1], hi[1], lo[1]);
        // four blocks at a time, so that a product does not wait for the one before it
        constexpr int W = D / 16, G = W % 2 == 0 ? 2 : 1;
#pragma unroll
        for (int j = 0; j < W; j += G) {
            float t[2 * G][4];
            uint32_t y[G][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int i = 0; i < G; ++i) {
                    widen<T>(x[2 * h][j + i], y[i][0], y[i][1]);
                    widen<T>(x[2 * h + 1][j + i], y[i][2], y[i][3]);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (h == 0) mma_tf32_first(t[2 * i + e], hi[0], y[i][e], y[i][2 + e]);
                        else mma_tf32(t[2 * i + e], hi[1], y[i][e], y[i][2 + e]);
                    }
                }
#pragma unroll
                for (int i = 0; i < G; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) mma_tf32(t[2 * i + e], lo[h], y[i][e], y[i][2 + e]);
            }
#pragma unroll
            for (int i = 0; i < 2 * G; ++i) {
                float (&to)[4] = o[2 * j + i];
                const float2 a = add2(make_float2(to[0], to[1]), make_float2(t[i][0], t[i][1])),
                             b = add2(make_float2(to[2], to[3]), make_float2(t[i][2], t[i][3]));
                to[0] = a.x;
                to[1] = a.y;
                to[2] = b.x;
                to[3] = b.y;
            }
        }
    }
    // A NaN among the sums of any thread (or infinities of both signs).
    __device__ __forceinline__ bool bad() const {
        float2 t = make_float2(0.0f, 0.0f);
        const float2 one = make_float2(1.0f, 1.0f);
#pragma unroll
        for (int nb = 0; nb < D / 8; ++nb) {
            t = fma2(make_float2(o[nb][0], o[nb][1]), one, t);
            t = fma2(make_float2(o[nb][2], o[nb][3]), one, t);
        }
        const float u = t.x + t.y;
        return __any_sync(kAll, u != u);
    }
    // All of a chunk: the weights w[2][4] with the staged rows.  drop, used: see
    // drop_unused.
    template <int PITCH>
    __device__ __forceinline__ void add_chunk(const float (&w)[2][4], unsigned stage, int g, int c, bool drop,
                                              unsigned used) {
        uint32_t x[4][D / 16];
#pragma unroll
        for (int j = 0; j < 4; ++j) read_sum<D>(x[j], stage + 2 * c * PITCH + (8 * (j >> 1) + (j & 1)) * PITCH, g);
        if (drop) drop_unused(x, used);
        add(w, x);
    }
    // Row g (i = 0) or g + 8 (i = 1) to its D elements at p.  Of every group of
    // blocks this thread holds consecutive elements, first those of column 2c.
    template <typename O>
    __device__ __forceinline__ void store(O *p, int i, int c) const {
#pragma unroll
        for (int j = 0; j < D / 64; ++j) put<O, 8>(p + 64 * j + 16 * c, 8 * j, i);
        if constexpr (D % 64 >= 32) put<O, 4>(p + D / 64 * 64 + 8 * c, D / 64 * 8, i);
        if constexpr (D % 32 != 0) put<O, 2>(p + D / 32 * 32 + 4 * c, D / 8 - 2, i);
    }
    template <typename O, int N>
    __device__ __forceinline__ void put(O *p, int nb, int i) const {
        float x[2 * N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
            x[e] = o[nb + e][2 * i];
            x[N + e] = o[nb + e][2 * i + 1];
        }
        if constexpr (sizeof(O) == 4) {
#pragma unroll
            for (int e = 0; e < N / 2; ++e)
                reinterpret_cast<float4 *>(p)[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
        } else if constexpr (N >= 4) {
#pragma unroll
            for (int e = 0; e < N / 4; ++e)
                reinterpret_cast<uint4 *>(p)[e] =
                    make_uint4(narrow2<T>(x[8 * e], x[8 * e + 1]), narrow2<T>(x[8 * e + 2], x[8 * e + 3]),
                               narrow2<T>(x[8 * e + 4], x[8 * e + 5]), narrow2<T>(x[8 * e + 6], x[8 * e + 7]));
        } else {
            *reinterpret_cast<uint2 *>(p) = make_uint2(narrow2<T>(x[0], x[1]), narrow2<T>(x[2], x[3]));
        }
    }
};

// A piece of work: chunks [ch0, ch1) of a tile, heads h (and following) of one
// system, whose key heads start at kh.
struct TileWork {
    int row0, b, h, kh, slot, ch0, ch1;
};

// The pieces of work a warp takes, every `stride`-th of the list ordered by
// system, key head, tile and query head: the warps of the GPU sweep the pattern
// together, one key head (or group) after the other, so that the rows it gathers
// stay in the L2 cache.
struct Cursor {
    unsigned x;                // place within a (system, key head group): item * groups + group
    int b, kh;                 // system, first key head
    __device__ __forceinline__ unsigned item(unsigned groups) const { return groups == 1 ? x : x / groups; }
    __device__ __forceinline__ int head(unsigned groups, int share) const {
        return kh * share + (groups == 1 ? 0 : (int)(x % groups) * (share / (int)groups));
    }
};
struct Stride {
    unsigned per_y, x;         // the stride in the cursor's three digits
    int b, kh, n_kh, kv_heads;
    __device__ __forceinline__ Stride(unsigned by, unsigned items, unsigned groups, int n_kh_, int kv_heads_)
        : per_y(items * groups), n_kh(n_kh_), kv_heads(kv_heads_) {
        const Cursor c = at(by);
        x = c.x;
        b = c.b;
        kh = c.kh;
    }
    __device__ __forceinline__ Cursor at(unsigned place) const {
        const unsigned y = place / per_y, ky = (unsigned)(kv_heads / n_kh);
        Cursor c;
        c.x = place - y * per_y;
        c.b = (int)(y / ky);
        c.kh = (int)(y - (unsigned)c.b * ky) * n_kh;
        return c;
    }
    __device__ __forceinline__ void move(Cursor &c) const {
        c.x += x;
        c.kh += kh;
        c.b += b;
        if (c.x >= per_y) {
            c.x -= per_y;
            c.kh += n_kh;
        }
        if (c.kh >= kv_heads) {
            c.kh -= kv_heads;
            ++c.b;
        }
    }
};

__device__ __forceinline__ int2 item_range(const AttnArgs &a, unsigned it) {
    if (a.item_chunks) return __ldg(a.item_chunks + it);
    return make_int2(__ldg(a.chunk0 + it), __ldg(a.chunk0 + it + 1));
}

__device__ __forceinline__ TileWork tile_work(const AttnArgs &a, const Cursor &c, unsigned groups, int share, int rows_log) {
    TileWork w;
    const unsigned it = c.item(groups);
    w.b = c.b;
    w.kh = c.kh;
    w.h = c.head(groups, share);
    w.row0 = (a.item_unit ? __ldg(a.item_unit + it) : (int)it) << rows_log;
    w.slot = a.item_unit ? __ldg(a.item_slot + it) : -1;
    const int2 r = item_range(a, it);
    w.ch0 = r.x;
    w.ch1 = r.y;
    return w;
}

// Brings the lines of a tile's rows, which will be loaded soon, into the L2 cache:
// lane m < 16 names row m of its matrix product, of D elements.
template <typename T, int D>
__device__ __forceinline__ void prefetch_rows(const T *base, int64_t stride, int64_t head, int rows_log, int row0, int n_rows,
                                              int lane) {
    const int r = row0 + (lane & ((1 << rows_log) - 1));
    if (lane < kTileRows && r < n_rows) {
        const T *p = base + (int64_t)r * stride + (lane >> rows_log) * head;
#pragma unroll
        for (int i = 0; i < D; i += 64) asm volatile("prefetch.global.L2 [%0];" :: "l"(p + i));
    }
}

// What a thread keeps of a chunk: rows g's and g + 8's bits and, with ENTRIES,
// their first entries.
template <bool ENTRIES>
struct Chunk {
    unsigned bits[2];
    int at[2];
    template <bool PACK>
    __device__ __forceinline__ void load(const TileChunk *chunks, int ch, const TileRows<PACK> &t) {
        const TileChunk *p = chunks + ch;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            bits[i] = __ldg(p->bits + t.r[i]);
            if constexpr (ENTRIES) at[i] = __ldg(p->start + t.r[i]);
        }
    }
    // Entries of rows g and g + 8 at columns 8 blk + 2c (the next column's entry
    // follows if the row stores both).
    // times: the log of how often the chunk repeats a column.
    __device__ __forceinline__ int entry(int i, int blk, int c, int times = 0) const {
        return at[i] + (__popc(bits[i] & ((1u << (8 * blk + 2 * c)) - 1u)) >> times);
    }
    // The stored values of this thread's 8 pairs, 0 where nothing is stored.
    __device__ __forceinline__ void values(float (&x)[2][4], const float *vals, int c, int times = 0) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const unsigned mine = bits[i] >> (2 * c);
#pragma unroll
            for (int blk = 0; blk < 2; ++blk) {
                const float *p = vals + entry(i, blk, c, times);
                x[blk][2 * i] = mine & pair_bit(blk, 0) ? __ldg(p) : 0.0f;
                x[blk][2 * i + 1] = mine & pair_bit(blk, 1) ? __ldg(p + (times ? 0 : mine >> (8 * blk) & 1)) : 0.0f;
            }
        }
    }
};

__device__ __forceinline__ void cp_async16(unsigned dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

// A warp's ring of stages: two gathered tensors of HEADS heads, 16 rows each,
// and with STAT four numbers a column and head.  The padded pitch beats pieces
// permuted in an unpadded row (by 7 % on the 1024 x 1024 grid): no
// address arithmetic at a read.  Three stages where 12 warps' rings (8 with STAT) fit an SM.
template <int D, int HEADS, bool STAT>
struct Ring {
    static constexpr int kPieces = D / 8 * HEADS;                       // of a row
    static constexpr int kPitch = (kPieces + 7) / 8 * 128 + 16;
    static constexpr int kTensor = 16 * kPitch;
    static constexpr int kStage = 2 * kTensor + (STAT ? 16 * 16 * HEADS : 0);
    static constexpr int kStages = kStage <= (STAT ? 5632 : 5120) ? 3 : 2;
    static constexpr int kBytes = kStage * kStages;
    static constexpr bool kEven = 32 % kPieces == 0;                    // a lane has one piece of every row it copies

    // Where this lane's pieces start in a tensor, with a head's stride in bytes.
    static __device__ __forceinline__ const char *source(const void *base, int64_t head_bytes, int lane) {
        const char *p = static_cast<const char *>(base);
        if constexpr (!kEven) return p;
        const int x = lane % kPieces;
        return p + x / (D / 8) * head_bytes + x % (D / 8) * 16;
    }
    // Copies of both tensors' rows of the columns in `col` (lane r: column r).  times:
    // the log of how often a column is repeated, for the next heads (head0, head1
    // bytes apart).
    static __device__ __forceinline__ void gather(unsigned stage, const char *p0, unsigned stride0, const char *p1,
                                                  unsigned stride1, unsigned col, int lane, int times = 0,
                                                  int64_t head0 = 0, int64_t head1 = 0) {
#pragma unroll
        for (int i = 0; i < kPieces / 2; ++i) {
            const int x = i * 32 + lane, r = kEven ? lane / kPieces + i * (32 / kPieces) : x / kPieces;
            const int p = kEven ? lane % kPieces : x - r * kPieces;
            const unsigned cl = __shfl_sync(kAll, col, r), dst = stage + r * kPitch + p * 16;
            const int more = kEven ? 0 : p * 16;       // several heads are even (whole powers of two)
            const char *s0 = p0 + (uint64_t)cl * stride0 + more, *s1 = p1 + (uint64_t)cl * stride1 + more;
            if (times) {
                s0 += (r & ((1 << times) - 1)) * head0;
                s1 += (r & ((1 << times) - 1)) * head1;
            }
            cp_async16(dst, s0);
            cp_async16(dst + kTensor, s1);
        }
    }
};

__device__ __forceinline__ unsigned chunk_column(const TileChunk *chunks, int ch, int lane, int n_cols) {
#if SLA_DEBUG_BOUNDS
    return (unsigned)SLA_IDX(__ldg(chunks[ch].col + (lane & 15)), n_cols, kBndColumn);
#else
    (void)n_cols;
    return (unsigned)__ldg(chunks[ch].col + (lane & 15));
#endif
}

// Entry range of row r of the tile in the item (every lane r < 16 its own row); times:
// the log of how often a column is repeated.
__device__ __forceinline__ void row_range(const TileChunk *chunks, const TileWork &w, int lane, int times, int &t0, int &t1) {
    t0 = t1 = 0;
    if (lane < kTileRows && w.ch0 < w.ch1) {
        t0 = t1 = __ldg(chunks[w.ch0].start + lane);
        for (int ch = w.ch0; ch < w.ch1; ++ch) t1 += __popc((unsigned)__ldg(chunks[ch].bits + lane)) >> times;
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
    row_range(a.chunks, w, lane, 0, s0, s1);
    const T *qb = static_cast<const T *>(a.q) + w.b * a.qs[0] + w.h * a.qs[2];
    const T *kb = static_cast<const T *>(a.k) + w.b * a.ks[0] + w.kh * a.ks[2];
    const T *vb = static_cast<const T *>(a.v) + w.b * a.vs[0] + w.kh * a.vs[2];
    const float scale = (float)a.scale, none = neg_inf<float>();
    for (int r = 0; r < 1 << a.rows_log && w.row0 + r < a.n_rows; ++r) {
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
            const float ref = top == none ? 0.0f : top, fix = exp_acc(m - ref), p = exp_acc(s - ref);
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
            if (lane == 0) store_lse(a, at, m, l);
        } else {
            const int64_t at = part_index(w.slot, a.n_slots, w.b, 1 << a.rows_log, r, a.heads, w.h);
            float *p = static_cast<float *>(a.part) + at * a.dim;
#pragma unroll
            for (int i = 0; i < kSlowVec; ++i)
                if (i * 32 + lane < a.dim) p[i * 32 + lane] = acc[i];
            if (lane == 0) static_cast<float2 *>(a.part_ml)[at] = make_float2(m, l);
        }
    }
}

// The producing side of a warp's ring: copies chunk after chunk, across the
// pieces of work, ahead of the consuming loop.  `open(cursor)` is called at the
// first chunk of a piece, `copy(stage, col)` for every chunk.
template <typename R>
struct Feed {
    Cursor cur;
    unsigned left, col;                    // pieces of work not yet begun; columns of the chunk at `at`
    int at, end;
    int2 next;                             // chunks of the piece after this one
    int write;
    bool more;

    // The next chunk, if there is one.
    template <typename Open>
    __device__ __forceinline__ void seek(const AttnArgs &a, const Stride &stride, unsigned groups, Open &&open) {
        while (at == end) {
            if (left == 0) {
                more = false;
                at = end > 0 ? end - 1 : 0;      // some chunk, for the load that follows
                return;
            }
            --left;
            at = next.x;
            end = next.y;
            open(cur);
            if (left > 0) {
                stride.move(cur);
                next = item_range(a, cur.item(groups));
            }
        }
    }
    template <typename Open>
    __device__ __forceinline__ void start(const AttnArgs &a, const Cursor &c, unsigned count, const Stride &stride, unsigned groups,
                                          int lane, int n_cols, Open &&open) {
        cur = c;
        left = count;
        at = end = 0;
        write = 0;
        more = true;
        if (count > 0) next = item_range(a, cur.item(groups));
        seek(a, stride, groups, open);
        col = chunk_column(a.chunks, at, lane, n_cols);
    }
    // The columns are loaded in every call, needed or not: a load under a condition
    // would be waited for where its paths join, not where it is used.
    template <typename Open, typename Copy>
    __device__ __forceinline__ void advance(const AttnArgs &a, const Stride &stride, unsigned groups, int lane, int n_cols, unsigned ring,
                                            Open &&open, Copy &&copy) {
        if (more) {
            copy(ring + write, col);
            write = write == (R::kStages - 1) * R::kStage ? 0 : write + R::kStage;
            if (++at == end) seek(a, stride, groups, open);
        }
        cp_commit();
        col = chunk_column(a.chunks, at, lane, n_cols);
    }
};

// What the consuming loop needs of the chunks to come, loaded as the feed passes
// them and so across the pieces of work too: bits and first entries, and with VALS
// the stored values one chunk ahead.  base: the values of system 0; times: see Chunk.
template <bool VALS, typename R>
struct Ahead {
    static constexpr bool kTwo = R::kStages == 3;        // the feed is two chunks ahead, or one
    Chunk<VALS> now, c0, c1;                             // the chunk at hand and the next ones
    float x[2][4], x_next[2][4];
    int b0, b1;

    template <bool PACK>
    __device__ __forceinline__ void first(const TileChunk *chunks, int at, int b, const TileRows<PACK> &rows) {
        c0.load(chunks, at, rows);
        b0 = b;
    }
    template <bool PACK>
    __device__ __forceinline__ void second(const TileChunk *chunks, int at, int b, const TileRows<PACK> &rows) {
        c1.load(chunks, at, rows);
        b1 = b;
    }
    __device__ __forceinline__ void start(const float *base, int64_t nnz, int c, int times = 0) {
        if constexpr (VALS) c0.values(x_next, base + b0 * nnz, c, times);
    }
    // Takes the next chunk; then `passed` with the chunk the feed is about to copy.
    __device__ __forceinline__ void take(const float *base, int64_t nnz, int c, int times = 0) {
        now = c0;
        if constexpr (VALS) {
#pragma unroll
            for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[blk][e] = x_next[blk][e];
            if constexpr (kTwo) c1.values(x_next, base + b1 * nnz, c, times);
        }
        if constexpr (kTwo) {
            c0 = c1;
            b0 = b1;
        }
    }
    template <bool PACK>
    __device__ __forceinline__ void passed(const TileChunk *chunks, int at, int b, const TileRows<PACK> &rows) {
        if constexpr (kTwo) second(chunks, at, b, rows);
        else first(chunks, at, b, rows);
    }
    // With the feed one chunk ahead the next values are loaded when its bits are there.
    __device__ __forceinline__ void late(const float *base, int64_t nnz, int c, int times = 0) {
        if constexpr (VALS && !kTwo) c0.values(x_next, base + b0 * nnz, c, times);
    }
};

// Pieces of work of this warp out of `total`.
__device__ __forceinline__ unsigned my_share(unsigned total, unsigned &first, unsigned &stride) {
    first = blockIdx.x * kTileWarps + (threadIdx.x >> 5);
    stride = gridDim.x * kTileWarps;
    return first < total ? (total - first + stride - 1) / stride : 0;
}

// KH key heads a warp; with one, the query heads of the tile share it.
// Blocks an SM, here and below: 3 while the sums and the own rows leave room in 168
// registers, else 2.  (1024 x 1024 grid, 2 heads of 32 a warp: 524 us with 3, 597
// with 2, 536 with 4 and spills; forward of the graph 202, 222 and 297.)
template <typename T, int D, int KH, bool VALS, bool PACK>
__global__ void __launch_bounds__(kTileThreads, D * KH <= 64 && !(PACK && VALS) ? 3 : 2)
tile_forward_kernel(const __grid_constant__ AttnArgs a, unsigned total) {
    using R = Ring<D, KH, false>;
    extern __shared__ __align__(128) char smem[];
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, share = a.heads / a.kv_heads;
    const unsigned ring = (unsigned)__cvta_generic_to_shared(smem) + (threadIdx.x >> 5) * R::kBytes;
    const unsigned groups = PACK ? (unsigned)share >> (4 - a.rows_log) : (unsigned)share;    // of query heads on a key head
    const TileRows<PACK> rows(a.rows_log, g);
    const unsigned qst = (unsigned)a.qs[1] * 2, kst = (unsigned)a.ks[1] * 2, vst = (unsigned)a.vs[1] * 2;
    const float scale = score_scale<VALS>(a.scale), none = neg_inf<float>();
    unsigned first, by;
    const unsigned count = my_share(total, first, by);
    if (count == 0) return;
    const Stride stride(by, (unsigned)a.n_items, groups, KH, a.kv_heads);
    Cursor now = stride.at(first);
    Feed<R> feed;
    const char *kb = nullptr, *vb = nullptr;             // of the piece the feed is at, and its system
    int fb = 0;
    auto open = [&](const Cursor &f) {
        fb = f.b;
        kb = R::source(static_cast<const T *>(a.k) + f.b * a.ks[0] + f.kh * a.ks[2], a.ks[2] * 2, lane);
        vb = R::source(static_cast<const T *>(a.v) + f.b * a.vs[0] + f.kh * a.vs[2], a.vs[2] * 2, lane);
        const unsigned it = f.item(groups);
        const int row0 = (a.item_unit ? __ldg(a.item_unit + it) : (int)it) << a.rows_log;
        prefetch_rows<T, D * KH>(static_cast<const T *>(a.q) + f.b * a.qs[0] + f.head(groups, share) * a.qs[2], a.qs[1],
                                 a.qs[2], a.rows_log, row0, a.n_rows, lane);
    };
    auto copy = [&](unsigned st, unsigned col) { R::gather(st, kb, kst, vb, vst, col, lane); };
    feed.start(a, now, count, stride, groups, lane, a.n_cols, open);
    Ahead<VALS, R> meta;
    meta.first(a.chunks, feed.at, fb, rows);
    feed.advance(a, stride, groups, lane, a.n_cols, ring, open, copy);
    if constexpr (meta.kTwo) {
        meta.second(a.chunks, feed.at, fb, rows);
        feed.advance(a, stride, groups, lane, a.n_cols, ring, open, copy);
    }
    meta.start(a.vals_f, a.nnz, c);
    int st_read = 0;
    TileWork w_next = tile_work(a, now, groups, share, PACK ? a.rows_log : 4);
    for (unsigned piece = 0; piece < count; ++piece) {
        const TileWork w = w_next;
        if (piece + 1 < count) stride.move(now);
        w_next = tile_work(a, now, groups, share, PACK ? a.rows_log : 4);
        const int n = w.ch1 - w.ch0;
        Own<D> q[KH];
#pragma unroll
        for (int j = 0; j < KH; ++j)
            q[j].load(static_cast<const T *>(a.q) + w.b * a.qs[0] + (w.h + j) * a.qs[2], qst, a.qs[2], rows, w.row0, a.n_rows, c);
        Sums<T, D> acc[KH];
        float m[KH][2], l[KH][2];
#pragma unroll
        for (int j = 0; j < KH; ++j) {
            acc[j].zero();
            m[j][0] = m[j][1] = l[j][0] = l[j][1] = 0.0f;
        }
        for (int ch = 0; ch < n; ++ch) {
            meta.take(a.vals_f, a.nnz, c);
            cp_wait<R::kStages - 2>();
            __syncwarp();
            meta.passed(a.chunks, feed.at, fb, rows);
            feed.advance(a, stride, groups, lane, a.n_cols, ring, open, copy);
            const unsigned stage = ring + st_read;
            st_read = st_read == (R::kStages - 1) * R::kStage ? 0 : st_read + R::kStage;
            const auto &x = meta.x;
            unsigned mine[2] = {meta.now.bits[0] >> (2 * c), meta.now.bits[1] >> (2 * c)}, used = 0;
            bool drop = false;
            if constexpr (VALS) {
                bool out = false;                       // a stored pair that a value of -inf leaves out
#pragma unroll
                for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (x[blk][e] == none) {
                            mine[e >> 1] &= ~pair_bit(blk, e);
                            out = true;
                        }
                drop = __any_sync(kAll, out);
                if (drop) {
                    if (!__any_sync(kAll, (mine[0] | mine[1]) & 0x303u)) {              // nothing left
                        meta.late(a.vals_f, a.nnz, c);
                        continue;
                    }
                    used = (mine[0] | mine[1]) & 0x303u;
                    used = (used | used >> 6) & 15u;
                }
            }
#pragma unroll
            for (int j = 0; j < KH; ++j) {
                const unsigned at = stage + (KH == 1 ? 0 : j * (D * 2));
                float s[2][4], t[2][4], far[2] = {none, none};
                score_products<T, D, R::kPitch>(s, q[j], at, g, c);
                if (j == 0) meta.late(a.vals_f, a.nnz, c);
#pragma unroll
                for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        t[blk][e] = relative<VALS>(s[blk][e], scale, x[blk][e], m[j][e >> 1]);
                        t[blk][e] = mine[e >> 1] & pair_bit(blk, e) ? t[blk][e] : none;
                        far[e >> 1] = fmaxf(far[e >> 1], t[blk][e]);
                    }
                // Any reference that keeps a row's first weights between 2^-20 and 2^8 will
                // do; 0 mostly is one.  It moves when a score is beyond: up at any time,
                // down only while the row has no weight.
                constexpr float kUnit = VALS ? kLn2 : 1.0f;
                const bool up = far[0] > 8.0f * kUnit || far[1] > 8.0f * kUnit;
                const bool down = (far[0] < -20.0f * kUnit && l[j][0] == 0.0f && far[0] != none) ||
                                  (far[1] < -20.0f * kUnit && l[j][1] == 0.0f && far[1] != none);
                if (__any_sync(kAll, up || down)) {
                    // Taken from the scores themselves: a difference to a reference of -1e10,
                    // say, would hold none of their digits.
                    float sum[2] = {l[j][0], l[j][1]}, top[2] = {none, none}, f[2];
#pragma unroll
                    for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (mine[e >> 1] & pair_bit(blk, e))
                                top[e >> 1] = fmaxf(top[e >> 1], relative<VALS>(s[blk][e], scale, x[blk][e], 0.0f));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
#pragma unroll
                        for (int o = 1; o < 4; o += o) {
                            top[i] = fmaxf(top[i], __shfl_xor_sync(kAll, top[i], o));
                            sum[i] += __shfl_xor_sync(kAll, sum[i], o);
                        }
                        const float to = top[i] == none ? m[j][i] : (sum[i] == 0.0f ? top[i] : fmaxf(m[j][i], top[i]));
                        f[i] = to == m[j][i] || sum[i] == 0.0f ? 1.0f : weight<VALS>(m[j][i] - to);
                        l[j][i] *= f[i];
                        m[j][i] = to;
                    }
                    acc[j].scale(f[0], f[1]);
#pragma unroll
                    for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            t[blk][e] = relative<VALS>(s[blk][e], scale, x[blk][e], m[j][e >> 1]);
                            t[blk][e] = mine[e >> 1] & pair_bit(blk, e) ? t[blk][e] : none;
                        }
                }
#pragma unroll
                for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[blk][e] = weight<VALS>(t[blk][e]);
                        l[j][e >> 1] += s[blk][e];
                    }
                acc[j].template add_chunk<R::kPitch>(s, at + R::kTensor, g, c, VALS && drop, used);
            }
        }
        // A NaN among the sums, or a sum of weights that is none (which the outputs
        // would not show).
        bool bad = false;
#pragma unroll
        for (int j = 0; j < KH; ++j) bad = acc[j].bad() || __any_sync(kAll, l[j][0] != l[j][0] || l[j][1] != l[j][1]) || bad;
        if (bad) {
            const int heads = KH == 1 ? kTileRows >> a.rows_log : KH;
            for (int j = 0; j < heads; ++j) {
                TileWork one = w;
                one.h = w.h + j;
                one.kh = KH == 1 ? w.kh : w.kh + j;
                slow_forward<T>(a, one);
            }
            continue;
        }
        const int64_t at0 = ((int64_t)w.b * a.n_rows + w.row0) * a.heads + w.h;     // row row0, head h
        const unsigned step = (unsigned)a.heads;
#pragma unroll
        for (int j = 0; j < KH; ++j) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                l[j][i] += __shfl_xor_sync(kAll, l[j][i], 1);
                l[j][i] += __shfl_xor_sync(kAll, l[j][i], 2);
            }
            if (w.slot < 0) acc[j].scale(l[j][0] > 0.0f ? __fdividef(1.0f, l[j][0]) : 0.0f,
                                         l[j][1] > 0.0f ? __fdividef(1.0f, l[j][1]) : 0.0f);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = rows.r[i], h = rows.h[i] + j;
                if (w.row0 + r >= a.n_rows) continue;
                // no weight: lse is -inf
                const float top = l[j][i] == 0.0f ? none : (VALS ? m[j][i] : m[j][i] * kLn2);
                if (w.slot < 0) {
                    const int64_t o = at0 + (uint64_t)(unsigned)r * step + h;
                    acc[j].store(static_cast<T *>(a.out) + o * D, i, c);
                    if (a.wide) acc[j].store(static_cast<float *>(a.wide) + o * D, i, c);
                    if (c == 0) {
                        if (a.lse_pairs) {
                            // The sum takes what m's return to natural units rounds away, so that the
                            // two agree when the backward goes back to units of log 2.
                            float sum = l[j][i];
                            if (!VALS && sum > 0.0f) sum *= exp2_of(fminf(fmaxf(m[j][i] - top * kLog2e, -64.0f), 64.0f));
                            static_cast<float2 *>(a.lse)[o] = make_float2(top, sum);
                        } else {
                            static_cast<float *>(a.lse)[o] = top + __log2f(l[j][i] == 0.0f ? 1.0f : l[j][i]) * kLn2;
                        }
                    }
                } else {
                    const int64_t at = part_index(w.slot, a.n_slots, w.b, 1 << a.rows_log, r, a.heads, w.h + h);
                    acc[j].store(static_cast<float *>(a.part) + at * D, i, c);
                    if (c == 0) static_cast<float2 *>(a.part_ml)[at] = make_float2(top, l[j][i]);
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
    row_range(a.chunks, w, lane, 0, s0, s1);
    const T *kb = static_cast<const T *>(a.k) + w.b * a.ks[0] + w.kh * a.ks[2];
    const T *vb = static_cast<const T *>(a.v) + w.b * a.vs[0] + w.kh * a.vs[2];
    const float scale = (float)a.scale, none = neg_inf<float>();
    for (int r = 0; r < 1 << a.rows_log && w.row0 + r < a.n_rows; ++r) {
        const int t0 = __shfl_sync(kAll, s0, r), t1 = __shfl_sync(kAll, s1, r);
        const int64_t row = w.row0 + r, at = ((int64_t)w.b * a.n_rows + row) * a.heads + w.h;
        float q[kSlowVec], go[kSlowVec], o[kSlowVec], acc[kSlowVec] = {};
        slow_load(q, static_cast<const T *>(a.q) + w.b * a.qs[0] + row * a.qs[1] + w.h * a.qs[2], a.dim, lane);
        slow_load(go, static_cast<const T *>(a.dout) + w.b * a.ds[0] + row * a.ds[1] + w.h * a.ds[2], a.dim, lane);
        slow_load(o, static_cast<const float *>(a.o) + at * a.dim, a.dim, lane);
        const float delta = slow_dot(go, o);
        const float2 ml = static_cast<const float2 *>(a.lse)[at];
        const float inv = 1.0f / ml.y;
        for (int t = t0; t < t1 && ml.y != 0.0f; ++t) {
            const int64_t col = SLA_IDX((int64_t)__ldg(a.colind + t), a.n_cols, kBndColumn);
            const float x = load_value<float>(a.vals, a.vals_f64, w.b * a.nnz + t);
            if (x == none) continue;
            float k[kSlowVec], v[kSlowVec];
            slow_load(k, kb + col * a.ks[1], a.dim, lane);
            slow_load(v, vb + col * a.vs[1], a.dim, lane);
            const float p = exp_acc(fmaf(slow_dot(q, k), scale, x) - ml.x) * inv;
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
                    static_cast<float *>(a.part)[part_index(w.slot, a.n_slots, w.b, 1 << a.rows_log, r, a.heads, w.h) * a.dim + d] =
                        acc[i] * scale;
            }
    }
}

// (m, 1 / l, D / l) with D = dout . o of every row and head, for both kernels below; m
// in the unit of relative(), -inf where the row has no weight.  A weight's derivative
// p (dp - D) is then exp(s - m) (dp / l - D / l), one multiply-add as without l.
// G lanes a row and head, 8 elements each.  Bound by memory: 100 k rows, 8 heads of
// 64, 326 MB in 54 to 60 us (5.4 to 6.0 TB/s).
template <typename T, int G>
__global__ void __launch_bounds__(256) tile_delta_kernel(const __grid_constant__ AttnArgs a, int64_t count, float unit) {
    const int64_t x = (blockIdx.x * (int64_t)256 + threadIdx.x) / G;
    const int l = threadIdx.x % G;
    if (x - threadIdx.x % 32 / G >= count) return;       // whole warps
    const int64_t row = x / a.heads, b = row / a.n_rows;
    const int h = (int)(x - row * a.heads);
    float s = 0.0f;
    if (x < count && l * 8 < a.dim) {
        const uint4 d = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(a.dout) + b * a.ds[0] +
                                                              (row - b * a.n_rows) * a.ds[1] + h * a.ds[2]) + l);
        const float4 *o = reinterpret_cast<const float4 *>(static_cast<const float *>(a.o) + x * a.dim) + 2 * l;
        const float4 o0 = __ldg(o), o1 = __ldg(o + 1);
        uint32_t e[8];
        widen<T>(d.x, e[0], e[1]);
        widen<T>(d.y, e[2], e[3]);
        widen<T>(d.z, e[4], e[5]);
        widen<T>(d.w, e[6], e[7]);
        const float y[8] = {o0.x, o0.y, o0.z, o0.w, o1.x, o1.y, o1.z, o1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(__uint_as_float(e[i]), y[i], s);
    }
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
    if (x < count && l == 0) {
        const float2 ml = __ldg(static_cast<const float2 *>(a.lse) + x);
        const float inv = 1.0f / ml.y;
        // a sum that is a NaN may come with m = -inf, which would say that there is none
        const float m = ml.y == 0.0f ? neg_inf<float>() : (ml.y != ml.y ? ml.y : ml.x * unit);
        a.stat[(b * a.heads + h) * a.n_rows + (row - b * a.n_rows)] = make_float4(m, inv, s * inv, 0.0f);
    }
}

// By A's rows: dq, and ds of every entry if asked for.
// With values two blocks an SM from 64 elements a warp on: three would spill (graph of
// 100 k rows, 8 heads of 64: 207 us against 224; of 32, 122 against 166; of 48, 220
// against 199).
template <typename T, int D, int KH, bool VALS, bool PACK>
__global__ void __launch_bounds__(kTileThreads, D * KH <= (VALS ? 48 : 64) && !(PACK && VALS) ? 3 : 2)
tile_bwd_rows_kernel(const __grid_constant__ AttnArgs a, unsigned total) {
    using R = Ring<D, KH, false>;
    extern __shared__ __align__(128) char smem[];
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, share = a.heads / a.kv_heads;
    const unsigned ring = (unsigned)__cvta_generic_to_shared(smem) + (threadIdx.x >> 5) * R::kBytes;
    const unsigned groups = PACK ? (unsigned)share >> (4 - a.rows_log) : (unsigned)share;    // of query heads on a key head
    const TileRows<PACK> rows(a.rows_log, g);
    const unsigned qst = (unsigned)a.qs[1] * 2, kst = (unsigned)a.ks[1] * 2, vst = (unsigned)a.vs[1] * 2,
                   dst = (unsigned)a.ds[1] * 2;
    const float scale = score_scale<VALS>(a.scale), none = neg_inf<float>();
    unsigned first, by;
    const unsigned count = my_share(total, first, by);
    if (count == 0) return;
    const Stride stride(by, (unsigned)a.n_items, groups, KH, a.kv_heads);
    Cursor now = stride.at(first);
    Feed<R> feed;
    const char *kb = nullptr, *vb = nullptr;
    int fb = 0;
    auto open = [&](const Cursor &f) {
        fb = f.b;
        kb = R::source(static_cast<const T *>(a.k) + f.b * a.ks[0] + f.kh * a.ks[2], a.ks[2] * 2, lane);
        vb = R::source(static_cast<const T *>(a.v) + f.b * a.vs[0] + f.kh * a.vs[2], a.vs[2] * 2, lane);
        const unsigned it = f.item(groups);
        const int row0 = (a.item_unit ? __ldg(a.item_unit + it) : (int)it) << a.rows_log;
        const int h = f.head(groups, share);
        prefetch_rows<T, D * KH>(static_cast<const T *>(a.q) + f.b * a.qs[0] + h * a.qs[2], a.qs[1], a.qs[2], a.rows_log,
                                 row0, a.n_rows, lane);
        prefetch_rows<T, D * KH>(static_cast<const T *>(a.dout) + f.b * a.ds[0] + h * a.ds[2], a.ds[1], a.ds[2], a.rows_log,
                                 row0, a.n_rows, lane);
    };
    auto copy = [&](unsigned st, unsigned col) { R::gather(st, kb, kst, vb, vst, col, lane); };
    feed.start(a, now, count, stride, groups, lane, a.n_cols, open);
    Ahead<VALS, R> meta;
    meta.first(a.chunks, feed.at, fb, rows);
    feed.advance(a, stride, groups, lane, a.n_cols, ring, open, copy);
    if constexpr (meta.kTwo) {
        meta.second(a.chunks, feed.at, fb, rows);
        feed.advance(a, stride, groups, lane, a.n_cols, ring, open, copy);
    }
    meta.start(a.vals_f, a.nnz, c);
    int st_read = 0;
    TileWork w_next = tile_work(a, now, groups, share, PACK ? a.rows_log : 4);
    for (unsigned piece = 0; piece < count; ++piece) {
        const TileWork w = w_next;
        if (piece + 1 < count) stride.move(now);
        w_next = tile_work(a, now, groups, share, PACK ? a.rows_log : 4);
        const int n = w.ch1 - w.ch0;
        Own<D> q[KH], go[KH];
        float m[KH][2], inv[KH][2], delta[KH][2];        // delta: D / l
        Sums<T, D> acc[KH];
#pragma unroll
        for (int j = 0; j < KH; ++j) {
            const int h = w.h + j;
            q[j].load(static_cast<const T *>(a.q) + w.b * a.qs[0] + h * a.qs[2], qst, a.qs[2], rows, w.row0, a.n_rows, c);
            go[j].load(static_cast<const T *>(a.dout) + w.b * a.ds[0] + h * a.ds[2], dst, a.ds[2], rows, w.row0, a.n_rows, c);
            acc[j].zero();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int64_t row = w.row0 + rows.r[i];
                float4 st = make_float4(none, 0.0f, 0.0f, 0.0f);
                if (row < a.n_rows) st = __ldg(a.stat + ((int64_t)w.b * a.heads + h + rows.h[i]) * a.n_rows + row);
                m[j][i] = st.x;
                inv[j][i] = st.y;
                delta[j][i] = st.z;
            }
        }
        float *ds_out = VALS && a.ds_out ? a.ds_out + ((int64_t)w.b * a.heads + w.h) * a.nnz : nullptr;
        for (int ch = 0; ch < n; ++ch) {
            meta.take(a.vals_f, a.nnz, c);
            cp_wait<R::kStages - 2>();
            __syncwarp();
            meta.passed(a.chunks, feed.at, fb, rows);
            feed.advance(a, stride, groups, lane, a.n_cols, ring, open, copy);
            const unsigned stage = ring + st_read;
            st_read = st_read == (R::kStages - 1) * R::kStage ? 0 : st_read + R::kStage;
            const auto &x = meta.x;
            const Chunk<VALS> &cur = meta.now;
            const unsigned there[2] = {cur.bits[0] >> (2 * c), cur.bits[1] >> (2 * c)};
            unsigned mine[2] = {there[0], there[1]}, used = 0;
            bool drop = false;
            if constexpr (VALS) {
                bool out = false;
#pragma unroll
                for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (x[blk][e] == none) {
                            mine[e >> 1] &= ~pair_bit(blk, e);
                            out = true;
                        }
                drop = __any_sync(kAll, out);
                if (drop) {
                    used = (mine[0] | mine[1]) & 0x303u;
                    used = (used | used >> 6) & 15u;
                }
            }
#pragma unroll
            for (int j = 0; j < KH; ++j) {
                const unsigned at = stage + (KH == 1 ? 0 : j * (D * 2));
                float s[2][4], dp[2][4];
                score_products<T, D, R::kPitch>(s, q[j], at, g, c);
                score_products<T, D, R::kPitch>(dp, go[j], at + R::kTensor, g, c);
                if (j == 0) meta.late(a.vals_f, a.nnz, c);
                const unsigned on[2] = {m[j][0] == none ? 0u : mine[0], m[j][1] == none ? 0u : mine[1]};    // rows with weights
#pragma unroll
                for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = e >> 1;
                        s[blk][e] = weight<VALS>(relative<VALS>(s[blk][e], scale, x[blk][e], m[j][i])) *
                                    fmaf(dp[blk][e], inv[j][i], -delta[j][i]);
                        s[blk][e] = on[i] & pair_bit(blk, e) ? s[blk][e] : 0.0f;
                    }
                if (VALS && ds_out) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int blk = 0; blk < 2; ++blk) {
                            float *p = ds_out + (j + rows.h[i]) * a.nnz + cur.entry(i, blk, c);
                            if (there[i] & pair_bit(blk, 0)) p[0] = s[blk][2 * i];
                            if (there[i] & pair_bit(blk, 1)) p[there[i] >> (8 * blk) & 1] = s[blk][2 * i + 1];
                        }
                }
                acc[j].template add_chunk<R::kPitch>(s, at, g, c, VALS && drop, used);
            }
        }
        if (!a.dq) continue;
        bool bad = false;
#pragma unroll
        for (int j = 0; j < KH; ++j) bad = acc[j].bad() || bad;
        if (bad) {
            const int heads = KH == 1 ? kTileRows >> a.rows_log : KH;
            for (int j = 0; j < heads; ++j) {
                TileWork one = w;
                one.h = w.h + j;
                one.kh = KH == 1 ? w.kh : w.kh + j;
                slow_bwd_rows<T>(a, one);
            }
            continue;
        }
#pragma unroll
        for (int j = 0; j < KH; ++j) {
            acc[j].scale((float)a.scale, (float)a.scale);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = rows.r[i], h = w.h + rows.h[i] + j;
                if (w.row0 + r >= a.n_rows) continue;
                if (w.slot < 0)
                    acc[j].store(static_cast<T *>(a.dq) + (((int64_t)w.b * a.n_rows + w.row0 + r) * a.heads + h) * D, i, c);
                else
                    acc[j].store(static_cast<float *>(a.part) +
                                     part_index(w.slot, a.n_slots, w.b, 1 << a.rows_log, r, a.heads, h) * D, i, c);
            }
        }
    }
}

// dk and dv of the tile's rows of A^T, entry by entry.
template <typename T>
__device__ __noinline__ void slow_bwd_cols(const AttnArgs &a, const TileWork &w, bool want_dk, bool want_dv) {
    const int lane = threadIdx.x & 31, share = a.heads / a.kv_heads;
    int s0, s1;
    row_range(a.chunks, w, lane, 4 - a.rows_log, s0, s1);
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
                const float4 st = a.stat[((int64_t)w.b * a.heads + h) * a.n_rows + i];
                if (x == none || st.x == none) continue;
                float q[kSlowVec], go[kSlowVec];
                slow_load(q, static_cast<const T *>(a.q) + w.b * a.qs[0] + i * a.qs[1] + h * a.qs[2], a.dim, lane);
                slow_load(go, static_cast<const T *>(a.dout) + w.b * a.ds[0] + i * a.ds[1] + h * a.ds[2], a.dim, lane);
                const float e2 = exp2f(a.vals ? (fmaf(slow_dot(q, k), scale, x) - st.x) * kLog2e
                                             : fmaf(slow_dot(q, k), scale * kLog2e, -st.x));
                const float p = e2 * st.y, ds = e2 * fmaf(slow_dot(go, v), st.y, -st.z);
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

// By A^T's rows: dk (DK) and dv (DV) of 16 columns of A for KH key heads, the
// query heads that share one following each other.  Wide heads take two launches:
// both sums and both own operands would not fit the registers, and 3 blocks an SM
// would spill (246 us with 2, 396 with 3 on the graph above).  The values come in
// A^T's order (tile_values_kernel).
template <typename T, int D, int KH, bool DK, bool DV, bool VALS, bool PACK>
__global__ void __launch_bounds__(kTileThreads, 2)
tile_bwd_cols_kernel(const __grid_constant__ AttnArgs a, unsigned total) {
    using R = Ring<D, KH, true>;
    extern __shared__ __align__(128) char smem[];
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, share = a.heads / a.kv_heads;
    const TileRows<false> rows(4, g);
    // PACK: a chunk holds every column (a query row) once for each of 2^times heads
    const int times = PACK ? 4 - a.rows_log : 0, groups = share >> times;
    const unsigned ring = (unsigned)__cvta_generic_to_shared(smem) + (threadIdx.x >> 5) * R::kBytes;
    const unsigned qst = (unsigned)a.qs[1] * 2, kst = (unsigned)a.ks[1] * 2, vst = (unsigned)a.vs[1] * 2,
                   dst = (unsigned)a.ds[1] * 2;
    const float scale = score_scale<VALS>(a.scale), none = neg_inf<float>();
    unsigned first, by;
    const unsigned count = my_share(total, first, by);
    if (count == 0) return;
    // A piece is a tile; the shared heads (or groups of them) follow each other and its
    // sums are written after the last one.
    const Stride stride(by, (unsigned)a.n_items, 1, KH, a.kv_heads);
    Cursor now = stride.at(first);
    Feed<R> feed = {};
    const char *qb = nullptr, *gb = nullptr;
    const float4 *stat = nullptr;
    int begin = 0, fh = 0;                               // first chunk of the feed's tile, its shared head
    auto open_head = [&](int b, int h) {
        qb = R::source(static_cast<const T *>(a.q) + b * a.qs[0] + h * a.qs[2], a.qs[2] * 2, lane);
        gb = R::source(static_cast<const T *>(a.dout) + b * a.ds[0] + h * a.ds[2], a.ds[2] * 2, lane);
        stat = a.stat + ((int64_t)b * a.heads + h) * a.n_rows;
    };
    int fb = 0, fkh = 0;
    auto open = [&](const Cursor &f) {
        begin = feed.at;
        fh = 0;
        fb = f.b;
        fkh = f.kh;
        open_head(f.b, f.kh * share);
        const int row0 = (a.item_unit ? __ldg(a.item_unit + f.x) : (int)f.x) * kTileRows;
        prefetch_rows<T, D * KH>(static_cast<const T *>(a.k) + f.b * a.ks[0] + f.kh * a.ks[2], a.ks[1], 0, 4, row0, a.n_cols, lane);
        if (DK)
            prefetch_rows<T, D * KH>(static_cast<const T *>(a.v) + f.b * a.vs[0] + f.kh * a.vs[2], a.vs[1], 0, 4, row0, a.n_cols, lane);
    };
    auto copy = [&](unsigned st, unsigned col) {
        if constexpr (PACK) R::gather(st, qb, qst, gb, dst, col, lane, times, a.qs[2] * 2, a.ds[2] * 2);
        else R::gather(st, qb, qst, gb, dst, col, lane);
#pragma unroll
        for (int j = 0; j < KH; j += 2) {               // lanes 16 to 31: the next head
            const int jj = KH == 1 ? 0 : j + (lane >> 4);
            if (KH > 1 || lane < 16)
                cp_async16(st + 2 * R::kTensor + (jj * 16 + (lane & 15)) * 16,
                           stat + (int64_t)(PACK ? lane & ((1 << times) - 1) : jj) * a.n_rows + col);
        }
        if (KH == 1 && feed.at + 1 == feed.end && fh + 1 < groups) {    // the tile again, with its next heads
            ++fh;
            open_head(fb, fkh * share + (fh << times));
            feed.at = begin - 1;
        }
    };
    feed.start(a, now, count, stride, 1, lane, a.n_rows, open);
    Ahead<VALS, R> meta;
    meta.first(a.chunks, feed.at, fb, rows);
    feed.advance(a, stride, 1, lane, a.n_rows, ring, open, copy);
    if constexpr (meta.kTwo) {
        meta.second(a.chunks, feed.at, fb, rows);
        feed.advance(a, stride, 1, lane, a.n_rows, ring, open, copy);
    }
    meta.start(a.vals_t, a.nnz, c, times);
    int st_read = 0;
    TileWork w_next = tile_work(a, now, 1, share, 4);
    for (unsigned piece = 0; piece < count; ++piece) {
        const TileWork w = w_next;
        if (piece + 1 < count) stride.move(now);
        w_next = tile_work(a, now, 1, share, 4);
        Own<D> k[KH], v[DK ? KH : 1];
        Sums<T, D> dk[DK ? KH : 1], dv[DV ? KH : 1];
#pragma unroll
        for (int j = 0; j < KH; ++j) {
            k[j].load(static_cast<const T *>(a.k) + w.b * a.ks[0] + (w.kh + j) * a.ks[2], kst, 0, rows, w.row0, a.n_cols, c);
            if constexpr (DK) {
                v[j].load(static_cast<const T *>(a.v) + w.b * a.vs[0] + (w.kh + j) * a.vs[2], vst, 0, rows, w.row0, a.n_cols, c);
                dk[j].zero();
            }
            if constexpr (DV) dv[j].zero();
        }
        const int n = w.ch1 - w.ch0, steps = n * (KH == 1 ? groups : 1);
        for (int x = 0; x < steps; ++x) {
            meta.take(a.vals_t, a.nnz, c, times);
            cp_wait<R::kStages - 2>();
            __syncwarp();
            meta.passed(a.chunks, feed.at, fb, rows);
            feed.advance(a, stride, 1, lane, a.n_rows, ring, open, copy);
            const unsigned stage = ring + st_read;
            st_read = st_read == (R::kStages - 1) * R::kStage ? 0 : st_read + R::kStage;
            unsigned mine[2] = {meta.now.bits[0] >> (2 * c), meta.now.bits[1] >> (2 * c)}, used = 0;
            const auto &val = meta.x;
#pragma unroll
            for (int j = 0; j < KH; ++j) {
                const unsigned at = stage + j * (D * 2);
                float s[2][4], dp[2][4];
                score_products<T, D, R::kPitch>(s, k[j], at, g, c);
                if constexpr (DK) score_products<T, D, R::kPitch>(dp, v[j], at + R::kTensor, g, c);
                if (j == 0) meta.late(a.vals_t, a.nnz, c, times);
                const unsigned sp = stage + 2 * R::kTensor + j * 256 + c * 32;
                unsigned live[2] = {mine[0], mine[1]};
                bool out = false;                       // a stored pair without a part: its row or value is left out
#pragma unroll
                for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                    for (int col = 0; col < 2; ++col) {
                        const uint4 st = lds16(sp + blk * 128 + col * 16);      // the statistics of column 2c + col
                        const float m = __uint_as_float(st.x), inv = __uint_as_float(st.y), delta = __uint_as_float(st.z);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int e = 2 * i + col;
                            if (m == none || (VALS && val[blk][e] == none)) {
                                out = out || (live[i] & pair_bit(blk, e));
                                live[i] &= ~pair_bit(blk, e);
                            }
                            const bool on = live[i] & pair_bit(blk, e);
                            const float p = weight<VALS>(relative<VALS>(s[blk][e], scale, val[blk][e], m));
                            if constexpr (DV) s[blk][e] = on ? p * inv : 0.0f;
                            if constexpr (DK) dp[blk][e] = on ? p * fmaf(dp[blk][e], inv, -delta) : 0.0f;
                        }
                    }
                const bool drop = VALS && __any_sync(kAll, out);
                used = (live[0] | live[1]) & 0x303u;
                used = (used | used >> 6) & 15u;
                if constexpr (DV) dv[j].template add_chunk<R::kPitch>(s, at + R::kTensor, g, c, drop, used);
                if constexpr (DK) dk[j].template add_chunk<R::kPitch>(dp, at, g, c, drop, used);
            }
        }
        bool bad = false;
#pragma unroll
        for (int j = 0; j < KH; ++j) {
            if constexpr (DK) bad = dk[j].bad() || bad;
            if constexpr (DV) bad = dv[j].bad() || bad;
        }
        if (bad) {
            for (int j = 0; j < KH; ++j) {
                TileWork one = w;
                one.kh = w.kh + j;
                slow_bwd_cols<T>(a, one, DK, DV);
            }
            continue;
        }
#pragma unroll
        for (int j = 0; j < KH; ++j) {
            if constexpr (DK) dk[j].scale((float)a.scale, (float)a.scale);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = g + 8 * i;
                if (w.row0 + r >= a.n_cols) continue;
                if (w.slot < 0) {
                    const int64_t o = (((int64_t)w.b * a.n_cols + w.row0 + r) * a.kv_heads + w.kh + j) * D;
                    if constexpr (DK)
                        if (a.dk) dk[j].store(static_cast<T *>(a.dk) + o, i, c);
                    if constexpr (DV)
                        if (a.dv) dv[j].store(static_cast<T *>(a.dv) + o, i, c);
                } else {
                    float *p = static_cast<float *>(a.part) +
                               part_index(w.slot, a.n_slots, w.b, kTileRows, r, a.kv_heads, w.kh + j) * 2 * D;
                    if constexpr (DK) dk[j].store(p, i, c);
                    if constexpr (DV) dv[j].store(p + D, i, c);
                }
            }
        }
    }
}

// The values as 32-bit numbers, in A^T's order with perm.
__global__ void __launch_bounds__(256)
tile_values_kernel(int64_t nnz, int batch, const int32_t *__restrict__ perm, const void *vals, int f64,
                   float *__restrict__ out) {
    const int64_t t = blockIdx.x * (int64_t)256 + threadIdx.x;
    if (t >= nnz) return;
    const int64_t e = perm ? SLA_IDX((int64_t)__ldg(perm + t), nnz, kBndEntry) : t;
    for (int b = 0; b < batch; ++b) out[b * nnz + t] = load_value<float>(vals, f64, b * nnz + e);
}

sla_status tile_values(const AttnArgs &a, const int32_t *perm, float *out, cudaStream_t s) {
    if (a.nnz == 0) return SLA_OK;
    tile_values_kernel<<<blocks_of(a.nnz), 256, 0, s>>>(a.nnz, a.batch, perm, a.vals, a.vals_f64, out);
    SLA_CHECK_LAUNCH();
    return SLA_OK;
}

// -------------------------------------------------------------- launches ----
enum { kTileFwd, kTileBwdRows, kTileBwdCols };

// As many blocks as run at once, each warp going through the work in strides.  How
// many that is, is asked once a kernel and device.
template <auto KERNEL>
sla_status launch_stream(const AttnArgs &a, int64_t total, int ring, cudaStream_t s) {
    constexpr int kDevices = 64;
    static std::atomic<int> resident[kDevices];
    const int bytes = ring * kTileWarps;
    int dev = 0;
    SLA_CHECK_CUDA(cudaGetDevice(&dev));
    if (bytes > 48 * 1024)
        SLA_CHECK_CUDA(cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    int most = dev < kDevices ? resident[dev].load(std::memory_order_acquire) : 0;
    if (most == 0) {
        int per_sm = 0, sms = 0;
        SLA_CHECK_CUDA(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, KERNEL, kTileThreads, bytes));
        SLA_CHECK_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
        most = (per_sm > 0 ? per_sm : 1) * sms;
        if (dev < kDevices) resident[dev].store(most, std::memory_order_release);
    }
    const int64_t blocks = (total + kTileWarps - 1) / kTileWarps;
    KERNEL<<<(unsigned)(blocks < most ? blocks : most), kTileThreads, bytes, s>>>(a, (unsigned)total);
    SLA_CHECK_LAUNCH();
    return SLA_OK;
}

// KH key heads a warp.
template <typename T, int D, int KH, bool VALS>
sla_status launch_tile(int what, const AttnArgs &a, cudaStream_t s) {
    const bool cols = what == kTileBwdCols;
    const int64_t total = (int64_t)a.n_items * (cols ? 1 : (a.heads / a.kv_heads) >> (4 - a.rows_log)) * a.batch *
                          (a.kv_heads / KH);
    SLA_REQUIRE(total < INT_MAX, "sla_attention: too many rows, systems and heads");
    if (total == 0) return SLA_OK;
    constexpr int row_bytes = Ring<D, KH, false>::kBytes;
    if constexpr (KH == 1) {
        if (what == kTileFwd && a.rows_log < 4) return launch_stream<tile_forward_kernel<T, D, 1, VALS, true>>(a, total, row_bytes, s);
        if (what == kTileBwdRows && a.rows_log < 4) return launch_stream<tile_bwd_rows_kernel<T, D, 1, VALS, true>>(a, total, row_bytes, s);
    }
    if (what == kTileFwd) return launch_stream<tile_forward_kernel<T, D, KH, VALS, false>>(a, total, row_bytes, s);
    if (what == kTileBwdRows) return launch_stream<tile_bwd_rows_kernel<T, D, KH, VALS, false>>(a, total, row_bytes, s);
    constexpr int bytes = Ring<D, KH, true>::kBytes;
    auto cols_of = [&](auto pack) -> sla_status {
        constexpr bool PACK = decltype(pack)::value;
        if constexpr (D * KH <= 64) {
            return launch_stream<tile_bwd_cols_kernel<T, D, KH, true, true, VALS, PACK>>(a, total, bytes, s);
        } else {
            sla_status st = a.dv ? launch_stream<tile_bwd_cols_kernel<T, D, KH, false, true, VALS, PACK>>(a, total, bytes, s) : SLA_OK;
            if (st == SLA_OK && a.dk) st = launch_stream<tile_bwd_cols_kernel<T, D, KH, true, false, VALS, PACK>>(a, total, bytes, s);
            return st;
        }
    };
    if constexpr (KH == 1)
        if (a.rows_log < 4) return cols_of(std::true_type{});
    return cols_of(std::false_type{});
}

template <typename T>
sla_status launch_delta(const AttnArgs &a, cudaStream_t s) {
    const int64_t count = (int64_t)a.batch * a.n_rows * a.heads;
    if (count == 0) return SLA_OK;
    const float unit = a.vals ? 1.0f : kLog2e;
    auto go = [&](auto *kernel, int lanes) -> sla_status {
        kernel<<<blocks_of(count * lanes), 256, 0, s>>>(a, count, unit);
        SLA_CHECK_LAUNCH();
        return SLA_OK;
    };
    if (a.dim <= 16) return go(tile_delta_kernel<T, 2>, 2);
    if (a.dim <= 32) return go(tile_delta_kernel<T, 4>, 4);
    if (a.dim <= 64) return go(tile_delta_kernel<T, 8>, 8);
    return go(tile_delta_kernel<T, 16>, 16);
}

// Key heads a warp: as many as fill 128 bytes of a gathered row, if every query
// head has its own and their number allows (1024 x 1024 grid, heads of 32: 524 us
// with two, 655 with one).
template <typename T, int D, bool VALS>
sla_status launch_tile_heads(int what, const AttnArgs &a, cudaStream_t s) {
    if constexpr (D <= 32) {
        constexpr int K = 64 / D;
        if (a.heads == a.kv_heads && a.kv_heads % K == 0) return launch_tile<T, D, K, VALS>(what, a, s);
    }
    return launch_tile<T, D, 1, VALS>(what, a, s);
}

template <typename T, int D>
sla_status launch_tile(int what, const AttnArgs &a, cudaStream_t s) {
    return a.vals ? launch_tile_heads<T, D, true>(what, a, s) : launch_tile_heads<T, D, false>(what, a, s);
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

sla_status build_tiles(AttnTiles *t, const AttnPlan &parts, int rows, int times, int n_rows, const int32_t *rowptr, const int32_t *colind,
                       cudaStream_t s) {
    const int n = parts.n_items, U = parts.n_units;
    DeviceScratch tmp(s);
    unsigned *count = tmp.get<unsigned>((size_t)n + 1), *chunks = tmp.get<unsigned>((size_t)U + 1);
    void *ws = tmp.get<char>(scan_ws_bytes((int64_t)n + 1));
    if (!count || !chunks || !ws || !alloc_array(&t->chunk0, (size_t)U + 1)) {
        set_error("attention plan: out of device memory");
        return SLA_ERR_OOM;
    }
    const unsigned grid = blocks_of(((int64_t)n + 1) * 32, 128);
    tile_columns_kernel<false><<<grid, 128, 0, s>>>(rows, times, n_rows, rowptr, colind, n, parts.seg_len, parts.item_unit,
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
    SLA_CHECK_CUDA(cudaMemsetAsync(t->chunks, 0, (size_t)(total > 0 ? total : 1) * sizeof(TileChunk), s));
    tile_columns_kernel<true><<<grid, 128, 0, s>>>(rows, times, n_rows, rowptr, colind, n, parts.seg_len, parts.item_unit,
                                                   parts.item_seg, nullptr, count, t->chunk0, t->chunks);
    SLA_CHECK_LAUNCH();
    SLA_CHECK_CUDA(cudaStreamSynchronize(s));
    t->built = true;
    return SLA_OK;
}

// 32-bit values are read in place; 64-bit ones are rounded to a.vals_w first
// (the backward's row kernel comes before its column kernel, which reuses it).
template <typename T> sla_status attn_tile_forward(AttnArgs a, cudaStream_t s) {
    a.vals_f = static_cast<const float *>(a.vals);
    if (a.vals && a.vals_f64) {
        const sla_status st = tile_values(a, nullptr, a.vals_w, s);
        if (st != SLA_OK) return st;
        a.vals_f = a.vals_w;
    }
    return launch_tile_of<T>(kTileFwd, a, s);
}
template <typename T> sla_status attn_tile_bwd_rows(AttnArgs a, cudaStream_t s) {
    a.vals_f = static_cast<const float *>(a.vals);
    if (a.vals && a.vals_f64) {
        const sla_status st = tile_values(a, nullptr, a.vals_w, s);
        if (st != SLA_OK) return st;
        a.vals_f = a.vals_w;
    }
    const sla_status st = launch_delta<T>(a, s);
    if (st != SLA_OK || (!a.dq && !a.ds_out)) return st;
    return launch_tile_of<T>(kTileBwdRows, a, s);
}
template <typename T> sla_status attn_tile_bwd_cols(AttnArgs a, cudaStream_t s) {
    if (a.vals) {
        const sla_status st = tile_values(a, a.perm, a.vals_w, s);
        if (st != SLA_OK) return st;
        a.vals_t = a.vals_w;
    }
    return launch_tile_of<T>(kTileBwdCols, a, s);
}
template sla_status attn_tile_forward<__nv_bfloat16>(AttnArgs, cudaStream_t);
template sla_status attn_tile_forward<__half>(AttnArgs, cudaStream_t);
template sla_status attn_tile_bwd_rows<__nv_bfloat16>(AttnArgs, cudaStream_t);
template sla_status attn_tile_bwd_rows<__half>(AttnArgs, cudaStream_t);
template sla_status attn_tile_bwd_cols<__nv_bfloat16>(AttnArgs, cudaStream_t);
template sla_status attn_tile_bwd_cols<__half>(AttnArgs, cudaStream_t);

}  // namespace sla
