// Attention over a CSR pattern: row i of the pattern is a query that attends to
// the columns stored in that row, with the stored values (one per entry) added
// to the scores.  The autograd companion of the matrix product on the same
// handle: the forward gathers k and v by A's columns, the backward gathers by
// A's rows and, for the keys' gradients, by A^T's (no atomics: every sum has a
// fixed order).  Formulas: sla_attention.cuh.
#include "sla_attention.cuh"

#include <algorithm>
#include <climits>
#include <cmath>
#include <initializer_list>
#include <new>
#include <utility>

namespace sla {

// ----------------------------------------------------------------- plan ----
namespace {

__global__ void unit_len_kernel(int n_rows, int rows, int n_units, const int32_t *__restrict__ rowptr,
                                unsigned *len) {
    const int u = blockIdx.x * blockDim.x + threadIdx.x;
    if (u > n_units) return;
    int m = 0;
    if (u < n_units)
        for (int64_t i = (int64_t)u * rows; i < min((int64_t)n_rows, ((int64_t)u + 1) * rows); ++i)
            m = max(m, rowptr[i + 1] - rowptr[i]);
    len[u] = (unsigned)m;
}

// Segments, slots (segments of split units) and split units of every unit; units up
// to `whole` are not split.
__global__ void unit_split_kernel(int n_units, int seg_len, int whole, const unsigned *__restrict__ len, unsigned *nseg,
                                  unsigned *slots, unsigned *multi, unsigned *most) {
    const int u = blockIdx.x * blockDim.x + threadIdx.x;
    if (u > n_units) return;
    unsigned n = 0;
    if (u < n_units) n = len[u] <= (unsigned)whole ? 1u : (len[u] + seg_len - 1) / seg_len;
    nseg[u] = n;
    slots[u] = n > 1 ? n : 0;
    multi[u] = n > 1 ? 1 : 0;
    if (n > 1) atomicMax(most, n);
}

__global__ void unit_fill_kernel(int n_units, const unsigned *__restrict__ item0, const unsigned *__restrict__ slot0,
                                 const unsigned *__restrict__ multi0, int32_t *item_unit, int32_t *item_seg,
                                 int32_t *item_slot, int32_t *multi_unit, int32_t *multi_slot, int seg_len,
                                 const int32_t *__restrict__ chunk0, int2 *item_chunks) {
    const int u = blockIdx.x * blockDim.x + threadIdx.x;
    if (u > n_units) return;
    if (u == n_units) {
        multi_slot[multi0[u]] = (int32_t)slot0[u];
        return;
    }
    const unsigned i0 = item0[u], n = item0[u + 1] - i0;
    for (unsigned k = 0; k < n; ++k) {
        item_unit[i0 + k] = u;
        item_seg[i0 + k] = (int32_t)k;
        item_slot[i0 + k] = n > 1 ? (int32_t)(slot0[u] + k) : -1;
        if (item_chunks) {
            const long long from = chunk0[u] + (long long)k * seg_len, to = from + seg_len;
            item_chunks[i0 + k] = make_int2((int)from, (int)min(to, (long long)chunk0[u + 1]));
        }
    }
    if (n > 1) {
        multi_unit[multi0[u]] = u;
        multi_slot[multi0[u]] = (int32_t)slot0[u];
    }
}

void free_plan(AttnPlan *p) {
    cudaFree(p->item_unit);
    cudaFree(p->item_seg);
    cudaFree(p->item_slot);
    cudaFree(p->item_chunks);
    cudaFree(p->multi_unit);
    cudaFree(p->multi_slot);
    *p = AttnPlan();
}

// Lengths of tiles in chunks.
__global__ void tile_len_kernel(int n_units, const int32_t *__restrict__ chunk0, unsigned *len) {
    const int u = blockIdx.x * blockDim.x + threadIdx.x;
    if (u <= n_units) len[u] = u < n_units ? (unsigned)(chunk0[u + 1] - chunk0[u]) : 0u;
}

// Items of units with the lengths len (device, [n_units + 1]).  seg_len > 0: a
// given segment length; else one that makes about `fill` items when the units
// are few, at least `least`, and at least the root of a 16th of the longest unit:
// a segment is walked alone, then the unit's segments are joined by one block, 16
// warps taking 4 at a time.  (One row of 65536 entries, a head of 64 elements: 31 us,
// 41 with the root of a 64th, 33 of an 8th; 67 without, and for tiles 47 -> 21.)
// Units up to `whole`, or `share` items' share of the work, are not split.
sla_status build_items(AttnPlan *p, unsigned *len, int seg_len, int64_t fill, int least, int whole, int share,
                       const int32_t *chunk0, cudaStream_t s) {
    const int U = p->n_units;
    DeviceScratch tmp(s);
    unsigned *nseg = tmp.get<unsigned>((size_t)U + 1), *slots = tmp.get<unsigned>((size_t)U + 1),
             *multi = tmp.get<unsigned>((size_t)U + 1);
    void *ws = tmp.get<char>(scan_ws_bytes((int64_t)U + 1));
    unsigned *most = tmp.get<unsigned>(1);
    if (!nseg || !slots || !multi || !ws || !most) {
        set_error("attention plan: out of device memory");
        return SLA_ERR_OOM;
    }
    sla_status st;
    const bool chosen = seg_len <= 0;
    if (chosen) {
        unsigned total = 0;
        st = exclusive_scan(len, nseg, (int64_t)U + 1, ws, s);
        if (st != SLA_OK) return st;
        SLA_CHECK_CUDA(cudaMemcpyAsync(&total, nseg + U, sizeof total, cudaMemcpyDeviceToHost, s));
        SLA_CHECK_CUDA(cudaStreamSynchronize(s));
        const int64_t mean = ((int64_t)total + fill - 1) / fill;
        seg_len = (int)std::max<int64_t>(least, mean);
        whole = (int)std::min<int64_t>(INT_MAX, std::max<int64_t>(whole, mean * share));
    }
    unsigned *vec[3] = {nseg, slots, multi};
    unsigned tot[4] = {0, 0, 0, 1};
    for (int pass = 0;; ++pass) {
        SLA_CHECK_CUDA(cudaMemsetAsync(most, 0, sizeof(unsigned), s));
        unit_split_kernel<<<blocks_of((int64_t)U + 1), 256, 0, s>>>(U, seg_len, whole, len, nseg, slots, multi, most);
        SLA_CHECK_LAUNCH();
        SLA_CHECK_CUDA(cudaMemcpyAsync(&tot[3], most, sizeof(unsigned), cudaMemcpyDeviceToHost, s));
        SLA_CHECK_CUDA(cudaStreamSynchronize(s));
        const int root = (int)std::sqrt((double)tot[3] * seg_len / 16.0);
        if (!chosen || pass > 0 || root <= seg_len) break;
        seg_len = root;
    }
    p->seg_len = seg_len;
    for (int i = 0; i < 3; ++i) {
        st = exclusive_scan(vec[i], vec[i], (int64_t)U + 1, ws, s);
        if (st != SLA_OK) return st;
        SLA_CHECK_CUDA(cudaMemcpyAsync(&tot[i], vec[i] + U, sizeof(unsigned), cudaMemcpyDeviceToHost, s));
    }
    SLA_CHECK_CUDA(cudaStreamSynchronize(s));
    p->n_items = (int32_t)tot[0];
    p->n_slots = (int32_t)tot[1];
    p->n_multi = (int32_t)tot[2];
    p->most_segs = (int32_t)tot[3];
    if (p->n_multi > 0) {
        if (!alloc_array(&p->item_unit, tot[0]) || !alloc_array(&p->item_seg, tot[0]) ||
            !alloc_array(&p->item_slot, tot[0]) || !alloc_array(&p->multi_unit, tot[2]) ||
            !alloc_array(&p->multi_slot, (size_t)tot[2] + 1) || (chunk0 && !alloc_array(&p->item_chunks, tot[0]))) {
            set_error("attention plan: out of device memory");
            return SLA_ERR_OOM;
        }
        unit_fill_kernel<<<blocks_of((int64_t)U + 1), 256, 0, s>>>(U, nseg, slots, multi, p->item_unit, p->item_seg,
                                                                   p->item_slot, p->multi_unit, p->multi_slot, seg_len,
                                                                   chunk0, p->item_chunks);
        SLA_CHECK_LAUNCH();
        SLA_CHECK_CUDA(cudaStreamSynchronize(s));
    }
    return SLA_OK;
}

// Enough items to fill the GPU when there are few units: 8 tiles an SM, a warp each,
// or 128 rows, a few lanes each.  A level counts on 8 times as many systems and heads
// as the one before, so it splits 8 times less.  Rows up to kWhole entries, or 4 items'
// share of the work, are not split, nor tiles up to kWhole columns: a short part
// spends more on its partial result than on its entries.  Measured, forward pass:
//   tiles, 24 an SM against 8: 300 rows over 1500 columns, 64 systems and heads,
//   112 -> 116 us and a join of 22; 513 rows of 256 entries, 2 key heads of 128
//   elements, 23 -> 28 us;
//   rows, float32, 8, 64 and 128 an SM: 30000 rows of 20 entries and one of 20000, 8
//   heads of 32, 1150, 205 and 137 us; 64 full rows over 4096 columns, 292, 60 and 45 us;
//   rows whole up to 5 shares against 4: 513 rows of 256 entries, 8 heads of 32, 66
//   against 46 us (training 256, 184); 4000 rows of 100, a head of 64, 22 against 29
//   (training 128, 134).
int64_t fill_of(const Csr *h, int level, bool tiled) {
    return std::max<int64_t>(1, (int64_t)h->num_sms * (tiled ? 8 : 128) >> (3 * level));
}
constexpr int kWhole = 64;

constexpr int kRowKind = -1;             // plans of rows, not tiles

AttnPlan &plan_at(Csr *h, int kind, bool transposed, int level) {
    return kind == kRowKind ? h->attn->row[transposed][level] : h->attn->tile[transposed][kind][level];
}

sla_status ensure_plan(Csr *h, int kind, bool transposed, int level, cudaStream_t s);

// One level of one direction's row plans, or of a kind of tiles (and the tiles).
sla_status build_plans(Csr *h, int kind, bool transposed, int level, cudaStream_t s) {
    const bool tiled = kind != kRowKind;
    AttnPlan *p = &plan_at(h, kind, transposed, level);
    AttnTiles *tiles = tiled ? &h->attn->tiles[transposed][kind] : nullptr;
    const int n = transposed ? h->n_cols : h->n_rows;
    const int32_t *rowptr = transposed ? h->rowptrT : h->rowptr, *colind = transposed ? h->colindT : h->colind;
    p->rows = tiled ? kTileRows >> (transposed ? 0 : kind) : 1;
    p->n_units = (n + p->rows - 1) / p->rows;
    const int U = p->n_units;
    // no row that any level would split (the lengths of A's rows are known)
    if (U == 0 || (!tiled && !transposed && h->row_max <= kWhole)) {
        p->n_items = U;
        p->built = true;
        return SLA_OK;
    }
    if (level > 0) {                     // a level splits what the one before it splits, or less
        const sla_status st = ensure_plan(h, kind, transposed, 0, s);
        if (st != SLA_OK) return st;
        const AttnPlan &finest = plan_at(h, kind, transposed, 0);
        if (finest.n_multi == 0) {
            *p = finest;                 // no arrays
            return SLA_OK;
        }
    }
    DeviceScratch tmp(s);
    unsigned *len = tmp.get<unsigned>((size_t)U + 1);
    if (!len) {
        set_error("attention plan: out of device memory");
        return SLA_ERR_OOM;
    }
    const unsigned grid = blocks_of((int64_t)U + 1);
    if (!tiled || !tiles->built) {
        unit_len_kernel<<<grid, 256, 0, s>>>(n, p->rows, U, rowptr, len);
        SLA_CHECK_LAUNCH();
    }
    sla_status st;
    if (tiled) {
        if (!tiles->built) {
            // columns are gathered by parts of 256 entries of a tile's longest row
            AttnPlan parts;
            parts.n_units = U;
            st = build_items(&parts, len, 256, 0, 0, 0, 0, nullptr, s);
            if (st == SLA_OK) st = build_tiles(tiles, parts, p->rows, transposed ? 1 << kind : 1, n, rowptr, colind, s);
            free_plan(&parts);
            if (st != SLA_OK) return st;
        }
        tile_len_kernel<<<grid, 256, 0, s>>>(U, tiles->chunk0, len);
        SLA_CHECK_LAUNCH();
    }
    if (tiled) st = build_items(p, len, 0, fill_of(h, level, true), kWhole / 16, kWhole / 16, 1, tiles->chunk0, s);
    else st = build_items(p, len, 0, fill_of(h, level, false), kWhole / 4, kWhole, 4, nullptr, s);
    if (st == SLA_OK) p->built = true;
    return st;
}

void free_tiles(AttnTiles *t) {
    cudaFree(t->chunk0);
    cudaFree(t->chunks);
    *t = AttnTiles();
}

sla_status ensure_plan(Csr *h, int kind, bool transposed, int level, cudaStream_t s) {
    AttnPlan *p = &plan_at(h, kind, transposed, level);
    if (p->built) return SLA_OK;
    sla_status st = SLA_ERR_OOM;
    try {
        st = build_plans(h, kind, transposed, level, s);
    } catch (const std::bad_alloc &) {
        set_error("sla_attention_prepare: out of host memory");
    }
    if (st != SLA_OK) {
        cudaStreamSynchronize(s);
        free_plan(p);
        if (kind != kRowKind && !h->attn->tiles[transposed][kind].built) free_tiles(&h->attn->tiles[transposed][kind]);
    }
    return st;
}

}  // namespace

void use_plan(AttnArgs &a, const AttnPlan &p) {
    a.n_items = p.n_items;
    a.n_slots = p.n_slots;
    a.seg_len = p.seg_len;
    a.item_unit = p.item_unit;
    a.item_seg = p.item_seg;
    a.item_slot = p.item_slot;
    a.item_chunks = p.item_chunks;
}

static void use_tiles(AttnArgs &a, const Csr *h, bool transposed, int kind) {
    const AttnTiles &t = h->attn->tiles[transposed][kind];
    a.rows_log = 4 - kind;
    a.chunk0 = t.chunk0;
    a.chunks = t.chunks;
}

void free_attn_plans(Csr *h) {
    if (!h->attn) return;
    for (int t = 0; t < 2; ++t)
        for (int l = 0; l < kAttnLevels; ++l) {
            free_plan(&h->attn->row[t][l]);
            for (int k = 0; k < kTileKinds; ++k) free_plan(&h->attn->tile[t][k][l]);
        }
    for (int t = 0; t < 2; ++t)
        for (AttnTiles &x : h->attn->tiles[t]) free_tiles(&x);
    delete h->attn;
    h->attn = nullptr;
}

// ---------------------------------------------------------- row kernels ----
// A group of L lanes takes one (system, item, head); lane l holds the elements
// (i * L + l) * VEC + e of the head.  Neighbouring groups take neighbouring
// heads, so a warp reads consecutive memory of a gathered row.  The entries of
// the item are walked STEP at a time with their loads issued together.
// Bound by the gathers (2 * dim elements an entry and head, mostly from L1 and L2)
// and, for short rows, by the instructions around them.  128 systems of a 32 x 32
// grid, 4 heads of 32 float32 elements (67 MB a tensor): forward 98 us, dq and the
// stored (p, ds) 150 us, dk and dv 96 us, 2.7 to 3.0 TB/s of the bytes that cannot
// be left out.
namespace {

constexpr int kAttnThreads = 128;

template <int L>
__device__ __forceinline__ unsigned group_mask() {
    if constexpr (L == 32) return 0xffffffffu;
    else return ((1u << L) - 1u) << ((threadIdx.x & 31) & ~(L - 1));
}

template <int L, typename A>
__device__ __forceinline__ A group_sum(A v, unsigned mask) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o);
    return v;
}

// Head blocks: `hb` (a power of two) consecutive heads of an item sit in
// neighbouring groups; blockIdx.y counts systems and head blocks.
struct Item { int64_t b; int row, t0, t1, slot, h; };

template <int L>
__device__ __forceinline__ bool load_item(Item &r, const AttnArgs &a, unsigned y, int heads, int hb_log) {
    const unsigned blocks = (unsigned)heads >> hb_log, b = y / blocks;
    const unsigned group = threadIdx.x / L;
    const int64_t it = (int64_t)blockIdx.x * ((kAttnThreads / L) >> hb_log) + (group >> hb_log);
    if (it >= a.n_items) return false;
    r.b = b;
    r.h = (int)(((y - b * blocks) << hb_log) + (group & ((1u << hb_log) - 1u)));
    r.row = a.item_unit ? __ldg(a.item_unit + it) : (int)it;
    r.t0 = __ldg(a.rowptr + r.row);
    r.t1 = __ldg(a.rowptr + r.row + 1);
    r.slot = -1;
    if (a.item_unit) {
        r.slot = __ldg(a.item_slot + it);
        const int64_t begin = (int64_t)r.t0 + (int64_t)__ldg(a.item_seg + it) * a.seg_len;
        const int64_t end = begin + (r.slot < 0 ? INT_MAX : a.seg_len);     // whole rows may be longer
        r.t0 = (int)begin;
        r.t1 = (int)(end < r.t1 ? end : (int64_t)r.t1);
    }
    return true;
}

// The vectors of one head this lane holds; 32-bit ones in pairs, for the
// two-wide multiply-add.
template <typename T, int VEC, int L, int NV>
struct Frag {
    using A = typename AccOf<T>::type;
    static constexpr int N = NV * VEC;
    static constexpr bool kPairs = sizeof(A) == 4 && N % 2 == 0;
    A x[N];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] = (A)0;
    }
    template <typename I>
    __device__ __forceinline__ void load(const I *p, int dim, int lane) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int d = (i * L + lane) * VEC;
            if (d < dim) {
                const Pack<I, VEC> r = load_pack<I, VEC>(p + d);
#pragma unroll
                for (int e = 0; e < VEC; ++e) x[i * VEC + e] = to_acc(r.e[e]);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) x[i * VEC + e] = (A)0;
            }
        }
    }
    __device__ __forceinline__ A dot(const Frag &y) const {
        if constexpr (kPairs) {
            float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int e = 0; e < N; e += 2) s = fma2(make_float2(x[e], x[e + 1]), make_float2(y.x[e], y.x[e + 1]), s);
            return s.x + s.y;
        } else {
            A s = (A)0;
#pragma unroll
            for (int e = 0; e < N; ++e) s = fma(x[e], y.x[e], s);
            return s;
        }
    }
    __device__ __forceinline__ void axpy(A w, const Frag &y) {
        if constexpr (kPairs) {
#pragma unroll
            for (int e = 0; e < N; e += 2) {
                const float2 r = fma2(make_float2(w, w), make_float2(y.x[e], y.x[e + 1]), make_float2(x[e], x[e + 1]));
                x[e] = r.x;
                x[e + 1] = r.y;
            }
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) x[e] = fma(w, y.x[e], x[e]);
        }
    }
    __device__ __forceinline__ void scale(A w) {
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] *= w;
    }
    __device__ __forceinline__ bool bad() const {
        bool b = false;
#pragma unroll
        for (int e = 0; e < N; ++e) b = b || x[e] != x[e];
        return b;
    }
    template <typename O>
    __device__ __forceinline__ void store(O *p, int dim, int lane) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int d = (i * L + lane) * VEC;
            if (d < dim) {
                Pack<O, VEC> r;
#pragma unroll
                for (int e = 0; e < VEC; ++e) r.e[e] = from_acc<O>(x[i * VEC + e]);
                if constexpr (sizeof(O) * VEC % 16 == 0) {
#pragma unroll
                    for (int e = 0; e < (int)sizeof(O) * VEC / 16; ++e)
                        reinterpret_cast<uint4 *>(p + d)[e] = reinterpret_cast<uint4 *>(&r)[e];
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) p[d + e] = r.e[e];
                }
            }
        }
    }
    // Partial sums, wherever they lie.
    __device__ __forceinline__ void store_odd(A *p, int dim, int lane) const {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int d = (i * L + lane) * VEC + e;
                if (d < dim) p[d] = x[i * VEC + e];
            }
    }
};

// Values of the STEP entries from t on (the last entry's beyond t1); -inf leaves
// an entry out, as does a place beyond t1.
template <typename A, int STEP>
__device__ __forceinline__ void load_values(A (&w)[STEP], const AttnArgs &a, int64_t b, int t, int t1) {
    const int64_t at = b * a.nnz;
    if (!a.vals) {
#pragma unroll
        for (int u = 0; u < STEP; ++u) w[u] = (A)0;
    } else if (!a.vals_f64) {
        const float *p = static_cast<const float *>(a.vals) + at;
#pragma unroll
        for (int u = 0; u < STEP; ++u) w[u] = (A)__ldg(p + min(t + u, t1 - 1));
    } else {
#pragma unroll
        for (int u = 0; u < STEP; ++u) w[u] = load_value<A>(a.vals, 1, at + min(t + u, t1 - 1));
    }
#pragma unroll
    for (int u = 0; u < STEP; ++u) w[u] = t + u < t1 ? w[u] : neg_inf<A>();
}

template <typename T, int VEC, int L, int NV, int STEP>
__global__ void __launch_bounds__(kAttnThreads) attn_fwd_rows_kernel(const __grid_constant__ AttnArgs a, int hb_log) {
    using A = typename AccOf<T>::type;
    using F = Frag<T, VEC, L, NV>;
    const int lane = threadIdx.x & (L - 1);
    const unsigned mask = group_mask<L>(), n_y = ((unsigned)a.heads >> hb_log) * (unsigned)a.batch;
    for (unsigned y = blockIdx.y; y < n_y; y += gridDim.y) {
        Item it;
        if (!load_item<L>(it, a, y, a.heads, hb_log)) return;
        const int h = it.h, kh = h / (a.heads / a.kv_heads);
        F q, acc;
        q.load(static_cast<const T *>(a.q) + it.b * a.qs[0] + it.row * a.qs[1] + h * a.qs[2], a.dim, lane);
        acc.zero();
        const T *kb = static_cast<const T *>(a.k) + it.b * a.ks[0] + kh * a.ks[2];
        const T *vb = static_cast<const T *>(a.v) + it.b * a.vs[0] + kh * a.vs[2];
        const A scale = (A)a.scale, none = neg_inf<A>();
        A m = none, l = (A)0;
        for (int t = it.t0; t < it.t1; t += STEP) {
            F kf[STEP], vf[STEP];
            A s[STEP], w[STEP];
            load_values<A, STEP>(w, a, it.b, t, it.t1);
#pragma unroll
            for (int u = 0; u < STEP; ++u) {
                const int64_t c = SLA_IDX((int64_t)__ldg(a.colind + min(t + u, it.t1 - 1)), a.n_cols, kBndColumn);
                kf[u].load(kb + c * a.ks[1], a.dim, lane);
                vf[u].load(vb + c * a.vs[1], a.dim, lane);
            }
            A top = m;
#pragma unroll
            for (int u = 0; u < STEP; ++u) {
                const A d = group_sum<L>(q.dot(kf[u]), mask);
                s[u] = w[u] == none ? none : fma(d, scale, w[u]);
                top = fmax(top, s[u]);
            }
            const A ref = top == none ? (A)0 : top;
            if (t > it.t0) {
                const A fix = exp_acc(m - ref);
                acc.scale(fix);
                l *= fix;
            }
            m = top;
#pragma unroll
            for (int u = 0; u < STEP; ++u) {
                const A p = exp_acc(s[u] - ref);
                l += p;
                if (w[u] != none) acc.axpy(p, vf[u]);    // what v holds elsewhere does not matter
            }
        }
        if (it.slot < 0) {
            const int64_t at = (it.b * a.n_rows + it.row) * a.heads + h;
            acc.scale(l > (A)0 || l != l ? (A)1 / l : (A)0);   // no entry left: zeros
            acc.store(static_cast<T *>(a.out) + at * a.dim, a.dim, lane);
            if (a.wide) acc.store(static_cast<A *>(a.wide) + at * a.dim, a.dim, lane);
            if (lane == 0) store_lse<A>(a, at, m, l);
        } else {
            const int64_t at = part_index(it.slot, a.n_slots, (int)it.b, 1, 0, a.heads, h);
            acc.store_odd(static_cast<A *>(a.part) + at * a.dim, a.dim, lane);
            if (lane == 0) {
                static_cast<A *>(a.part_ml)[at * 2] = m;
                static_cast<A *>(a.part_ml)[at * 2 + 1] = l;
            }
        }
    }
}

// Joins the segments of split rows: a block of W warps a (system, split unit,
// row, head).  A lane holds the elements lane + 32 i of the head; the warps take
// the segments in turn, 4 at a time with their loads in flight together, and
// are added up in order.
template <typename A, int W>
__device__ __forceinline__ A join_block(A v, A *red, bool take_max) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const A u = __shfl_xor_sync(0xffffffffu, v, o);
        v = take_max ? fmax(v, u) : v + u;
    }
    if constexpr (W > 1) {
        __syncthreads();
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int w = 1; w < W; ++w) v = take_max ? fmax(v, red[w]) : v + red[w];
    }
    return v;
}

struct JoinAt { int b, h, r, s0, n; int64_t row; };
__device__ __forceinline__ bool join_at(JoinAt &j, int64_t w, int n_rows, int rows, int heads, int n_multi,
                                        const int32_t *multi_unit, const int32_t *multi_slot) {
    j.h = (int)(w % heads);
    j.r = (int)(w / heads % rows);
    const int mu = (int)(w / heads / rows % n_multi);
    j.b = (int)(w / heads / rows / n_multi);
    j.row = (int64_t)__ldg(multi_unit + mu) * rows + j.r;
    j.s0 = __ldg(multi_slot + mu);
    j.n = __ldg(multi_slot + mu + 1) - j.s0;
    return j.row < n_rows;
}

template <typename T, int W>
__global__ void __launch_bounds__(32 * W)
attn_join_kernel(const AttnArgs a, int rows, int n_multi, const int32_t *__restrict__ multi_unit,
                 const int32_t *__restrict__ multi_slot) {
    using A = typename AccOf<T>::type;
    __shared__ A red[W];
    __shared__ A sums[W > 1 ? W : 1][W > 1 ? 256 : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    JoinAt j;
    if (!join_at(j, blockIdx.x, a.n_rows, rows, a.heads, n_multi, multi_unit, multi_slot)) return;
    const int64_t from = part_index(j.s0, a.n_slots, j.b, rows, j.r, a.heads, j.h), seg = (int64_t)rows * a.heads;
    const int64_t step = seg * a.dim;
    const A *p = static_cast<const A *>(a.part) + from * a.dim, *ml = static_cast<const A *>(a.part_ml) + from * 2;
    const A none = neg_inf<A>();
    A m = none, l = (A)0;
    for (int s = threadIdx.x; s < j.n; s += 32 * W) m = fmax(m, ml[s * seg * 2]);
    m = join_block<A, W>(m, red, true);
    const A ref = m == none ? (A)0 : m;
    for (int s = threadIdx.x; s < j.n; s += 32 * W) l += ml[s * seg * 2 + 1] * exp_acc(ml[s * seg * 2] - ref);
    l = join_block<A, W>(l, red, false);
    const A inv = l > (A)0 || l != l ? (A)1 / l : (A)0;
    A x[8] = {};
    for (int s = warp; s < j.n; s += 4 * W) {
        A w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) w[u] = s + u * W < j.n ? exp_acc(ml[(s + u * W) * seg * 2] - ref) : (A)0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i * 32 + lane < a.dim)
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (s + u * W < j.n) x[i] = fma(w[u], p[(s + u * W) * step + i * 32 + lane], x[i]);
    }
    if constexpr (W > 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sums[warp][i * 32 + lane] = x[i];
        __syncthreads();
    }
    const int64_t at = ((int64_t)j.b * a.n_rows + j.row) * a.heads + j.h;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int d = i * 32 + lane;
        if (d >= a.dim || i % W != warp) continue;
        A y = x[i];
        if constexpr (W > 1) {
            y = sums[0][d];
#pragma unroll
            for (int w = 1; w < W; ++w) y += sums[w][d];
        }
        static_cast<T *>(a.out)[at * a.dim + d] = from_acc<T>(y * inv);
        if (a.wide) static_cast<A *>(a.wide)[at * a.dim + d] = y * inv;
    }
    if (threadIdx.x == 0) store_lse<A>(a, at, m, l);
}

// Gradients by A's rows: p and ds of every entry and head, and dq.
template <typename T, int VEC, int L, int NV, int STEP>
__global__ void __launch_bounds__(kAttnThreads) attn_bwd_rows_kernel(const __grid_constant__ AttnArgs a, int hb_log) {
    using A = typename AccOf<T>::type;
    using F = Frag<T, VEC, L, NV>;
    const int lane = threadIdx.x & (L - 1);
    const unsigned mask = group_mask<L>(), n_y = ((unsigned)a.heads >> hb_log) * (unsigned)a.batch;
    for (unsigned y = blockIdx.y; y < n_y; y += gridDim.y) {
        Item it;
        if (!load_item<L>(it, a, y, a.heads, hb_log)) return;
        const int h = it.h, kh = h / (a.heads / a.kv_heads);
        const int64_t at = (it.b * a.n_rows + it.row) * a.heads + h;
        F q, go, acc;
        q.load(static_cast<const T *>(a.q) + it.b * a.qs[0] + it.row * a.qs[1] + h * a.qs[2], a.dim, lane);
        go.load(static_cast<const T *>(a.dout) + it.b * a.ds[0] + it.row * a.ds[1] + h * a.ds[2], a.dim, lane);
        acc.load(static_cast<const A *>(a.o) + at * a.dim, a.dim, lane);
        const A delta = group_sum<L>(go.dot(acc), mask);
        const A m = static_cast<const A *>(a.lse)[2 * at], l = static_cast<const A *>(a.lse)[2 * at + 1];
        const A inv = (A)1 / l;
        acc.zero();
        const T *kb = static_cast<const T *>(a.k) + it.b * a.ks[0] + kh * a.ks[2];
        const T *vb = static_cast<const T *>(a.v) + it.b * a.vs[0] + kh * a.vs[2];
        const A scale = (A)a.scale, none = neg_inf<A>();
        A *pds = static_cast<A *>(a.pds) + (it.b * a.nnz * a.heads + h) * 2;
        for (int t = it.t0; t < it.t1; t += STEP) {
            F kf[STEP], vf[STEP];
            A w[STEP], p[STEP], ds[STEP];
            load_values<A, STEP>(w, a, it.b, t, it.t1);
#pragma unroll
            for (int u = 0; u < STEP; ++u) {
                const int64_t c = SLA_IDX((int64_t)__ldg(a.colind + min(t + u, it.t1 - 1)), a.n_cols, kBndColumn);
                kf[u].load(kb + c * a.ks[1], a.dim, lane);
                vf[u].load(vb + c * a.vs[1], a.dim, lane);
            }
#pragma unroll
            for (int u = 0; u < STEP; ++u) {
                p[u] = q.dot(kf[u]);
                ds[u] = go.dot(vf[u]);
            }
#pragma unroll
            for (int u = 0; u < STEP; ++u) {
                const bool on = w[u] != none && l != (A)0;
                p[u] = group_sum<L>(p[u], mask);
                ds[u] = group_sum<L>(ds[u], mask);
                p[u] = on ? exp_acc(fma(p[u], scale, w[u]) - m) * inv : (A)0;
                ds[u] = on ? p[u] * (ds[u] - delta) : (A)0;
                if (on) acc.axpy(ds[u], kf[u]);
            }
            if (a.pds) {
                // lane u writes entry t + u
#pragma unroll
                for (int u = 0; u < STEP; ++u)
                    if (lane == u % L && t + u < it.t1) {
                        A *e = pds + (int64_t)(t + u) * a.heads * 2;
                        if constexpr (sizeof(A) == 4) *reinterpret_cast<float2 *>(e) = make_float2(p[u], ds[u]);
                        else *reinterpret_cast<double2 *>(e) = make_double2(p[u], ds[u]);
                    }
            }
        }
        if (!a.dq) continue;
        acc.scale(scale);
        if (it.slot < 0) acc.store(static_cast<T *>(a.dq) + at * a.dim, a.dim, lane);
        else
            acc.store_odd(static_cast<A *>(a.part) +
                              part_index(it.slot, a.n_slots, (int)it.b, 1, 0, a.heads, h) * a.dim, a.dim, lane);
    }
}

// Gradients by A^T's rows, from the stored p and ds: dk and dv.  Partial sums
// of a split row: dk then dv.
template <typename T, int VEC, int L, int NV, int STEP>
__global__ void __launch_bounds__(kAttnThreads) attn_bwd_cols_kernel(const __grid_constant__ AttnArgs a, int hb_log) {
    using A = typename AccOf<T>::type;
    using F = Frag<T, VEC, L, NV>;
    const int lane = threadIdx.x & (L - 1), share = a.heads / a.kv_heads;
    const unsigned n_y = ((unsigned)a.kv_heads >> hb_log) * (unsigned)a.batch;
    for (unsigned y = blockIdx.y; y < n_y; y += gridDim.y) {
        Item it;
        if (!load_item<L>(it, a, y, a.kv_heads, hb_log)) return;
        F dk, dv;
        // Entries that were left out have p = ds = 0; what q and dout hold there (a
        // NaN, say) must not matter, but skipping them would make the loads wait for
        // p, so that is done only when a sum ends as a NaN.
        auto sums = [&](auto careful) {
            dk.zero();
            dv.zero();
            for (int h = it.h * share; h < (it.h + 1) * share; ++h) {
                const T *qb = static_cast<const T *>(a.q) + it.b * a.qs[0] + h * a.qs[2];
                const T *gb = static_cast<const T *>(a.dout) + it.b * a.ds[0] + h * a.ds[2];
                const A *pds = static_cast<const A *>(a.pds) + (it.b * a.nnz * a.heads + h) * 2;
                for (int t = it.t0; t < it.t1; t += STEP) {
                    F qf[STEP], gf[STEP];
                    A p[STEP], ds[STEP];
#pragma unroll
                    for (int u = 0; u < STEP; ++u) {
                        const int at = min(t + u, it.t1 - 1);
                        const int64_t i = SLA_IDX((int64_t)__ldg(a.colind + at), a.n_rows, kBndColumn);
                        const int64_t e = SLA_IDX((int64_t)__ldg(a.perm + at), a.nnz, kBndEntry);
                        qf[u].load(qb + i * a.qs[1], a.dim, lane);
                        gf[u].load(gb + i * a.ds[1], a.dim, lane);
                        if constexpr (sizeof(A) == 4) {
                            const float2 x = __ldg(reinterpret_cast<const float2 *>(pds + e * a.heads * 2));
                            p[u] = x.x;
                            ds[u] = x.y;
                        } else {
                            const double2 x = __ldg(reinterpret_cast<const double2 *>(pds + e * a.heads * 2));
                            p[u] = x.x;
                            ds[u] = x.y;
                        }
                    }
#pragma unroll
                    for (int u = 0; u < STEP; ++u) {
                        if constexpr (decltype(careful)::value) {
                            if (t + u >= it.t1 || p[u] == (A)0) continue;
                        }
                        dk.axpy(t + u < it.t1 ? ds[u] : (A)0, qf[u]);
                        dv.axpy(t + u < it.t1 ? p[u] : (A)0, gf[u]);
                    }
                }
            }
        };
        sums(std::false_type{});
        if (dk.bad() || dv.bad()) sums(std::true_type{});
        dk.scale((A)a.scale);
        if (it.slot < 0) {
            const int64_t at = ((it.b * a.n_cols + it.row) * a.kv_heads + it.h) * a.dim;
            if (a.dk) dk.store(static_cast<T *>(a.dk) + at, a.dim, lane);
            if (a.dv) dv.store(static_cast<T *>(a.dv) + at, a.dim, lane);
        } else {
            A *p = static_cast<A *>(a.part) +
                   part_index(it.slot, a.n_slots, (int)it.b, 1, 0, a.kv_heads, it.h) * 2 * a.dim;
            dk.store_odd(p, a.dim, lane);
            dv.store_odd(p + a.dim, a.dim, lane);
        }
    }
}

// out0 (and out1) of split rows: the segments' sums added in order, `width`
// elements a partial, the first `dim` for out0, the next for out1.
template <typename T, int W>
__global__ void __launch_bounds__(32 * W)
attn_join_sums_kernel(const typename AccOf<T>::type *__restrict__ part, int n_rows, int n_slots, int rows,
                      int heads, int dim, int width, int n_multi, const int32_t *__restrict__ multi_unit,
                      const int32_t *__restrict__ multi_slot, T *out0, T *out1) {
    using A = typename AccOf<T>::type;
    __shared__ A sums[W > 1 ? W : 1][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    JoinAt j;
    if (!join_at(j, blockIdx.x, n_rows, rows, heads, n_multi, multi_unit, multi_slot)) return;
    const int64_t step = (int64_t)rows * heads * width;
    const A *p = part + part_index(j.s0, n_slots, j.b, rows, j.r, heads, j.h) * width;
    const int64_t at = (((int64_t)j.b * n_rows + j.row) * heads + j.h) * dim;
    for (int d0 = 0; d0 < width; d0 += 32) {
        const int d = d0 + lane;
        A x = (A)0;
        if (d < width) {
#pragma unroll 8
            for (int s = warp; s < j.n; s += W) x += p[s * step + d];
        }
        if constexpr (W > 1) {
            __syncthreads();
            sums[warp][lane] = x;
            __syncthreads();
            x = sums[0][lane];
#pragma unroll
            for (int w = 1; w < W; ++w) x += sums[w][lane];
        }
        T *out = d < dim ? out0 : out1;
        if (out && d < width && warp == 0) out[at + (d < dim ? d : d - dim)] = from_acc<T>(x);
    }
}

// dvals_t = sum over the heads of ds_t, in the values' type; the same from
// [B][heads][nnz].
template <typename V>
__global__ void __launch_bounds__(256)
attn_dvals_heads_kernel(int64_t count, int64_t nnz, int heads, const float *__restrict__ ds, V *__restrict__ dvals) {
    const int64_t t = blockIdx.x * (int64_t)256 + threadIdx.x;
    if (t >= count) return;
    const float *p = ds + t / nnz * nnz * heads + t % nnz;
    float x = 0.0f;
    for (int h = 0; h < heads; ++h) x += p[h * nnz];
    dvals[t] = (V)x;
}

template <typename A, typename V>
__global__ void __launch_bounds__(256)
attn_dvals_kernel(int64_t count, int heads, const A *__restrict__ pds, V *__restrict__ dvals) {
    const int64_t t = blockIdx.x * (int64_t)256 + threadIdx.x;
    if (t >= count) return;
    A x = (A)0;
    for (int h = 0; h < heads; ++h) x += pds[(t * heads + h) * 2 + 1];
    dvals[t] = (V)x;
}

}  // namespace

// Warps a joined row: one while segments are few (one batch of loads each) and the
// rows many (513 rows of 256 entries, 8 query heads of 128: forward 37 us, 58 with
// 8), else 8 (one row of 1024 entries: 9.8 us, 11.6 with 1), and 16 where a few rows
// have many segments (one row of 4096 entries, 8 heads of 64: 11.7 us, 13.9 with 8; the
// 125 tiles of 2000 rows 20.2, 32.8 with 16).  Sums without a softmax take 8: 16 were
// no faster.
int join_warps(int64_t blocks, int most_segs) {
    if (blocks > 1024) return most_segs <= 16 ? 1 : 8;
    return most_segs <= 64 ? 8 : 16;
}

template <typename T>
sla_status attn_join(const AttnArgs &a, const AttnPlan &p, cudaStream_t s) {
    const int64_t blocks = (int64_t)a.batch * p.n_multi * p.rows * a.heads;
    SLA_REQUIRE(blocks < INT_MAX, "sla_attention: too many split rows, systems and heads");
    if (blocks == 0) return SLA_OK;
    const int warps = join_warps(blocks, p.most_segs);
    auto *kernel = warps == 1 ? attn_join_kernel<T, 1> : (warps == 8 ? attn_join_kernel<T, 8> : attn_join_kernel<T, 16>);
    kernel<<<(unsigned)blocks, 32 * warps, 0, s>>>(a, p.rows, p.n_multi, p.multi_unit, p.multi_slot);
    SLA_CHECK_LAUNCH();
    return SLA_OK;
}

template <typename T>
sla_status attn_join_sums(const AttnArgs &a, const AttnPlan &p, int n_rows, int heads, int width, void *out0, void *out1,
                          cudaStream_t s) {
    const int64_t blocks = (int64_t)a.batch * p.n_multi * p.rows * heads;
    SLA_REQUIRE(blocks < INT_MAX, "sla_attention: too many split rows, systems and heads");
    if (blocks == 0) return SLA_OK;
    const auto *part = static_cast<const typename AccOf<T>::type *>(a.part);
    T *o0 = static_cast<T *>(out0), *o1 = static_cast<T *>(out1);
    const int warps = join_warps(blocks, p.most_segs);
    auto *kernel = warps == 1 ? attn_join_sums_kernel<T, 1> : attn_join_sums_kernel<T, 8>;
    kernel<<<(unsigned)blocks, warps == 1 ? 32 : 256, 0, s>>>(part, n_rows, p.n_slots, p.rows, heads, a.dim, width, p.n_multi,
                                                              p.multi_unit, p.multi_slot, o0, o1);
    SLA_CHECK_LAUNCH();
    return SLA_OK;
}

namespace {

// -------------------------------------------------------------- launches ----
enum { kFwd, kBwdRows, kBwdCols };

template <typename T, int VEC, int L, int NV, int STEP>
sla_status launch_rows(int what, const AttnArgs &a, cudaStream_t s) {
    const int heads = what == kBwdCols ? a.kv_heads : a.heads;
    int hb = 0;                          // the largest power of two that divides the heads and fits a block
    while ((2 << hb) <= kAttnThreads / L && heads % (2 << hb) == 0) ++hb;
    const int64_t x = ((int64_t)a.n_items + ((kAttnThreads / L) >> hb) - 1) / ((kAttnThreads / L) >> hb);
    const int64_t y = (int64_t)(heads >> hb) * a.batch;
    SLA_REQUIRE(x < INT_MAX && y < INT_MAX, "sla_attention: too many rows, systems and heads");
    if (x == 0) return SLA_OK;
    const dim3 grid((unsigned)x, (unsigned)(y < 65535 ? y : 65535));
    if (what == kFwd) attn_fwd_rows_kernel<T, VEC, L, NV, STEP><<<grid, kAttnThreads, 0, s>>>(a, hb);
    else if (what == kBwdRows) attn_bwd_rows_kernel<T, VEC, L, NV, STEP><<<grid, kAttnThreads, 0, s>>>(a, hb);
    else attn_bwd_cols_kernel<T, VEC, L, NV, STEP><<<grid, kAttnThreads, 0, s>>>(a, hb);
    SLA_CHECK_LAUNCH();
    return SLA_OK;
}

// Entries in flight: 4 or 5, whichever leaves fewer places empty on a row of mean
// length (a 5-point row in one step instead of two: the 128 systems above take 98,
// 150 and 96 us with 5, 112, 166 and 102 with 4); 2 where the registers hold no
// more.
template <typename T, int VEC, int L, int NV>
sla_status launch_rows(int what, const AttnArgs &a, cudaStream_t s) {
    constexpr int bytes = NV * VEC * (int)sizeof(typename AccOf<T>::type);
    if constexpr (bytes <= 32) {
        const int64_t rows = what == kBwdCols ? a.n_cols : a.n_rows, mean = (a.nnz + rows - 1) / (rows > 0 ? rows : 1);
        if ((mean + 4) / 5 * 5 < (mean + 3) / 4 * 4) return launch_rows<T, VEC, L, NV, 5>(what, a, s);
        return launch_rows<T, VEC, L, NV, 4>(what, a, s);
    } else {
        return launch_rows<T, VEC, L, NV, 2>(what, a, s);
    }
}

// Lanes and vectors a lane by the head's width.  Two 16-byte vectors a lane share
// the loop's instructions (32 float32 elements: 97 us with 4 lanes, 123 with 8); a
// group's load still covers 64 bytes or more where the head has them.
template <typename T>
sla_status launch_rows_of(int what, const AttnArgs &a, bool vec, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    if (vec) {
        const int n = a.dim / V;
        if (n <= 4) return launch_rows<T, V, 4, 1>(what, a, s);
        if (n <= 8) return launch_rows<T, V, 4, 2>(what, a, s);
        if (n <= 16) return launch_rows<T, V, 8, 2>(what, a, s);
        if (n <= 32) return launch_rows<T, V, 16, 2>(what, a, s);
        if (n <= 64) return launch_rows<T, V, 32, 2>(what, a, s);
        return launch_rows<T, V, 32, 4>(what, a, s);
    }
    if (a.dim <= 64) return launch_rows<T, 1, 32, 2>(what, a, s);
    return launch_rows<T, 1, 32, 8>(what, a, s);
}

bool on_16_bytes(const void *p, const int64_t st[3], size_t size) {
    if ((uintptr_t)p & 15) return false;
    for (int i = 0; i < 3; ++i)
        if ((st[i] * (int64_t)size) & 15) return false;
    return true;
}

size_t acc_size(int32_t dt) { return dt == SLA_F64 ? 8 : 4; }

template <typename T>
sla_status attn_forward(const Csr *h, const AttnPlan &p, AttnArgs a, bool tiled, int kind, cudaStream_t s) {
    using A = typename AccOf<T>::type;
    use_plan(a, p);
    use_tiles(a, h, false, kind);
    sla_status st;
    if constexpr (sizeof(T) == 2) {
        if (tiled) {
            st = attn_tile_forward<T>(a, s);
            return st != SLA_OK ? st : attn_join<T>(a, p, s);
        }
    }
    const int64_t dense[3] = {(int64_t)a.dim, (int64_t)a.dim, (int64_t)a.dim};
    const bool vec = a.dim % (16 / (int)sizeof(T)) == 0 && on_16_bytes(a.q, a.qs, sizeof(T)) &&
                     on_16_bytes(a.k, a.ks, sizeof(T)) && on_16_bytes(a.v, a.vs, sizeof(T)) &&
                     on_16_bytes(a.out, dense, sizeof(T)) && on_16_bytes(a.wide, dense, sizeof(A));
    st = launch_rows_of<T>(kFwd, a, vec, s);
    return st != SLA_OK ? st : attn_join<T>(a, p, s);
}

template <typename A, typename V>
sla_status attn_dvals(const AttnArgs &a, bool tiled, cudaStream_t s) {
    const int64_t entries = (int64_t)a.batch * a.nnz;
    if (entries == 0) return SLA_OK;
    if (tiled)
        attn_dvals_heads_kernel<V><<<blocks_of(entries), 256, 0, s>>>(entries, a.nnz, a.heads, a.ds_out,
                                                                     static_cast<V *>(a.dvals));
    else
        attn_dvals_kernel<A, V><<<blocks_of(entries), 256, 0, s>>>(entries, a.heads, static_cast<const A *>(a.pds),
                                                                   static_cast<V *>(a.dvals));
    SLA_CHECK_LAUNCH();
    return SLA_OK;
}

template <typename T>
sla_status attn_backward(const Csr *h, const AttnPlan &p, const AttnPlan &pt, AttnArgs a, bool tiled, int kind,
                         cudaStream_t s) {
    using A = typename AccOf<T>::type;
    const int64_t dense[3] = {(int64_t)a.dim, (int64_t)a.dim, (int64_t)a.dim};
    const bool vec = a.dim % (16 / (int)sizeof(T)) == 0 && on_16_bytes(a.q, a.qs, sizeof(T)) &&
                     on_16_bytes(a.k, a.ks, sizeof(T)) && on_16_bytes(a.v, a.vs, sizeof(T)) &&
                     on_16_bytes(a.dout, a.ds, sizeof(T)) && on_16_bytes(a.o, dense, sizeof(A)) &&
                     on_16_bytes(a.dq, dense, sizeof(T)) && on_16_bytes(a.dk, dense, sizeof(T)) &&
                     on_16_bytes(a.dv, dense, sizeof(T));
    use_plan(a, p);
    use_tiles(a, h, false, kind);
    sla_status st;
    if constexpr (sizeof(T) == 2) st = tiled ? attn_tile_bwd_rows<T>(a, s) : launch_rows_of<T>(kBwdRows, a, vec, s);
    else st = launch_rows_of<T>(kBwdRows, a, vec, s);
    if (st != SLA_OK) return st;
    if (a.dq && (st = attn_join_sums<T>(a, p, a.n_rows, a.heads, a.dim, a.dq, nullptr, s)) != SLA_OK) return st;
    if (a.dvals) {
        st = a.vals_f64 ? attn_dvals<A, double>(a, tiled, s) : attn_dvals<A, float>(a, tiled, s);
        if (st != SLA_OK) return st;
    }
    if (!a.dk && !a.dv) return SLA_OK;
    use_plan(a, pt);
    use_tiles(a, h, true, kind);
    a.rowptr = h->rowptrT;
    a.colind = h->colindT;
    a.perm = h->permT;
    if constexpr (sizeof(T) == 2) st = tiled ? attn_tile_bwd_cols<T>(a, s) : launch_rows_of<T>(kBwdCols, a, vec, s);
    else st = launch_rows_of<T>(kBwdCols, a, vec, s);
    if (st != SLA_OK) return st;
    return attn_join_sums<T>(a, pt, a.n_cols, a.kv_heads, 2 * a.dim, a.dk, a.dv, s);
}

// Workspace pieces: what the backward keeps for every entry (row kernels) or
// row (tile kernels), then the partial sums of split rows.
struct AttnWs {
    size_t pds = 0, stat = 0, ds = 0, vals_w = 0, part = 0, part_ml = 0;
    size_t total() const {
        return align_up(pds) + align_up(stat) + align_up(ds) + align_up(vals_w) + align_up(part) + align_up(part_ml);
    }
};

const AttnPlan &plan_of(const Csr *h, const sla_attn_opts *o, bool transposed) {
    const int l = attn_level(h, o);
    if (!attn_tiled(o)) return h->attn->row[transposed][l];
    return h->attn->tile[transposed][attn_tile_kind(o)][l];
}

// `what`: as for sla_attention_workspace_bytes.
AttnWs attn_ws(const Csr *h, const sla_attn_opts *o, int what) {
    const size_t acc = acc_size(o->dtype), B = (size_t)h->batch, H = (size_t)o->heads, D = (size_t)o->dim;
    const AttnPlan &p = plan_of(h, o, false), &pt = plan_of(h, o, true);
    const bool tiled = attn_tiled(o), vals = !(what & SLA_ATTN_NO_VALS), dvals = vals && !(what & SLA_ATTN_NO_DVALS),
               dq = !(what & SLA_ATTN_NO_DQ), cols = !(what & SLA_ATTN_NO_DK_DV);
    AttnWs w;
    // the values as the tiles read them: in 32 bits, and for dk and dv in A^T's order
    if (tiled && vals && (h->dtype == SLA_F64 || ((what & 1) && cols))) w.vals_w = B * (size_t)h->nnz * sizeof(float);
    if (!(what & 1)) {
        w.part = B * p.n_slots * p.rows * H * D * acc;
        w.part_ml = B * p.n_slots * p.rows * H * 2 * acc;
        return w;
    }
    if (tiled) {
        w.stat = B * H * (size_t)h->n_rows * sizeof(float4);
        if (dvals) w.ds = B * H * (size_t)h->nnz * sizeof(float);
    } else if (cols || dvals) {
        w.pds = B * (size_t)h->nnz * H * 2 * acc;
    }
    if (dq) w.part = B * p.n_slots * p.rows * H * D * acc;
    if (cols) w.part = std::max(w.part, B * pt.n_slots * pt.rows * (size_t)o->kv_heads * 2 * D * acc);
    return w;
}

sla_status check_opts(const char *fn, const sla_attn_opts *o) {
    SLA_REQUIRE(o != nullptr, "%s: NULL options", fn);
    SLA_REQUIRE(o->dtype >= SLA_F64 && o->dtype <= SLA_F16, "%s: bad dtype %d", fn, o->dtype);
    SLA_REQUIRE(o->heads >= 1 && o->kv_heads >= 1 && o->heads % o->kv_heads == 0 && o->heads <= 65536,
                "%s: heads must be a positive multiple of kv_heads (%d, %d)", fn, o->heads, o->kv_heads);
    SLA_REQUIRE(o->dim >= 1 && o->dim <= 256, "%s: dim must be in [1, 256] (got %d)", fn, o->dim);
    SLA_REQUIRE(o->scale == o->scale && o->scale <= DBL_MAX && o->scale >= -DBL_MAX, "%s: scale is not finite", fn);
    SLA_REQUIRE(o->lse_pairs == 0 || o->lse_pairs == 1, "%s: lse_pairs must be 0 or 1 (got %d)", fn, o->lse_pairs);
    return SLA_OK;
}

sla_status check_device(const char *fn, const Csr *h) {
    SLA_REQUIRE(h != nullptr, "%s: NULL handle", fn);
    int dev = -1;
    SLA_CHECK_CUDA(cudaGetDevice(&dev));
    SLA_REQUIRE(dev == h->device, "%s: the handle lives on device %d, the current device is %d", fn, h->device, dev);
    SLA_REQUIRE(h->nnz <= INT_MAX - 64, "%s: nnz=%lld, at most 2^31 - 65", fn, (long long)h->nnz);   // steps beyond a row's end
    SLA_REQUIRE(h->n_rows <= INT_MAX - 512 && h->n_cols <= INT_MAX - 512, "%s: more than 2^31 - 513 rows or columns", fn);
    return SLA_OK;
}

bool plans_ready(const Csr *h, const sla_attn_opts *o, bool backward) {
    if (!h->attn || (backward && !h->has_transpose)) return false;
    return plan_of(h, o, false).built && (!backward || plan_of(h, o, true).built);
}

sla_status prepare(Csr *h, const sla_attn_opts *o, bool backward, cudaStream_t s) {
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &cap) != cudaSuccess || cap != cudaStreamCaptureStatusNone) {
        cudaGetLastError();
        set_error("sla_attention: the plan is built on first use, which a stream capture cannot hold; call "
                  "sla_attention_prepare before capturing");
        return SLA_ERR_UNSUPPORTED;
    }
    if (!h->attn) {
        h->attn = new (std::nothrow) AttnPlans();
        if (!h->attn) {
            set_error("sla_attention_prepare: out of memory");
            return SLA_ERR_OOM;
        }
    }
    sla_status st = SLA_OK;
    // A^T's tiles count their columns, one for each of the sharing heads, in 32 bits
    if (backward && o && attn_tiled(o))
        SLA_REQUIRE((h->nnz << attn_tile_kind(o)) <= (int64_t)UINT_MAX - 64,
                    "sla_attention: nnz=%lld with %d heads sharing a key head, 16-bit gradients take 2^32 / %d entries",
                    (long long)h->nnz, 1 << attn_tile_kind(o), 1 << attn_tile_kind(o));
    if (backward && (st = ensure_transpose(h, s)) != SLA_OK) return st;
    for (int l = 0; l < kAttnLevels; ++l)
        for (int tiled = 0; tiled < 2; ++tiled) {
            if (o && (bool)tiled != attn_tiled(o)) continue;
            const int kind = tiled ? (o ? attn_tile_kind(o) : 0) : kRowKind;
            st = ensure_plan(h, kind, false, l, s);
            if (st == SLA_OK && backward) st = ensure_plan(h, kind, true, l, s);
            if (st != SLA_OK) return st;
        }
    return SLA_OK;
}

// The tile kernels read 16 bytes at a time.
sla_status check_tiled(const char *fn, const sla_attn_opts *o, std::initializer_list<const void *> dense,
                       std::initializer_list<std::pair<const void *, const int64_t *>> strided) {
    if (!attn_tiled(o)) return SLA_OK;
    bool ok = true;
    for (const void *p : dense) ok = ok && ((uintptr_t)p & 15) == 0;
    for (const auto &x : strided) {
        ok = ok && on_16_bytes(x.first, x.second, 2);
        SLA_REQUIRE(x.second[1] >= 0 && x.second[1] < (int64_t)1 << 31, "%s: row strides must be below 2^31 elements", fn);
    }
    SLA_REQUIRE(ok, "%s: 16-bit heads of a multiple of 16 elements need addresses and strides of a multiple of 16 bytes",
                fn);
    return SLA_OK;
}

AttnArgs make_args(const Csr *h, const sla_attn_opts *o, const void *q, const void *k, const void *v,
                   const void *vals) {
    AttnArgs a{};
    a.n_rows = h->n_rows;
    a.n_cols = h->n_cols;
    a.batch = h->batch;
    a.nnz = h->nnz;
    a.rowptr = h->rowptr;
    a.colind = h->colind;
    a.heads = o->heads;
    a.kv_heads = o->kv_heads;
    a.dim = o->dim;
    a.scale = o->scale;
    a.q = q;
    a.k = k;
    a.v = v;
    a.vals = vals;
    a.vals_f64 = h->dtype == SLA_F64;
    a.lse_pairs = o->lse_pairs;
    for (int i = 0; i < 3; ++i) {
        a.qs[i] = o->q_stride[i];
        a.ks[i] = o->k_stride[i];
        a.vs[i] = o->v_stride[i];
        a.ds[i] = o->do_stride[i];
    }
    return a;
}

}  // namespace
}  // namespace sla

using namespace sla;

extern "C" sla_status sla_attention_prepare(sla_csr_t hh, const sla_attn_opts *o, int32_t backward, void *stream) {
    SLA_RANGE("sla_attention_prepare");
    clear_error();
    Csr *h = reinterpret_cast<Csr *>(hh);
    sla_status st = check_device("sla_attention_prepare", h);
    if (st == SLA_OK && o) st = check_opts("sla_attention_prepare", o);
    if (st != SLA_OK || (o && plans_ready(h, o, backward != 0))) return st;
    return prepare(h, o, backward != 0, as_stream(stream));
}

extern "C" size_t sla_attention_workspace_bytes(sla_csr_t hh, const sla_attn_opts *o, int32_t backward) {
    const Csr *h = reinterpret_cast<const Csr *>(hh);
    clear_error();
    if (!h || check_opts("sla_attention_workspace_bytes", o) != SLA_OK || !plans_ready(h, o, backward & 1)) return 0;
    return attn_ws(h, o, backward).total();
}

extern "C" sla_status sla_attention(sla_csr_t hh, const void *q, const void *k, const void *v, const void *vals,
                                    void *out, void *out_wide, void *lse, const sla_attn_opts *o, void *ws,
                                    size_t ws_bytes, void *stream) {
    SLA_RANGE("sla_attention");
    clear_error();
    Csr *h = reinterpret_cast<Csr *>(hh);
    sla_status st = check_device("sla_attention", h);
    if (st == SLA_OK) st = check_opts("sla_attention", o);
    if (st != SLA_OK) return st;
    if (h->n_rows == 0) return SLA_OK;
    SLA_REQUIRE(q && out && lse && (h->n_cols == 0 || (k && v)), "sla_attention: NULL pointer");
    SLA_REQUIRE((uintptr_t)lse % (acc_size(o->dtype) << o->lse_pairs) == 0, "sla_attention: lse is not aligned");
    if (o->dtype == SLA_F64 || o->dtype == SLA_F32) out_wide = nullptr;
    st = check_tiled("sla_attention", o, {out, out_wide}, {{q, o->q_stride}, {k, o->k_stride}, {v, o->v_stride}});
    if (st != SLA_OK) return st;
    cudaStream_t s = as_stream(stream);
    if (!plans_ready(h, o, false) && (st = prepare(h, o, false, s)) != SLA_OK) return st;
    const AttnWs ww = attn_ws(h, o, vals ? 0 : SLA_ATTN_NO_VALS);
    const size_t need = ww.total();
    SLA_REQUIRE(need == 0 || (ws && ws_bytes >= need), "sla_attention: workspace too small (%zu < %zu)", ws_bytes, need);
    SLA_REQUIRE(((uintptr_t)ws & 255) == 0, "sla_attention: workspace must be 256-byte aligned");
    AttnArgs a = make_args(h, o, q, k, v, vals);
    a.out = out;
    a.wide = out_wide;
    a.lse = lse;
    Carver c(ws);
    a.vals_w = reinterpret_cast<float *>(c.take<char>(ww.vals_w));
    a.part = c.take<char>(ww.part);
    a.part_ml = c.take<char>(ww.part_ml);
    const AttnPlan &p = plan_of(h, o, false);
    const bool tiled = attn_tiled(o);
    const int kind = attn_tile_kind(o);
    switch (o->dtype) {
        case SLA_F64: return attn_forward<double>(h, p, a, tiled, kind, s);
        case SLA_F32: return attn_forward<float>(h, p, a, tiled, kind, s);
        case SLA_BF16: return attn_forward<__nv_bfloat16>(h, p, a, tiled, kind, s);
        default: return attn_forward<__half>(h, p, a, tiled, kind, s);
    }
}

extern "C" sla_status sla_attention_grad(sla_csr_t hh, const void *q, const void *k, const void *v, const void *vals,
                                         const void *out, const void *lse, const void *dout, void *dq, void *dk,
                                         void *dv, void *dvals, const sla_attn_opts *o, void *ws, size_t ws_bytes,
                                         void *stream) {
    SLA_RANGE("sla_attention_grad");
    clear_error();
    Csr *h = reinterpret_cast<Csr *>(hh);
    sla_status st = check_device("sla_attention_grad", h);
    if (st == SLA_OK) st = check_opts("sla_attention_grad", o);
    if (st != SLA_OK) return st;
    SLA_REQUIRE(o->lse_pairs, "sla_attention_grad: needs the statistics of a forward call with lse_pairs");
    SLA_REQUIRE((uintptr_t)lse % (2 * acc_size(o->dtype)) == 0, "sla_attention_grad: lse is not aligned to its pairs");
    SLA_REQUIRE(!dvals || vals, "sla_attention_grad: dvals without vals");
    SLA_REQUIRE(h->n_rows == 0 || (q && out && lse && dout), "sla_attention_grad: NULL pointer");
    SLA_REQUIRE(h->n_cols == 0 || (k && v), "sla_attention_grad: NULL pointer");
    st = check_tiled("sla_attention_grad", o, {out, dq, dk, dv},
                     {{q, o->q_stride}, {k, o->k_stride}, {v, o->v_stride}, {dout, o->do_stride}});
    if (st != SLA_OK) return st;
    cudaStream_t s = as_stream(stream);
    if (!dq && !dk && !dv && !dvals) return SLA_OK;
    if (!plans_ready(h, o, true) && (st = prepare(h, o, true, s)) != SLA_OK) return st;
    const AttnWs w = attn_ws(h, o, 1 | (vals ? 0 : SLA_ATTN_NO_VALS) | (dvals ? 0 : SLA_ATTN_NO_DVALS) |
                                       (dq ? 0 : SLA_ATTN_NO_DQ) | (dk || dv ? 0 : SLA_ATTN_NO_DK_DV));
    SLA_REQUIRE(w.total() == 0 || (ws && ws_bytes >= w.total()), "sla_attention_grad: workspace too small (%zu < %zu)",
                ws_bytes, w.total());
    SLA_REQUIRE(((uintptr_t)ws & 255) == 0, "sla_attention_grad: workspace must be 256-byte aligned");
    AttnArgs a = make_args(h, o, q, k, v, vals);
    a.o = out;
    a.lse = const_cast<void *>(lse);
    a.dout = dout;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.dvals = dvals;
    Carver c(ws);
    a.pds = w.pds ? c.take<char>(w.pds) : nullptr;
    a.stat = reinterpret_cast<float4 *>(c.take<char>(w.stat));
    a.ds_out = w.ds ? reinterpret_cast<float *>(c.take<char>(w.ds)) : nullptr;
    a.vals_w = reinterpret_cast<float *>(c.take<char>(w.vals_w));
    a.part = c.take<char>(w.part);
    const AttnPlan &p = plan_of(h, o, false), &pt = plan_of(h, o, true);
    const bool tiled = attn_tiled(o);
    const int kind = attn_tile_kind(o);
    switch (o->dtype) {
        case SLA_F64: return attn_backward<double>(h, p, pt, a, tiled, kind, s);
        case SLA_F32: return attn_backward<float>(h, p, pt, a, tiled, kind, s);
        case SLA_BF16: return attn_backward<__nv_bfloat16>(h, p, pt, a, tiled, kind, s);
        default: return attn_backward<__half>(h, p, pt, a, tiled, kind, s);
    }
}
