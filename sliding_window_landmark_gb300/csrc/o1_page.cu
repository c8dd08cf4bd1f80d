// The paged cache: rows of keys and values written into it, quantised on the
// way, and read back; and the C ABI of the cache and of the attention over it.
//
// Bound of both copies: HBM, each value read once and written once. A group of
// LPV lanes takes head rows, 8 values a lane: up to four heads of a position, all
// in flight, while the next position's page is looked up. Of 16-bit rows a lane
// takes 8 values in a row; of fp32 rows 4 and the 4 that lie 4 LPV further on, so
// that an instruction of either side covers whole lines. 32749 fp32 rows of 4
// heads of 128 to e4m3: 34 us replayed from a graph, 4.9 TB/s, and 33 in a loop of
// calls (a head at a time, each with its own look and addresses, took 43:
// instruction issue).
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "o1_page.cuh"

namespace {

constexpr int CP_THREADS = 256, CP_BLOCKS = 4;   // of a block; blocks an SM

struct Vec8 {
    float x[8];
};
__device__ __forceinline__ void put4(Vec8 &v, int i, float4 f) {
    v.x[i] = f.x;
    v.x[i + 1] = f.y;
    v.x[i + 2] = f.z;
    v.x[i + 3] = f.w;
}
__device__ __forceinline__ float4 get4(const Vec8 &v, int i) { return make_float4(v.x[i], v.x[i + 1], v.x[i + 2], v.x[i + 3]); }
// 4 e4m3 codes
__device__ __forceinline__ float4 codes4(uint32_t w) {
    uint32_t h[2];
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[0]) : "h"((uint16_t)w));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[1]) : "h"((uint16_t)(w >> 16)));
    const float2 a = __half22float2(*(const __half2 *)&h[0]), b = __half22float2(*(const __half2 *)&h[1]);
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ uint32_t pack2(const __nv_bfloat16 *, float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *(const uint32_t *)&h;
}
__device__ __forceinline__ uint32_t pack2(const __half *, float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *(const uint32_t *)&h;
}

// A lane's 8 values of a head's row of `width`: how they lie for rows of T, as
// loads and stores of a row of R (T, or the cache's type).
template <typename T, int LPV>
struct Lay {
    static constexpr bool APART = sizeof(T) == 4;   // two runs of 4
    static __device__ __forceinline__ int at(int lane, int half) { return APART ? 4 * lane + 4 * LPV * half : 8 * lane + 4 * half; }
    static __device__ __forceinline__ bool on(int lane, int half, int width) { return at(lane, half) < width; }
    static __device__ __forceinline__ Vec8 load(const float *p, int lane, int width) {
        Vec8 v;
        put4(v, 0, on(lane, 0, width) ? o1_ld4(p + at(lane, 0)) : make_float4(0.f, 0.f, 0.f, 0.f));
        put4(v, 4, on(lane, 1, width) ? o1_ld4(p + at(lane, 1)) : make_float4(0.f, 0.f, 0.f, 0.f));
        return v;
    }
    template <typename R>
    static __device__ __forceinline__ Vec8 load(const R *p, int lane, int width) {   // 16 bits
        Vec8 v;
        if (APART) {
            put4(v, 0, on(lane, 0, width) ? o1_ld4(p + at(lane, 0)) : make_float4(0.f, 0.f, 0.f, 0.f));
            put4(v, 4, on(lane, 1, width) ? o1_ld4(p + at(lane, 1)) : make_float4(0.f, 0.f, 0.f, 0.f));
        } else {
            const uint4 u = on(lane, 0, width) ? *(const uint4 *)(p + 8 * lane) : make_uint4(0u, 0u, 0u, 0u);
            const uint2 h[2] = {make_uint2(u.x, u.y), make_uint2(u.z, u.w)};
            put4(v, 0, o1_ld4((const R *)&h[0]));
            put4(v, 4, o1_ld4((const R *)&h[1]));
        }
        return v;
    }
    static __device__ __forceinline__ Vec8 load(const uint8_t *p, int lane, int width) {   // codes
        Vec8 v;
        uint2 u = make_uint2(0u, 0u);
        if (APART) {
            if (on(lane, 0, width)) u.x = *(const uint32_t *)(p + at(lane, 0));
            if (on(lane, 1, width)) u.y = *(const uint32_t *)(p + at(lane, 1));
        } else if (on(lane, 0, width)) {
            u = *(const uint2 *)(p + 8 * lane);
        }
        put4(v, 0, codes4(u.x));
        put4(v, 4, codes4(u.y));
        return v;
    }
    static __device__ __forceinline__ void store(float *p, const Vec8 &v, int lane, int width) {
        if (on(lane, 0, width)) o1_st4(p + at(lane, 0), get4(v, 0));
        if (on(lane, 1, width)) o1_st4(p + at(lane, 1), get4(v, 4));
    }
    template <typename R>
    static __device__ __forceinline__ void store(R *p, const Vec8 &v, int lane, int width) {
        if (APART) {
            if (on(lane, 0, width)) o1_st4(p + at(lane, 0), get4(v, 0));
            if (on(lane, 1, width)) o1_st4(p + at(lane, 1), get4(v, 4));
        } else if (on(lane, 0, width)) {
            *(uint4 *)(p + 8 * lane) = make_uint4(pack2(p, v.x[0], v.x[1]), pack2(p, v.x[2], v.x[3]), pack2(p, v.x[4], v.x[5]),
                                                  pack2(p, v.x[6], v.x[7]));
        }
    }
    static __device__ __forceinline__ void store(uint8_t *p, uint2 codes, int lane, int width) {
        if (APART) {
            if (on(lane, 0, width)) *(uint32_t *)(p + at(lane, 0)) = codes.x;
            if (on(lane, 1, width)) *(uint32_t *)(p + at(lane, 1)) = codes.y;
        } else if (on(lane, 0, width)) {
            *(uint2 *)(p + 8 * lane) = codes;
        }
    }
};

// A head's row, LPV lanes of 8 values, as e4m3 codes under a power of two:
// returns the byte e + 127. With max |x| = 1.m 2^(E - 127) the least e has
// 1.m 2^(E - 127) <= 1.75 2^8 2^e, so e + 127 = E - 8, one more where 1.m > 1.75
// (fraction above 0x600000), and at least 1, which also takes rows of zeros and
// subnormals. The factor 2^-e is a normal number and x 2^-e exact unless it
// falls below fp32's range, far below e4m3's.
template <int LPV>
__device__ __forceinline__ uint32_t quantise8(Vec8 v, uint2 &codes) {
    constexpr uint32_t INF = 0x7f800000u;
    uint32_t top = 0;   // of |x| as bits, which are in its order
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v.x[i]) & 0x7fffffffu);
#pragma unroll
    for (int m = 1; m < LPV; m <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
    if (__any_sync(0xffffffffu, top >= INF)) {   // infinities and NaN: apart from the maximum, and NaN
        top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t x = __float_as_uint(v.x[i]) & 0x7fffffffu;
            if (x >= INF) v.x[i] = NAN;
            else top = max(top, x);
        }
#pragma unroll
        for (int m = 1; m < LPV; m <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
    }
    const int e = max(1, (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0));
    const float f = __uint_as_float((uint32_t)(254 - e) << 23);
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint16_t two;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(v.x[2 * i + 1] * f), "f"(v.x[2 * i] * f));
        h[i] = two;
    }
    codes = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
    return (uint32_t)e;
}

// A head's row into the cache at `at` (null: nowhere); every lane of the group
// calls it, with zeros past the row's end.
template <typename L, typename C, int LPV>
struct Store {
    static __device__ __forceinline__ void row(C *at, uint8_t *, const Vec8 &v, int lane, int width) {
        if (at) L::store(at, v, lane, width);
    }
};
template <typename L, int LPV>
struct Store<L, uint8_t, LPV> {
    static __device__ __forceinline__ void row(uint8_t *at, uint8_t *exp, const Vec8 &v, int lane, int width) {
        uint2 codes;
        const uint32_t e = quantise8<LPV>(v, codes);
        if (!at) return;
        L::store(at, codes, lane, width);
        if (lane == 0) *exp = (uint8_t)e;
    }
};
template <typename L, typename C>
__device__ __forceinline__ Vec8 cached8(const C *at, const uint8_t *, int lane, int width) { return L::load(at, lane, width); }
template <typename L>
__device__ __forceinline__ Vec8 cached8(const uint8_t *at, const uint8_t *exp, int lane, int width) {
    Vec8 v = L::load(at, lane, width);
    const float f = pg_scale(*exp);
#pragma unroll
    for (int i = 0; i < 8; ++i) v.x[i] *= f;
    return v;
}

// One side (keys or values) of a copy.
template <typename T, typename C>
struct Side {
    T *rows;
    C *pool;
    uint8_t *exp;
    size_t stride;
    int width;
};
template <typename T, typename C>
__device__ __forceinline__ Side<T, C> side_of(const PgArgs &a, bool keys, bool write) {
    if (keys) return {(T *)(write ? a.k_in : a.k_out), (C *)a.k, a.ke, a.ks, a.d};
    return {(T *)(write ? a.v_in : a.v_out), (C *)a.v, a.ve, a.vs, a.dv};
}

// Rows of the table's sequences to their places or back. Work is counted in
// (live row, four heads); a block takes a run of it, a group of LPV lanes every
// GROUPS-th of the run.
template <typename T, typename C, int LPV, bool WRITE>
__device__ __forceinline__ void copy_run(const PgArgs &a, const PgTable &tab, bool keys) {
    using L = Lay<T, LPV>;
    constexpr int GROUPS = CP_THREADS / LPV, U = 4;
    const Side<T, C> s = side_of<T, C>(a, keys, WRITE);
    const int lane = threadIdx.x % LPV, grp = threadIdx.x / LPV, four = (a.G + U - 1) / U;
    const int64_t all = (int64_t)tab.total * four, turns = (all + GROUPS - 1) / GROUPS;
    const int64_t v0 = turns * blockIdx.x / gridDim.x * GROUPS, v1 = min(all, turns * (blockIdx.x + 1) / gridDim.x * GROUPS);
    int i = (int)((v0 + grp) / four), g = (int)(v0 + grp - (int64_t)i * four);   // of this group's next piece
    const int step_i = GROUPS / four, step_g = GROUPS - step_i * four;
    int n = 0;
    for (int hi = tab.n - 1; n < hi;) {   // the last sequence that starts at or before row i
        const int mid = (n + hi + 1) >> 1;
        if (tab.s[mid].before <= i) n = mid;
        else hi = mid - 1;
    }
    struct Piece {
        int row, page, at, g;   // row of the tensors, page (-1: none), row in it, first head
    };
    auto piece = [&](int64_t v) {
        Piece p = {0, -1, 0, U * g};
        if (v < v1) {
            while (n + 1 < tab.n && tab.s[n + 1].before <= i) ++n;
            const int r = i - tab.s[n].before, pos = tab.s[n].pos0 + r;
            p.row = tab.s[n].row0 + r;
            p.page = pg_page(a, tab.s[n].slot, pos);
            p.at = pos & ((1 << a.lpage) - 1);
        }
        g += step_g;
        i += step_i;
        if (g >= four) g -= four, ++i;
        return p;
    };
    const size_t head = (size_t)s.width << a.lpage;   // from a group's rows of a page to the next one's
    Piece p = piece(v0 + grp);
    for (int64_t v = v0; v < v1; v += GROUPS) {
        T *row = s.rows + (size_t)p.row * s.stride + (size_t)p.g * s.width;
        const bool live = p.page >= 0;
        const size_t place = (((size_t)max(p.page, 0) * a.G + p.g) << a.lpage) + p.at;
        C *at = s.pool + place * s.width;
        uint8_t *exp = sizeof(C) == 1 ? s.exp + place : nullptr;
        const int heads = live ? min(U, a.G - p.g) : 0;
        Vec8 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u < heads) {
                if (WRITE) x[u] = L::load((const T *)row + (size_t)u * s.width, lane, s.width);
                else x[u] = cached8<L>((const C *)at + u * head, exp + ((size_t)u << a.lpage), lane, s.width);
            } else {
                x[u] = {{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}};
            }
        }
        p = piece(v + GROUPS + grp);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (WRITE) {
                if (u < a.G) Store<L, C, LPV>::row(u < heads ? at + u * head : nullptr, exp + ((size_t)u << a.lpage), x[u], lane, s.width);
            } else if (u < heads) {
                L::store(row + (size_t)u * s.width, x[u], lane, s.width);
            }
        }
    }
}

template <typename T, typename C, int LPV, bool WRITE>
__global__ __launch_bounds__(CP_THREADS, CP_BLOCKS) void k_pg_copy(PgArgs a, const __grid_constant__ PgTable tab) {
    copy_run<T, C, LPV, WRITE>(a, tab, blockIdx.y == 0);
}

// A decode step's rows, a block a row: the look for an earlier row of the same
// place, then its head rows.
template <typename T, typename C, int LPV>
__device__ __forceinline__ void token_side(const PgArgs &a, const PgRow &pr, int page, bool keys) {
    using L = Lay<T, LPV>;
    constexpr int GROUPS = CP_THREADS / LPV;
    const Side<T, C> s = side_of<T, C>(a, keys, true);
    const int lane = threadIdx.x % LPV, grp = threadIdx.x / LPV, w = pr.pos & ((1 << a.lpage) - 1);
    for (int g0 = 0; g0 < a.G; g0 += GROUPS) {   // the same number of turns for every lane: shuffles inside
        const int g = min(g0 + grp, a.G - 1);
        const bool live = g0 + grp < a.G;
        Vec8 x = {{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}};
        if (live) x = L::load((const T *)s.rows + (size_t)blockIdx.x * s.stride + (size_t)g * s.width, lane, s.width);
        Store<L, C, LPV>::row(live ? pg_at(s.pool, a, page, g, w, s.width) : nullptr, sizeof(C) == 1 ? pg_at(s.exp, a, page, g, w, 1) : nullptr,
                              x, lane, s.width);
    }
}
template <typename T, typename C, int LPV>
__global__ __launch_bounds__(CP_THREADS) void k_pg_token_write(PgArgs a) {
    const int r = blockIdx.x;
    const PgRow pr = pg_token_row(a, r);
    if (pr.slot < 0) return;
    const int page = pg_page(a, pr.slot, pr.pos);
    int dup = 0;
    for (int i = threadIdx.x; i < r; i += CP_THREADS) {
        const PgRow o = pg_token_row(a, i);
        dup |= o.slot == pr.slot && o.pos == pr.pos;
    }
    if (__syncthreads_or(dup) || page < 0) return;
    token_side<T, C, LPV>(a, pr, page, true);
    token_side<T, C, LPV>(a, pr, page, false);
}

// LPV lanes of 8 values a head's row (a power of two that holds the wider side).
template <typename T, typename C, bool WRITE, int LPV>
void copy_launch_l(const PgArgs &a, const PgTable *tab, cudaStream_t st) {
    if (!tab) {
        if (WRITE) k_pg_token_write<T, C, LPV><<<a.rows, CP_THREADS, 0, st>>>(a);
        return;
    }
    // one wave of blocks over both sides, fewer where the rows do not fill them
    const int64_t work = (int64_t)tab->total * ((a.G + 3) / 4), turn = CP_THREADS / LPV, want = (work + turn - 1) / turn;
    const int64_t most = 152 * CP_BLOCKS / 2;
    k_pg_copy<T, C, LPV, WRITE><<<dim3((unsigned)(want < most ? want : most), 2), CP_THREADS, 0, st>>>(a, *tab);
}
template <typename T, typename C, bool WRITE>
void copy_launch_c(const PgArgs &a, const PgTable *tab, cudaStream_t st) {
    const int w = a.d > a.dv ? a.d : a.dv;
    if (w <= 64) copy_launch_l<T, C, WRITE, 8>(a, tab, st);
    else if (w <= 128) copy_launch_l<T, C, WRITE, 16>(a, tab, st);
    else copy_launch_l<T, C, WRITE, 32>(a, tab, st);
}
// tab null: a token batch
template <bool WRITE>
void copy_launch(const PgArgs &a, int dtype, int cache_dtype, const PgTable *tab, cudaStream_t st) {
    if (dtype == O1_F32 && cache_dtype == O1_BF16) copy_launch_c<float, __nv_bfloat16, WRITE>(a, tab, st);
    else if (dtype == O1_F32) copy_launch_c<float, uint8_t, WRITE>(a, tab, st);
    else if (dtype == O1_BF16 && cache_dtype == O1_BF16) copy_launch_c<__nv_bfloat16, __nv_bfloat16, WRITE>(a, tab, st);
    else if (dtype == O1_BF16) copy_launch_c<__nv_bfloat16, uint8_t, WRITE>(a, tab, st);
    else if (cache_dtype == O1_F16) copy_launch_c<__half, __half, WRITE>(a, tab, st);
    else copy_launch_c<__half, uint8_t, WRITE>(a, tab, st);
}

// ------------------------------------------------------------ host checks

bool pg_geom_ok(const o1_pg_geom *g) {
    if (!g) return false;
    if (g->groups < 1 || g->groups > 4096) return false;
    if (g->heads_per_group < 1 || g->heads_per_group > O1_MAX_HPG) return false;
    if (g->groups * g->heads_per_group > 65535) return false;
    const int unit = g->cache_dtype == O1_E4M3 ? 16 : 8;   // 16 bytes of a cached row
    if (g->d < 8 || g->d > O1_MAX_D || g->d % unit || g->dv < 8 || g->dv > O1_MAX_DV || g->dv % unit) return false;
    if (g->page < 16 || g->page > 256 || (g->page & (g->page - 1))) return false;
    if (g->window < 0 || !o1_dtype_ok(g->dtype) || !isfinite(g->scale) || !(g->scale > 0.f)) return false;
    return g->cache_dtype == O1_E4M3 || g->cache_dtype == (g->dtype == O1_F16 ? O1_F16 : O1_BF16);
}

// The parts of a cache as spans: keys, values, their exponents, the table.
struct PgSpans {
    O1Span s[5];
};
bool cache_ok(const o1_pg_geom &g, const o1_pg_cache *c, PgSpans &sp) {
    if (!c || !c->k || !c->v || !c->table) return false;
    if ((uintptr_t)c->k % 16 || (uintptr_t)c->v % 16 || (uintptr_t)c->k_exp % 16 || (uintptr_t)c->v_exp % 16 ||
        (uintptr_t)c->table % 16)
        return false;
    if (g.cache_dtype == O1_E4M3 && (!c->k_exp || !c->v_exp)) return false;
    if (c->n_pages < 1 || c->n_slots < 1 || c->width < 1) return false;
    const int64_t lim = (int64_t)1 << 31;
    if ((int64_t)c->width * g.page >= lim || (int64_t)g.groups * g.page * c->n_pages >= lim) return false;
    const size_t rows = (size_t)c->n_pages * g.groups * g.page, e = pg_cache_bytes(g.cache_dtype);
    const bool q = g.cache_dtype == O1_E4M3;
    sp = {{o1_span(c->k, rows * g.d * e), o1_span(c->v, rows * g.dv * e), o1_span(q ? c->k_exp : nullptr, rows),
           o1_span(q ? c->v_exp : nullptr, rows), o1_span(c->table, (size_t)c->n_slots * c->width * 4)}};
    return true;
}
bool meets(const PgSpans &sp, const O1Span &x) {
    for (const O1Span &s : sp.s)
        if (o1_spans_overlap(s, x)) return true;
    return false;
}
// Whether the parts that a write touches are apart from each other and the table.
bool apart(const PgSpans &sp) {
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 5; ++j)
            if (o1_spans_overlap(sp.s[i], sp.s[j])) return false;
    return true;
}

// The sequences of a call: ranges in bounds, rows apart and, for writes,
// positions of a slot apart. Sorted copies on the stack.
constexpr int PG_MAX_SEQ = 4096;
bool seqs_ok(const o1_pg_seq *s, int n, const o1_pg_geom &g, const o1_pg_cache &c, int total_rows, bool write) {
    struct Range {
        int64_t key;   // slot 2^32 + first position, or the first row
        int32_t n;
    } r[PG_MAX_SEQ];
    const auto apart = [&](int m) {
        std::sort(r, r + m, [](const Range &a, const Range &b) { return a.key < b.key; });
        for (int i = 1; i < m; ++i)
            if (r[i - 1].key + r[i - 1].n > r[i].key) return false;
        return true;
    };
    const int64_t len = (int64_t)c.width * g.page;
    int m = 0;
    for (int i = 0; i < n; ++i) {
        if (s[i].row0 < 0 || s[i].rows < 0 || s[i].slot < 0 || s[i].slot >= c.n_slots || s[i].pos0 < 0) return false;
        if ((int64_t)s[i].row0 + s[i].rows > total_rows || (int64_t)s[i].pos0 + s[i].rows > len) return false;
        if (s[i].rows) r[m++] = {s[i].row0, s[i].rows};
    }
    if (!apart(m)) return false;
    if (!write) return true;
    m = 0;
    for (int i = 0; i < n; ++i)
        if (s[i].rows) r[m++] = {((int64_t)s[i].slot << 32) + s[i].pos0, s[i].rows};
    return apart(m);
}

void fill(PgArgs &a, const o1_pg_geom &g, const o1_pg_cache &c) {
    a = PgArgs();
    a.k = c.k; a.v = c.v; a.ke = c.k_exp; a.ve = c.v_exp; a.table = c.table;
    a.n_pages = c.n_pages; a.n_slots = c.n_slots; a.width = c.width;
    a.G = g.groups; a.hpg = g.heads_per_group; a.d = g.d; a.dv = g.dv; a.window = g.window; a.scale = g.scale;
    for (a.lpage = 4; 1 << a.lpage < g.page;) ++a.lpage;
    a.wait_cycles = o1_wait_limit();
}

// Sequences of some rows in tables of PG_TABLE, counted by `count` of their rows.
template <typename Count, typename Launch>
void for_tables(const o1_pg_seq *seqs, int n_seq, Count count, Launch launch) {
    PgTable t;
    t.n = t.total = 0;
    for (int i = 0; i < n_seq; ++i) {
        if (!seqs[i].rows) continue;
        const int64_t c = count(seqs[i].rows);
        if (t.n == PG_TABLE || t.total + c > INT32_MAX) {
            launch(t);
            t.n = t.total = 0;
        }
        t.s[t.n++] = {seqs[i].row0, seqs[i].rows, seqs[i].slot, seqs[i].pos0, t.total};
        t.total += (int32_t)c;
    }
    if (t.n) launch(t);
}

int copy_seqs(const o1_pg_geom *geom, const o1_pg_cache *cache, const void *k, int64_t ks, const void *v, int64_t vs,
              const o1_pg_seq *seqs, int32_t n_seq, int32_t total_rows, bool write, cudaStream_t st) {
    if (!pg_geom_ok(geom)) return O1_ERR_UNSUPPORTED;
    const o1_pg_geom &g = *geom;
    PgSpans sp;
    if (!cache_ok(g, cache, sp) || (write && !apart(sp))) return O1_ERR_ARG;
    if (n_seq < 0 || n_seq > PG_MAX_SEQ || total_rows < 0) return O1_ERR_ARG;
    if (n_seq == 0) return O1_OK;
    if (!seqs || !seqs_ok(seqs, n_seq, g, *cache, total_rows, write)) return O1_ERR_ARG;
    if (total_rows == 0) return O1_OK;
    const O1Span kk = o1_row_span(k, g.dtype, g.groups, g.d, ks, total_rows),
                 vv = o1_row_span(v, g.dtype, g.groups, g.dv, vs, total_rows);
    if (!o1_rows_ok(kk) || !o1_rows_ok(vv) || meets(sp, kk) || meets(sp, vv)) return O1_ERR_ARG;
    if (!write && o1_spans_overlap(kk, vv)) return O1_ERR_ARG;
    PgArgs a;
    fill(a, g, *cache);
    if (write) a.k_in = k, a.v_in = v;
    else a.k_out = (void *)k, a.v_out = (void *)v;
    a.ks = (size_t)ks; a.vs = (size_t)vs;
    for_tables(seqs, n_seq, [](int rows) { return (int64_t)rows; }, [&](const PgTable &t) {
        if (write) copy_launch<true>(a, g.dtype, g.cache_dtype, &t, st);
        else copy_launch<false>(a, g.dtype, g.cache_dtype, &t, st);
    });
    return cudaGetLastError() == cudaSuccess ? O1_OK : O1_ERR_CUDA;
}

// Checks of the two attend calls; fills the kernels' arguments.
int attend_args(PgArgs &a, const o1_pg_geom &g, const o1_pg_cache *cache, void *scratch, size_t scratch_bytes,
                const void *q, int64_t qs, void *out, int64_t os, int32_t rows, const O1Span &slots, const O1Span &pos) {
    PgSpans sp;
    if (!cache_ok(g, cache, sp)) return O1_ERR_ARG;
    if (!scratch || (uintptr_t)scratch % 256 || scratch_bytes < o1_pg_scratch_bytes(&g, rows)) return O1_ERR_ARG;
    const int nh = g.groups * g.heads_per_group;
    const O1Span o = o1_row_span(out, g.dtype, nh, g.dv, os, rows), x = o1_row_span(q, g.dtype, nh, g.d, qs, rows),
                 sc = o1_span(scratch, scratch_bytes);
    if (!o1_rows_ok(o) || !o1_rows_ok(x)) return O1_ERR_ARG;
    for (const O1Span &w : {o, sc})   // what is written, against everything else
        if (meets(sp, w) || o1_spans_overlap(w, x) || o1_spans_overlap(w, slots) || o1_spans_overlap(w, pos)) return O1_ERR_ARG;
    if (o1_spans_overlap(o, sc)) return O1_ERR_ARG;
    fill(a, g, *cache);
    a.q = q; a.out = out; a.qs = (size_t)qs; a.os = (size_t)os;
    a.part = (float *)scratch;
    return O1_OK;
}

}  // namespace

extern "C" {

int o1_pg_write(const o1_pg_geom *geom, const o1_pg_cache *cache, const void *k, int64_t k_stride, const void *v,
                int64_t v_stride, const o1_pg_seq *seqs, int32_t n_seq, int32_t total_rows, void *stream) {
    return copy_seqs(geom, cache, k, k_stride, v, v_stride, seqs, n_seq, total_rows, true, (cudaStream_t)stream);
}

int o1_pg_read(const o1_pg_geom *geom, const o1_pg_cache *cache, const o1_pg_seq *seqs, int32_t n_seq, void *k,
               int64_t k_stride, void *v, int64_t v_stride, int32_t total_rows, void *stream) {
    return copy_seqs(geom, cache, k, k_stride, v, v_stride, seqs, n_seq, total_rows, false, (cudaStream_t)stream);
}

int o1_pg_token_write(const o1_pg_geom *geom, const o1_pg_cache *cache, const void *k, int64_t k_stride, const void *v,
                      int64_t v_stride, const int32_t *slots, const int64_t *pos, int32_t rows, void *stream) {
    if (!pg_geom_ok(geom)) return O1_ERR_UNSUPPORTED;
    const o1_pg_geom &g = *geom;
    PgSpans sp;
    if (!cache_ok(g, cache, sp) || !apart(sp)) return O1_ERR_ARG;
    if (rows < 0 || rows > 65536 || (uintptr_t)slots % 4 || (uintptr_t)pos % 8) return O1_ERR_ARG;
    if (rows == 0) return O1_OK;
    if (!pos || (!slots && rows > cache->n_slots)) return O1_ERR_ARG;
    const O1Span kk = o1_row_span(k, g.dtype, g.groups, g.d, k_stride, rows),
                 vv = o1_row_span(v, g.dtype, g.groups, g.dv, v_stride, rows);
    if (!o1_rows_ok(kk) || !o1_rows_ok(vv)) return O1_ERR_ARG;
    for (const O1Span &x : {kk, vv, o1_span(slots, (size_t)rows * 4), o1_span(pos, (size_t)rows * 8)})
        if (meets(sp, x)) return O1_ERR_ARG;
    PgArgs a;
    fill(a, g, *cache);
    a.k_in = k; a.v_in = v;
    a.ks = (size_t)k_stride; a.vs = (size_t)v_stride;
    a.slots = slots; a.pos = pos; a.rows = rows;
    copy_launch<true>(a, g.dtype, g.cache_dtype, nullptr, (cudaStream_t)stream);
    return cudaGetLastError() == cudaSuccess ? O1_OK : O1_ERR_CUDA;
}

size_t o1_pg_scratch_bytes(const o1_pg_geom *geom, int32_t rows) {
    if (!pg_geom_ok(geom) || rows < 1) return 0;
    return std::max(pg_rows_scratch(geom->dv), pg_tc_scratch(*geom, (int64_t)rows * geom->heads_per_group));
}

int o1_pg_chunk_attend(const o1_pg_geom *geom, const o1_pg_cache *cache, void *scratch, size_t scratch_bytes,
                       const void *q, int64_t q_stride, const o1_pg_seq *seqs, int32_t n_seq, void *out,
                       int64_t out_stride, int32_t total_rows, void *stream) {
    if (!pg_geom_ok(geom)) return O1_ERR_UNSUPPORTED;
    const o1_pg_geom &g = *geom;
    PgSpans sp;
    if (!cache_ok(g, cache, sp)) return O1_ERR_ARG;
    if (n_seq < 0 || n_seq > PG_MAX_SEQ || total_rows < 0) return O1_ERR_ARG;
    if (n_seq == 0) return O1_OK;
    if (!seqs || !seqs_ok(seqs, n_seq, g, *cache, total_rows, false)) return O1_ERR_ARG;
    if (total_rows == 0) return O1_OK;
    PgArgs a;
    const int rc = attend_args(a, g, cache, scratch, scratch_bytes, q, q_stride, out, out_stride, total_rows,
                               o1_span(nullptr, 0), o1_span(nullptr, 0));
    if (rc != O1_OK) return rc;
    // One kernel for all the sequences: the one for few vectors where a group's
    // fit into its units of 16, the tensor cores' where they do not. 32 sequences
    // behind 2000 positions, 4 groups of 4 heads of 128: of 4 rows 44 us with
    // either (bf16; fp32: 49 with the first and 66 with the second, bf16 over e4m3:
    // 37 and 48), of 5 rows 57 and 45 (72 and 66, 53 and 48), of 16 96 and 46 (124
    // and 68, 90 and 48). Rows of 256 the tensor cores' has earlier (4 rows: 69 and
    // 60), fp16 over e4m3, with two terms, later (5 rows: 53 and 65, 16: 90 and 67).
    int64_t most = 0;
    for (int i = 0; i < n_seq; ++i) most = std::max(most, (int64_t)seqs[i].rows * g.heads_per_group);
    if (most >= INT32_MAX - 511) return O1_ERR_ARG;   // vectors are counted in 32 bits
    const int tc = most > PG_ROWS_V ? pg_tc_vectors(g) : 0, unit = tc ? tc : PG_ROWS_V;
    cudaStream_t st = (cudaStream_t)stream;
    bool ok = true;
    for_tables(seqs, n_seq, [&](int rows) { return ((int64_t)rows * g.heads_per_group + unit - 1) / unit; }, [&](const PgTable &t) {
        const cudaError_t e = tc ? pg_launch_tc(a, g, t, (int64_t)total_rows * g.heads_per_group, st)
                                 : pg_launch_rows(a, g.dtype, g.cache_dtype, &t, st);
        ok = ok && e == cudaSuccess;
    });
    return ok ? O1_OK : O1_ERR_CUDA;
}

int o1_pg_token_attend(const o1_pg_geom *geom, const o1_pg_cache *cache, void *scratch, size_t scratch_bytes,
                       const void *q, int64_t q_stride, const int32_t *slots, const int64_t *pos, void *out,
                       int64_t out_stride, int32_t rows, void *stream) {
    if (!pg_geom_ok(geom)) return O1_ERR_UNSUPPORTED;
    const o1_pg_geom &g = *geom;
    PgSpans sp;
    if (!cache_ok(g, cache, sp)) return O1_ERR_ARG;
    if (rows < 0 || rows > 65536 || (uintptr_t)slots % 4 || (uintptr_t)pos % 8) return O1_ERR_ARG;
    if (rows == 0) return O1_OK;
    if (!pos || (!slots && rows > cache->n_slots)) return O1_ERR_ARG;
    PgArgs a;
    const int rc = attend_args(a, g, cache, scratch, scratch_bytes, q, q_stride, out, out_stride, rows,
                               o1_span(slots, (size_t)rows * 4), o1_span(pos, (size_t)rows * 8));
    if (rc != O1_OK) return rc;
    a.slots = slots; a.pos = pos; a.rows = rows;
    return pg_launch_rows(a, g.dtype, g.cache_dtype, nullptr, (cudaStream_t)stream) == cudaSuccess ? O1_OK : O1_ERR_CUDA;
}

int o1_pg_flags(uint32_t *flags, int32_t clear, void *stream) {
    if (!flags) return O1_ERR_ARG;
    return pg_flags(flags, clear, (cudaStream_t)stream);
}

}  // extern "C"
