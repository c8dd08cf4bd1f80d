// Internals of the paged cache: the argument block of its kernels, the tables
// of a launch, and the launchers.
#pragma once

#include "o1_rows.cuh"

// Sequences of one launch, passed by value.
#define PG_TABLE 128
// A sequence of a launch; `before`: what the kernel counts its work by (rows
// for the copies, units of rows for the attention) in the sequences before it.
struct PgSeq {
    int32_t row0, rows, slot, pos0, before;
};
struct PgTable {
    int32_t n, total;   // sequences, and the sum of what is counted
    PgSeq s[PG_TABLE];
};

struct PgArgs {
    const void *q;        // row tensors, and their strides in elements
    const void *k_in, *v_in;
    void *out, *k_out, *v_out;
    size_t qs, os, ks, vs;
    void *k, *v;          // the cache
    uint8_t *ke, *ve;
    const int32_t *table;
    int n_pages, n_slots, width;
    const int32_t *slots; // token batches
    const int64_t *pos;
    int rows;
    int G, hpg, d, dv, lpage, window;   // lpage: log2 of the page's positions
    float scale;
    float *part;          // scratch of the attention
    long long wait_cycles;
};

static inline size_t pg_cache_bytes(int t) { return t == O1_E4M3 ? 1 : 2; }

// Pointer to head row (page, g, r) of a pool of `width` values a row; 64-bit
// offsets, as a pool may hold more than 2^31 values.
template <typename C>
__device__ __forceinline__ C *pg_at(C *pool, const PgArgs &a, int page, int g, int r, int width) {
    return pool + ((((size_t)page * a.G + g) << a.lpage) + r) * width;
}
// The page of position p of a slot, or -1: out of range, or absent.
__device__ __forceinline__ int pg_page(const PgArgs &a, int slot, int p) {
    const int id = a.table[(size_t)slot * a.width + (p >> a.lpage)];
    return id >= 0 && id < a.n_pages ? id : -1;
}
// 2^(byte - 127), bytes 1 to 254
__device__ __forceinline__ float pg_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// A row of a token batch: its slot and position, or slot -1 (padding).
struct PgRow {
    int slot, pos;
};
__device__ __forceinline__ PgRow pg_token_row(const PgArgs &a, int r) {
    const int slot = a.slots ? a.slots[r] : r;
    const int64_t p = a.pos[r];
    const bool ok = slot >= 0 && slot < a.n_slots && p >= 0 && p < ((int64_t)a.width << a.lpage);
    return {ok ? slot : -1, ok ? (int)p : 0};
}

// ---------------------------------------------------------------- attention
// Work, for both kernels (a plan P: constants V, K, START, LEAST). A unit is up
// to V query vectors of a sequence (vector i: row i / hpg of its rows, head i %
// hpg of a group) and a group; its keys are tiles of K positions, and it costs
// its tiles and START more (queries, filling the pipeline, outputs). The costs of
// all units, one behind the other, are split evenly over the blocks of one wave
// (fewer where a block would get less than LEAST), whatever the lengths; a unit
// whose tiles such a border cuts leaves partial results (maximum, sum, weighted
// values), which k_pg_join adds up.
struct PgUnit {
    int slot;      // -1: padding, no tiles
    int row0;      // first row of the sequence in the row tensors
    int pos0;      // its position
    int vec0, nv;  // first vector, and vectors
    int lo, hi;    // positions attended by some vector: lo .. hi
    int first, last;   // the same of all of the sequence's rows
    template <int K>
    __device__ __forceinline__ int tiles() const {
        return slot < 0 ? 0 : hi / K - lo / K + 1;
    }
    __device__ __forceinline__ int pos(const PgArgs &a, int v) const { return pos0 + (vec0 + v) / a.hpg; }   // of vector v
};
// Unit u of a table (counted by units in `before`), or row u of a token batch.
template <int V>
__device__ __forceinline__ PgUnit pg_unit(const PgArgs &a, const PgTable &tab, int u) {
    PgUnit x;
    if (a.pos) {
        const PgRow r = pg_token_row(a, u);
        x = {r.slot, u, r.pos, 0, a.hpg, 0, 0, 0, r.pos};
    } else {
        int n = 0;
        for (int hi = tab.n - 1; n < hi;) {
            const int mid = (n + hi + 1) >> 1;
            if (tab.s[mid].before <= u) n = mid;
            else hi = mid - 1;
        }
        x = {tab.s[n].slot, tab.s[n].row0, tab.s[n].pos0, (u - tab.s[n].before) * V, 0, 0, 0, 0, tab.s[n].pos0 + tab.s[n].rows - 1};
        x.nv = (int)min((int64_t)V, (int64_t)tab.s[n].rows * a.hpg - x.vec0);
    }
    x.hi = x.pos(a, x.nv - 1);
    x.lo = a.window ? max(0, x.pos(a, 0) - a.window + 1) : 0;
    x.first = a.window ? max(0, x.pos0 - a.window + 1) : 0;
    return x;
}

// A block's share: costs `at` to `to` of all, the next in unit u, whose groups
// begin at `start`.
struct PgShare {
    int64_t at, to, start, total;
    int u, blocks;   // blocks that get a share
    __device__ __forceinline__ int64_t border(int b) const { return total * b / blocks; }   // first cost of block b
};
// All threads of the block call it; shared: THREADS / 32 + 2 words.
template <typename P, int THREADS>
__device__ __forceinline__ PgShare pg_share(const PgArgs &a, const PgTable &tab, int units, long long *shared) {
    constexpr int W = THREADS / 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = (units + THREADS - 1) / THREADS, u0 = min(units, tid * per), u1 = min(units, u0 + per);
    auto cost = [&](int u) -> int64_t {
        const int n = pg_unit<P::V>(a, tab, u).template tiles<P::K>();
        return n ? (int64_t)(n + P::START) * a.G : 0;
    };
    long long own = 0;
    for (int u = u0; u < u1; ++u) own += cost(u);
    long long before = own;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, before, m);
        if (lane >= m) before += o;
    }
    if (lane == 31) shared[warp] = before;
    if (tid == 0) shared[W] = units, shared[W + 1] = 0;
    __syncthreads();
    long long total = 0, base = 0;
    for (int w = 0; w < W; ++w) {
        if (w < warp) base += shared[w];
        total += shared[w];
    }
    PgShare s;
    s.total = total;
    s.blocks = (int)min((long long)gridDim.x, max(1ll, total / P::LEAST));
    s.at = (int)blockIdx.x < s.blocks ? s.border(blockIdx.x) : 0;
    s.to = (int)blockIdx.x < s.blocks ? s.border(blockIdx.x + 1) : 0;
    before += base - own;   // costs before this thread's units
    if (s.at < s.to && s.at >= before && s.at < before + own) {
        int u = u0;
        for (; u + 1 < u1; ++u) {
            const int64_t n = cost(u);
            if (s.at < before + n) break;
            before += n;
        }
        shared[W] = u;
        shared[W + 1] = before;
    }
    __syncthreads();
    s.u = (int)shared[W];
    s.start = shared[W + 1];
    return s;
}
// The next segment of a share: tiles t0 .. t1 - 1 of unit u and group g, nt in
// all; `start`, the cost where the unit begins.
struct PgSegment {
    int u, g, t0, t1, nt;
    int64_t start;
    PgUnit x;
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == nt; }
    // where its partial result goes: a segment that begins inside its unit is
    // its block's first, one that only ends inside it the block's last
    __device__ __forceinline__ int part() const { return blockIdx.x * 2 + (t0 > 0 ? 0 : 1); }
};
template <typename P>
__device__ __forceinline__ bool pg_next(const PgArgs &a, const PgTable &tab, int units, PgShare &s, PgSegment &o) {
    while (s.at < s.to && s.u < units) {
        o.x = pg_unit<P::V>(a, tab, s.u);
        o.nt = o.x.template tiles<P::K>();
        const int64_t each = o.nt ? o.nt + P::START : 0, end = s.start + each * a.G;
        if (s.at >= end) {   // no tiles, or all of its groups done
            ++s.u;
            s.start = end;
            continue;
        }
        o.u = s.u;
        o.g = (int)((s.at - s.start) / each);
        o.start = s.start + o.g * each;
        const int64_t to = min(s.to, o.start + each);
        o.t0 = (int)max((int64_t)0, s.at - o.start - P::START);
        o.t1 = (int)max((int64_t)0, to - o.start - P::START);
        s.at = to;
        if (o.t0 < o.t1) return true;
    }
    return false;
}

// What a block leaves of the units that its borders cut: the values [dv / 4][V][4]
// (a warp's threads hold a vector each, and their 16 bytes lie in a row) and the
// statistics [V][2] (maximum in log2 units, sum) of its first segment and of its
// last, and in its header the first one's unit.
struct PgHead {
    int last;       // the last block with a part of the unit; -1: none begins its tiles in the block before
    int row0, vec0, nv, g;
    int pad[3];
};
struct PgParts {
    PgHead *head;
    float *stat, *val;
};
__host__ __device__ inline PgParts pg_parts(float *p, int blocks, int vecs) {
    return {(PgHead *)p, p + (size_t)blocks * 8, p + (size_t)blocks * 8 + (size_t)blocks * 2 * vecs * 2};
}
// Columns c .. c + 3 of vector v of partial result ps.
__device__ __forceinline__ float4 *pg_val(const PgParts &p, size_t ps, int vecs, int dv, int v, int c) {
    return (float4 *)p.val + (ps * (dv >> 2) + (c >> 2)) * vecs + v;
}
static inline size_t pg_parts_bytes(int blocks, int vecs, int dv) {
    return o1_al256(((size_t)blocks * 8 + (size_t)blocks * 2 * vecs * (2 + dv)) * 4);
}
// The header of a block whose first segment is s: it holds the unit where the
// block's own border is the first inside its tiles.
template <typename P>
__device__ __forceinline__ void pg_head(PgHead *head, const PgShare &sh, const PgSegment &s) {
    if (s.t0 == 0 || sh.border(blockIdx.x - 1) > s.start + P::START) return;
    const int64_t end = s.start + P::START + s.nt;   // last: border(last + 1) >= end
    *head = {(int)((end * sh.blocks + sh.total - 1) / sh.total) - 1, s.x.row0, s.x.vec0, s.x.nv, s.g, {0, 0, 0}};
}
// A unit's vector in the row tensors.
__device__ __forceinline__ size_t pg_vec_at(const PgArgs &a, int row0, int vec, int g, size_t stride, int width) {
    const int r = vec / a.hpg, h = g * a.hpg + (vec - r * a.hpg);
    return (size_t)(row0 + r) * stride + (size_t)h * width;
}

// A softmax's weights are taken from a reference, which moves to `below` under the
// row's maximum where that passes it by more than `above` (log2 units). Of weights
// held in fp16 a row's largest is at least 2^7 and at most 2^15: they have their
// 11 bits down to 2^-21 of the largest, and are off by 2^-32 of it below.
struct PgReference {
    float above, below;
    constexpr explicit PgReference(bool f16) : above(f16 ? 15.f : 8.f), below(f16 ? 7.f : 0.f) {}
};

// Launches over the rows of a token batch (tab null) or the sequences of a
// table, counted in units of the launched kernel's vectors.
// o1_page_rows.cu: few query vectors a group, any geometry.
constexpr int PG_ROWS_V = 16;
cudaError_t pg_launch_rows(const PgArgs &a, int dtype, int cache_dtype, const PgTable *tab, cudaStream_t st);
size_t pg_rows_scratch(int dv);
// The partial results of a launch of `blocks` blocks, joined (chained behind it):
// laid out for `room` blocks and `vecs` vectors, of which a unit has `most` at most.
cudaError_t pg_launch_join(const PgArgs &a, int dtype, int blocks, int room, int vecs, int most, cudaStream_t st);
// o1_page_tc.cu: many query vectors, on tcgen05. pg_tc_vectors: a unit's, 0
// where it does not take the geometry.
int pg_tc_vectors(const o1_pg_geom &g);
size_t pg_tc_scratch(const o1_pg_geom &g, int64_t vectors);
cudaError_t pg_launch_tc(const PgArgs &a, const o1_pg_geom &g, const PgTable &tab, int64_t vectors, cudaStream_t st);
int pg_flags(uint32_t *flags, int clear, cudaStream_t st);
