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

// Attention of a few rows a group (o1_page_rows.cu): launches over the rows of
// a token batch (tab null) or the sequences of a table, and the scratch it takes
// for calls of up to `vectors` query vectors a group.
cudaError_t pg_launch_rows(const PgArgs &a, int dtype, int cache_dtype, const PgTable *tab, bool first, cudaStream_t st);
size_t pg_rows_scratch(int dv, int groups, int64_t vectors);
