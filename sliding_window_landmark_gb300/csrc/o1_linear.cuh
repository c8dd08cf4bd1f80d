// Internals of the linear layer (linear attention with a decay per head):
// the argument block of its kernels and the launchers.
#pragma once

#include "o1_rows.cuh"

// Sequences of one launch, passed by value.
#define LIN_TABLE 128
struct LinTable {
    o1_lin_seq s[LIN_TABLE];
};

// Rows of a tile of the chunk kernels.
#define LIN_CHUNK 128
// Rows of a segment at most: two tiles (k_lin_out weights the scores against
// one earlier tile).
#define LIN_SEG (2 * LIN_CHUNK)
// CTAs of their persistent grids: one an SM.
#define LIN_SMS 152
// A piece of a sequence in a pass of the chunk kernels: its rows in segments
// of LinArgs::seg (LIN_CHUNK or LIN_SEG), on the scratch's states seg0,
// seg0 + 1, ..., in tiles tile0, tile0 + 1, ... of LIN_CHUNK rows, and, for
// types that are split, in the panels' rows from prow0 on (a multiple of 16).
struct LinWork {
    int32_t row0, rows, slot, seg0, tile0, prow0;
};
struct LinWorkTable {
    int32_t n;
    LinWork w[LIN_TABLE];
};

struct LinArgs {
    float *state;              // [slots][nh][d][dv]
    const void *q, *k, *v;
    void *out;
    size_t qs, ks, vs, os;     // row strides, elements
    const float *decay;        // [nh] log decay
    const int *slots;          // token batches: slot of each row, or null
    int rows;                  // of the row tensors
    int nslots, G, hpg, nh, d, dv;
    float scale;
    int cols;                  // value columns of a CTA of the row kernel (a power of two)
    int seg;                   // rows of a segment of the chunk kernels
    long long wait_cycles;     // limit of the chunk kernels' waits (o1_set_wait_limit)
};

// e^{g n}, 1 at n = 0 whatever g (also -inf): the product g n keeps its
// rounding error as a second term, so that the power of a slow decay over
// many rows stays within a few roundings.
__device__ __forceinline__ float lin_pow(float g, int n) {
    if (n == 0) return 1.f;
    const float fn = (float)n;                        // exact below 2^24
    const float fl = (float)(n - (int)fn);
    const float x = __fmul_rn(g, fn);
    if (x <= -150.f) return 0.f;                      // below the smallest fp32 value
    const float e = fmaf(g, fn, -x) + g * fl;
    const float y = expf(x);
    return fmaf(y, e, y);
}

// Scratch of a pass: per segment, the increments (fp32, overwritten by two bf16
// terms of the entering states) and, for fp32, their third terms; then, for
// types of more than one bf16 term, the rows' term panels (per row).
static inline int lin_terms(int dtype) { return dtype == O1_BF16 ? 1 : dtype == O1_F16 ? 2 : 3; }
struct LinStates {
    size_t inc, third;
};
static inline LinStates lin_pass_states(int nh, int d, int dv, int dtype, int64_t segs) {
    const size_t n = (size_t)segs * nh * d * dv;
    return {o1_al256(4 * n), dtype == O1_F32 ? o1_al256(2 * n) : 0};
}
static inline size_t lin_pass_bytes(const o1_lin_geom &g, int64_t segs, int64_t prows) {
    const int nt = lin_terms(g.dtype), nh = g.groups * g.heads_per_group;
    const LinStates s = lin_pass_states(nh, g.d, g.dv, g.dtype, segs);
    const size_t row = (size_t)(nh + g.groups) * g.d + (size_t)g.groups * g.dv;
    return s.inc + s.third + (nt > 1 ? o1_al256((size_t)prows * row * 2 * nt) : 0);
}

// One pass of the chunk kernels (o1_linear_tc.cu) over the pieces of a table:
// `segs` segments, `tiles` tiles and `prows` panel rows in all, in a scratch of
// lin_pass_bytes. Launches only; false where a tensor map cannot be made.
// first: no kernel of this call stands before it in the stream.
bool lin_launch_pass(const LinArgs &a, int dtype, const LinWorkTable &t, int segs, int tiles, int prows, void *scratch,
                     bool first, cudaStream_t st);
// Flags its kernels raised on the current device (O1_FLAG_WAIT_EXPIRED), and
// their reset.
int lin_flags(uint32_t *flags, int clear, cudaStream_t st);
