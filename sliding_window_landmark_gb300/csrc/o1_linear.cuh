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
// CTAs of their persistent grids: one an SM.
#define LIN_SMS 152
// A piece of a sequence in a pass of the chunk kernels: its rows in segments
// of LinArgs::seg (a multiple of LIN_CHUNK), on the scratch's states seg0,
// seg0 + 1, ..., and in tiles tile0, tile0 + 1, ... of LIN_CHUNK rows.
struct LinWork {
    int32_t row0, rows, slot, seg0, tile0;
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

// One pass of the chunk kernels (o1_linear_tc.cu) over the pieces of a table,
// `segs` segments and `tiles` tiles in all; inc: [segs][nh][d][dv] fp32
// scratch. Launches only; false where a tensor map cannot be made.
bool lin_launch_pass(const LinArgs &a, int dtype, const LinWorkTable &t, int segs, int tiles, float *inc,
                     cudaStream_t st);
// Flags its kernels raised on the current device (O1_FLAG_WAIT_EXPIRED), and
// their reset.
int lin_flags(uint32_t *flags, int clear, cudaStream_t st);
