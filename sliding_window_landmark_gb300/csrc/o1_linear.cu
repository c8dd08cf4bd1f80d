// Linear attention with a decay per head: the row kernel (token batches,
// short sequences) and the C ABI of the linear layer. Per head h and row t
//   S = e^{g_h} S + k_t v_t^T,   out_t = scale q_t S.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "o1_linear.cuh"

namespace {

constexpr int ROW_THREADS = 256;

// The recurrence as it stands, one CTA per (sequence, head, slice of value
// columns). Thread (c, dg) holds value columns 4c .. 4c + 3 of every DG-th
// state row from dg on in registers, so the state is read once, advanced over
// the sequence's rows, and written once. A row's output is a sum over the
// state rows: lanes by shuffles, warps through shared memory.
//
// One step's decay is near + dec: 0 + e^g, or 1 + (e^g - 1) for slow decays.
// e^g rounded to fp32 is off by up to 2^-25 every step, the same way each
// time; over the 1 / |g| steps a slow state remembers that adds up to
// 2^-25 / |g|, while expm1f's error is 2^-24 |g| a step.
struct RowThread {
    int c, dg, DG, vl, col;   // column group, first state row, their step, lanes along the columns, column
    bool in;
    float near, dec;
    __device__ __forceinline__ RowThread(const LinArgs &a, int h, int col0) {
        vl = a.cols >> 2;   // a power of two, at most 32
        c = threadIdx.x & (vl - 1);
        dg = threadIdx.x / vl;
        DG = ROW_THREADS / vl;
        col = col0 + 4 * c;
        in = col < a.dv;
        const float g = a.decay[h];
        near = g > -0.35f ? 1.f : 0.f;
        dec = g > -0.35f ? expm1f(g) : expf(g);
    }
    __device__ __forceinline__ void step(float4 &s, float4 &acc, float k, float q, const float4 &v) const {
        s.x = fmaf(s.x, near, fmaf(s.x, dec, k * v.x));
        s.y = fmaf(s.y, near, fmaf(s.y, dec, k * v.y));
        s.z = fmaf(s.z, near, fmaf(s.z, dec, k * v.z));
        s.w = fmaf(s.w, near, fmaf(s.w, dec, k * v.w));
        acc.x = fmaf(q, s.x, acc.x);
        acc.y = fmaf(q, s.y, acc.y);
        acc.z = fmaf(q, s.z, acc.z);
        acc.w = fmaf(q, s.w, acc.w);
    }
    // the block's sum over the state rows, at the threads below vl; `red`
    // holds one row, read before the barrier of the next row on it
    __device__ __forceinline__ float4 sum(float4 acc, float4 (*red)[32]) const {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        for (int m = vl; m < 32; m <<= 1) {
            acc.x += __shfl_xor_sync(0xffffffffu, acc.x, m);
            acc.y += __shfl_xor_sync(0xffffffffu, acc.y, m);
            acc.z += __shfl_xor_sync(0xffffffffu, acc.z, m);
            acc.w += __shfl_xor_sync(0xffffffffu, acc.w, m);
        }
        if (lane < vl) red[warp][lane] = acc;
        __syncthreads();
        if (threadIdx.x < vl) {
            acc = red[0][threadIdx.x];
#pragma unroll
            for (int w = 1; w < ROW_THREADS / 32; ++w) {
                const float4 x = red[w][threadIdx.x];
                acc.x += x.x;
                acc.y += x.y;
                acc.z += x.z;
                acc.w += x.w;
            }
        }
        return acc;
    }
};
__device__ __forceinline__ float4 scaled(float4 x, float f) { return make_float4(x.x * f, x.y * f, x.z * f, x.w * f); }

// Token batch: row r on slot slots[r]. A row whose slot an earlier row names
// is padding (two CTAs on one state would race), so every CTA looks through
// the earlier rows' slots, under the state's loads: 1024 bf16 rows of 16 heads
// of 64 take 110 us, 103 without slots; 4096 of 16 heads of 128 1421 and 1264;
// 65536 fp32 rows of one head of 64 754 and 375. The state goes back before
// the output's sum. Bound: HBM, by the state (8 d dv bytes a head and step).
template <typename T, int NI>
__global__ __launch_bounds__(ROW_THREADS, 3) void k_lin_token(LinArgs a) {
    __shared__ float4 red[ROW_THREADS / 32][32];
    __shared__ float sq[O1_MAX_D], sk[O1_MAX_D];
    const int ns = (a.dv + a.cols - 1) / a.cols, h = blockIdx.y, g = h / a.hpg;
    const int r = blockIdx.x / ns, col0 = (blockIdx.x - r * ns) * a.cols;
    const int slot = a.slots ? a.slots[r] : r;
    if (slot < 0 || slot >= a.nslots) return;
    const RowThread t(a, h, col0);
    float *S = a.state + ((size_t)slot * a.nh + h) * a.d * a.dv + t.col;
    float4 s[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int di = t.dg + t.DG * i;
        s[i] = t.in && di < a.d ? *(const float4 *)(S + (size_t)di * a.dv) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const T *q = (const T *)a.q + (size_t)r * a.qs + (size_t)h * a.d;
    const T *k = (const T *)a.k + (size_t)r * a.ks + (size_t)g * a.d;
    const T *v = (const T *)a.v + (size_t)r * a.vs + (size_t)g * a.dv;
    const float4 vv = t.in ? o1_ld4(v + t.col) : make_float4(0.f, 0.f, 0.f, 0.f);
    if (threadIdx.x < a.d) {
        sq[threadIdx.x] = o1_ld1(q + threadIdx.x);
        sk[threadIdx.x] = o1_ld1(k + threadIdx.x);
    }
    int dup = 0;
    if (a.slots)
        for (int i = threadIdx.x; i < r; i += ROW_THREADS) dup |= a.slots[i] == slot;
    if (__syncthreads_or(dup)) return;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int di = t.dg + t.DG * i;
        if (di >= a.d) break;
        t.step(s[i], acc, sk[di], sq[di], vv);
        if (t.in) *(float4 *)(S + (size_t)di * a.dv) = s[i];
    }
    acc = t.sum(acc, red);
    if (threadIdx.x < t.vl && t.in)
        o1_st4((T *)a.out + (size_t)r * a.os + (size_t)h * a.dv + t.col, scaled(acc, a.scale));
}

// Sequences of a table, a few rows each. ROW_STEP rows of q, k and v at a time
// come into shared memory: loaded row by row, a row took the memory's latency
// (0.9 us).
constexpr int ROW_STEP = 16;
template <typename T, int NI>
__global__ __launch_bounds__(ROW_THREADS) void k_lin_rows(LinArgs a, const __grid_constant__ LinTable tab) {
    __shared__ float4 red[2][ROW_THREADS / 32][32];
    __shared__ float sq[ROW_STEP][O1_MAX_D], sk[ROW_STEP][O1_MAX_D];
    const int ns = (a.dv + a.cols - 1) / a.cols, h = blockIdx.y, g = h / a.hpg, tid = threadIdx.x;
    const int n = blockIdx.x / ns, col0 = (blockIdx.x - n * ns) * a.cols;
    const o1_lin_seq seq = tab.s[n];
    const RowThread t(a, h, col0);
    float *S = a.state + ((size_t)seq.slot * a.nh + h) * a.d * a.dv + t.col;
    const T *q = (const T *)a.q + (size_t)seq.row0 * a.qs + (size_t)h * a.d;
    const T *k = (const T *)a.k + (size_t)seq.row0 * a.ks + (size_t)g * a.d;
    const T *v = (const T *)a.v + (size_t)seq.row0 * a.vs + (size_t)g * a.dv + t.col;
    T *o = (T *)a.out + (size_t)seq.row0 * a.os + (size_t)h * a.dv + t.col;
    float4 s[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int di = t.dg + t.DG * i;
        s[i] = t.in && di < a.d ? *(const float4 *)(S + (size_t)di * a.dv) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int d4 = a.d / 4;
    for (int r0 = 0; r0 < seq.rows; r0 += ROW_STEP) {
        const int nr = min(ROW_STEP, seq.rows - r0);
        __syncthreads();
        for (int i = tid; i < nr * d4; i += ROW_THREADS) {
            const int r = i / d4, c = 4 * (i - r * d4);
            *(float4 *)&sq[r][c] = o1_ld4(q + (size_t)(r0 + r) * a.qs + c);
            *(float4 *)&sk[r][c] = o1_ld4(k + (size_t)(r0 + r) * a.ks + c);
        }
        __syncthreads();
        // values a few rows ahead of their use
        constexpr int AHEAD = 4;
        float4 vv[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            vv[j] = t.in && j < nr ? o1_ld4(v + (size_t)(r0 + j) * a.vs) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int r = 0; r < ROW_STEP; ++r) {
            if (r >= nr) break;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int di = t.dg + t.DG * i;
                const bool on = di < a.d;
                t.step(s[i], acc, on ? sk[r][on ? di : 0] : 0.f, on ? sq[r][on ? di : 0] : 0.f, vv[r % AHEAD]);
            }
            if (t.in && r + AHEAD < nr) vv[r % AHEAD] = o1_ld4(v + (size_t)(r0 + r + AHEAD) * a.vs);
            acc = t.sum(acc, red[r & 1]);
            if (tid < t.vl && t.in) o1_st4(o + (size_t)(r0 + r) * a.os, scaled(acc, a.scale));
        }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int di = t.dg + t.DG * i;
        if (t.in && di < a.d) *(float4 *)(S + (size_t)di * a.dv) = s[i];
    }
}

// Columns of a CTA: as many as fill a warp's width in memory, fewer while the
// grid has less than two CTAs an SM, and at most 8 registers of float4 a
// thread (cols * d <= 8 * 4 * 256).
int lin_cols(int d, int dv, long long seq_heads) {
    int cols = 8;
    while (cols < dv && cols < 128 && 2 * cols * d <= 8 * 4 * ROW_THREADS) cols *= 2;
    while (cols > 16 && seq_heads * ((dv + cols - 1) / cols) < 2 * 152) cols >>= 1;
    return cols;
}

template <typename T, int NI>
void rows_launch_ni(const LinArgs &a, const LinTable *t, int n, cudaStream_t st) {
    const dim3 grid((unsigned)(n * ((a.dv + a.cols - 1) / a.cols)), a.nh);
    if (t) k_lin_rows<T, NI><<<grid, ROW_THREADS, 0, st>>>(a, *t);
    else k_lin_token<T, NI><<<grid, ROW_THREADS, 0, st>>>(a);
}

template <typename T>
void rows_launch_t(const LinArgs &a, const LinTable *t, int n, cudaStream_t st) {
    const int DG = ROW_THREADS / (a.cols >> 2), ni = (a.d + DG - 1) / DG;
    if (ni <= 1) rows_launch_ni<T, 1>(a, t, n, st);
    else if (ni <= 2) rows_launch_ni<T, 2>(a, t, n, st);
    else if (ni <= 4) rows_launch_ni<T, 4>(a, t, n, st);
    else rows_launch_ni<T, 8>(a, t, n, st);
}

// One launch over the n sequences of a table, or the n rows of a token batch.
void rows_launch(LinArgs a, int dtype, const LinTable *t, int n, cudaStream_t st) {
    a.cols = lin_cols(a.d, a.dv, (long long)n * a.nh);
    if (dtype == O1_F32) rows_launch_t<float>(a, t, n, st);
    else if (dtype == O1_BF16) rows_launch_t<__nv_bfloat16>(a, t, n, st);
    else rows_launch_t<__half>(a, t, n, st);
}

bool lin_geom_ok(const o1_lin_geom *g) {
    if (!g) return false;
    if (g->groups < 1 || g->groups > 4096) return false;
    if (g->heads_per_group < 1 || g->heads_per_group > O1_MAX_HPG) return false;
    if (g->groups * g->heads_per_group > 65535) return false;   // heads are a grid's y
    if (g->d < 8 || g->d > O1_MAX_D || g->d % 8) return false;
    if (g->dv < 8 || g->dv > O1_MAX_DV || g->dv % 8) return false;
    return o1_dtype_ok(g->dtype) && isfinite(g->scale);
}

size_t slot_floats(const o1_lin_geom &g) {
    return (size_t)g.groups * g.heads_per_group * g.d * g.dv;
}

// Whether the states of that many slots have a size in bytes (64 bits).
bool slots_ok(const o1_lin_geom &g, int32_t slots) { return (size_t)slots <= SIZE_MAX / 4 / slot_floats(g); }

// Limits of a pass: its states are written, read, rewritten and read again and
// are kept to what stays in the L2; its scratch as a whole, and its rows, so
// that counts fit 32 bits. In passes of 32 / 48 / 64 / 96 / 128 MB of states a
// bf16 prompt of 32768 rows of 8 heads of 256 took 401 / 379 / 340 / 353 / 344
// us (fp16 647 / 622 / 562 / 580 / 571), of 16 heads of 128 253 / 238 / 218 /
// 232 / 218, 16384 rows of 64 heads of 128 with a key head each 548 / 517 / 475
// / 466 / 450; 16384 fp32 rows of 8 heads of 256 508 / 493 / 453 / 480 / 452.
constexpr size_t LIN_PASS_STATES = (size_t)64 << 20, LIN_PASS_BYTES = (size_t)256 << 20;
constexpr int64_t LIN_PASS_ROWS = 1 << 24;

// Whether a pass of that many segments and panel rows is within the limits
// (a single segment of one tile always is).
bool pass_within(const o1_lin_geom &g, int64_t segs, int64_t prows) {
    if (segs <= 1 && prows <= LIN_CHUNK) return true;
    return (size_t)segs * slot_floats(g) * 4 <= LIN_PASS_STATES && prows <= LIN_PASS_ROWS &&
           lin_pass_bytes(g, segs, prows) <= LIN_PASS_BYTES;
}

// Rows of a segment for a call of `tiles` tiles (LIN_CHUNK rows of a head, 128
// value columns). Longer segments write and read fewer states (4 d dv bytes a
// head each, several times over) and pay with scores against the earlier
// tiles of the segment. Prompts in us with 128 / 256 / 512 rows (512 from a
// build with any number of tiles a segment):
//                            bf16                fp16                fp32
//    4096, 8 heads of 256     58 /  49 /  58      88 /  82 / 101     132 / 128 / 161
//   32768, 8 heads of 256    461 / 340 / 343     697 / 564 / 617    1042 / 907 / 1069
//    4096, 16 heads of 128    41 /  37 /  45      61 /  58 /  72      92 /  92 / 116
//   32768, 16 heads of 128   273 / 217 / 231     422 / 375 / 430     644 / 633 / 737
//    4096, 64 heads of 128,  157 / 120 / 138     300 / 277 / 305     509 / 483 / 535
//   32768, a key head each  1250 / 947 / 962    2390 /2217 /2438    3946 /3795 /4221
// A call that does not fill the SMs is bound by the longest chain instead: 1077
// fp16 rows of 3 heads 19.7 us with 128 rows, 22.1 with 256 (before the scan
// took several rows a warp; 17.8 now).
int seg_rows(int64_t tiles) { return tiles <= LIN_SMS ? LIN_CHUNK : LIN_SEG; }

// Sequences of up to that many rows take the row kernel, longer ones the chunk
// kernels. Their times in us, E = nh d dv the elements of a sequence's states,
// from batches of 1 to 64 sequences of 1 to 32 rows alone and beside prompts of
// 100, 2047 and 4096 rows (16 heads of 128 bf16 and fp32, 8 of 256, 8 of 64):
//   row kernel    2.5, 0.36 a row of the longest sequence or 2.9e-7 E a row of
//                 them all, and the states' bytes, 1.2e-6 E a sequence
//   chunk kernels 14 (fp16 17, fp32 20) a pass, 5 + d / 32 (fp32 a third more)
//                 a further wave of tiles (of 128 rows, a head and 128 value
//                 columns), and 0.5 a MB of the pass's states once those
//                 outgrow the L2 (a quarter of that at half of 64 MB)
// so few short sequences beside a prompt go with its tiles, and many apart:
// 16 heads of 128, bf16, 2047 rows beside 4 of 16 rows 31 us as tiles and 39 by
// rows, beside 64 of 4 rows 114 and 67. fp16's waves are charged as bf16's: a
// third more sent 4 of 16 rows beside 2047 by rows, 49 us, where tiles take 41.
// A pass beyond the first is charged where what the limits and the scratch let
// into one does not fill the SMs: with a scratch of one state every short
// sequence among the tiles is a pass, 32 bf16 ones of 24 rows 96 launches.
// (Charged for all of them, 64 of 16 rows beside 32768 of 16 heads of 128 went
// by rows: bf16 318 us, 304 with the tiles.)
int row_max(const o1_lin_geom &g, const o1_lin_seq *s, int n, size_t scratch_bytes) {
    constexpr int TH = 6;
    const bool f32 = g.dtype == O1_F32;
    const int th[TH] = {0, 1, 4, 8, 16, lin_terms(g.dtype) == 1 ? 32 : 48};
    struct {
        int64_t seqs, rows, longest;
    } at[TH + 1] = {};   // of th[i - 1] + 1 .. th[i] rows; at[TH]: longer, in tiles
    for (int i = 0; i < n; ++i) {
        const int r = s[i].rows;
        int b = 0;
        while (b < TH && r > th[b]) ++b;
        at[b].seqs += b < TH ? 1 : (r - 1) / LIN_CHUNK + 1;
        at[b].rows += r;
        if (r > at[b].longest) at[b].longest = r;
    }
    const double E = (double)slot_floats(g), units = (double)(g.groups * g.heads_per_group) * ((g.dv + 127) / 128);
    const double fixed = f32 ? 20. : g.dtype == O1_F16 ? 17. : 14.;
    const double wave = (5. + g.d / 32.) * (f32 ? 1.33 : 1.);
    const double most = fmin((double)scratch_bytes, (double)LIN_PASS_BYTES);
    const double per_row = (double)lin_terms(g.dtype) * (lin_terms(g.dtype) > 1 ? 2. : 0.) *
                           ((double)(g.groups * g.heads_per_group + g.groups) * g.d + (double)g.groups * g.dv);
    const bool halves = at[TH].seqs * units > LIN_SMS;   // long sequences' segments are of two tiles
    int best = 0;
    double best_us = 0.;
    for (int t = 0; t < TH; ++t) {   // th[t] the longest by rows
        double seqs = 0., rows = 0., longest = 0., tiles = (double)at[TH].seqs, segs = halves ? tiles / 2 : tiles, us = 0.;
        double trows = (double)at[TH].rows;
        for (int b = 1; b < TH; ++b) {
            if (b <= t) {
                seqs += (double)at[b].seqs;
                rows += (double)at[b].rows;
                if (at[b].seqs) longest = (double)at[b].longest;
            } else {
                tiles += (double)at[b].seqs;
                segs += (double)at[b].seqs;
                trows += (double)at[b].rows;
            }
        }
        if (seqs) us += 2.5 + fmax(0.36 * longest, 2.9e-7 * E * rows) + 1.2e-6 * E * seqs;
        if (tiles) {
            const double state = (f32 ? 6. : 4.) * E;   // bytes of a segment, beside its panels
            const double hold = floor(fmin(LIN_PASS_STATES / (4. * E), most / (state + per_row * trows / segs)));
            const double passes = hold * units < LIN_SMS ? fmax(1., segs / fmax(1., hold)) : 1.;   // that do not fill the SMs
            const double mb = 1e-6 * state * segs, full = fmin(1., mb / passes / 64.);
            us += fixed * passes + fmax(0., ceil(units * tiles / LIN_SMS) - passes) * wave + 0.5 * mb * full * full;
        }
        if (t == 0 || us < best_us) best = th[t], best_us = us;
    }
    return best;
}
// The sequences of a call: ranges and slots in bounds and apart. Sorted
// copies on the stack (nothing is allocated for a call).
constexpr int LIN_MAX_SEQ = 4096;
bool seqs_ok(const o1_lin_seq *s, int n, int n_slots, int total_rows) {
    struct Range { int32_t row0, rows; } rng[LIN_MAX_SEQ];
    int32_t slot[LIN_MAX_SEQ];
    int nr = 0;
    for (int i = 0; i < n; ++i) {
        if (s[i].row0 < 0 || s[i].rows < 0 || s[i].slot < 0 || s[i].slot >= n_slots) return false;
        if ((int64_t)s[i].row0 + s[i].rows > total_rows) return false;
        slot[i] = s[i].slot;
        if (s[i].rows) rng[nr++] = {s[i].row0, s[i].rows};
    }
    std::sort(slot, slot + n);
    for (int i = 1; i < n; ++i)
        if (slot[i] == slot[i - 1]) return false;
    std::sort(rng, rng + nr, [](const Range &a, const Range &b) { return a.row0 < b.row0; });
    for (int i = 1; i < nr; ++i)
        if ((int64_t)rng[i - 1].row0 + rng[i - 1].rows > rng[i].row0) return false;
    return true;
}

// Shared argument checks of the two attend calls; fills the kernels' arguments.
int lin_args(LinArgs &a, float *state, int32_t n_slots, const o1_lin_geom &g, const void *q, int64_t q_stride,
             const void *k, int64_t k_stride, const void *v, int64_t v_stride, const float *log_decay, void *out,
             int64_t out_stride, int32_t rows, const O1Span &extra) {
    if (!state || (uintptr_t)state % 16 || n_slots < 1 || !slots_ok(g, n_slots) || !log_decay || (uintptr_t)log_decay % 4)
        return O1_ERR_ARG;
    const int nh = g.groups * g.heads_per_group;
    const O1Span sp[6] = {o1_row_span(out, g.dtype, nh, g.dv, out_stride, rows),
                          o1_span(state, slot_floats(g) * n_slots * 4),
                          o1_row_span(q, g.dtype, nh, g.d, q_stride, rows),
                          o1_row_span(k, g.dtype, g.groups, g.d, k_stride, rows),
                          o1_row_span(v, g.dtype, g.groups, g.dv, v_stride, rows),
                          o1_span(log_decay, (size_t)nh * 4)};
    for (int i = 0; i < 5; ++i)
        if (i != 1 && !o1_rows_ok(sp[i])) return O1_ERR_ARG;
    for (int i = 0; i < 2; ++i)   // what is written, against everything else
        for (int j = i + 1; j < 6; ++j)
            if (o1_spans_overlap(sp[i], sp[j])) return O1_ERR_ARG;
    for (const O1Span &x : sp)   // the scratch, or the slots of a token batch
        if (o1_spans_overlap(x, extra)) return O1_ERR_ARG;
    a = LinArgs();
    a.state = state;
    a.q = q; a.k = k; a.v = v; a.out = out;
    a.qs = (size_t)q_stride; a.ks = (size_t)k_stride; a.vs = (size_t)v_stride; a.os = (size_t)out_stride;
    a.decay = log_decay;
    a.rows = rows;
    a.nslots = n_slots;
    a.G = g.groups; a.hpg = g.heads_per_group; a.nh = nh; a.d = g.d; a.dv = g.dv;
    a.scale = g.scale;
    return O1_OK;
}

}  // namespace

extern "C" {

size_t o1_lin_state_bytes(const o1_lin_geom *geom, int32_t slots) {
    if (!lin_geom_ok(geom) || slots < 1 || !slots_ok(*geom, slots)) return 0;
    return slot_floats(*geom) * slots * 4;
}

size_t o1_lin_scratch_bytes(const o1_lin_geom *geom, int32_t rows, int32_t seqs) {
    if (!lin_geom_ok(geom) || rows < 1 || seqs < 1) return 0;
    // segments of LIN_CHUNK rows are the most states any split into segments
    // takes; a count past the limit of a pass is cut there, before it is
    // multiplied by a state (of at most 2^34 bytes)
    const int64_t segs = std::min((int64_t)rows / LIN_CHUNK + seqs, (int64_t)1 << 24);
    const size_t all = lin_pass_bytes(*geom, segs, (int64_t)rows + 16 * (int64_t)seqs);
    const size_t one = lin_pass_bytes(*geom, 1, LIN_CHUNK);
    size_t lim = lin_terms(geom->dtype) == 1 ? LIN_PASS_STATES : LIN_PASS_BYTES;
    lim = one > lim ? one : lim;
    return all < lim ? all : lim;
}

int o1_lin_chunk_attend(float *state, int32_t n_slots, const o1_lin_geom *geom, void *scratch, size_t scratch_bytes,
                        const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                        int64_t v_stride, const float *log_decay, const o1_lin_seq *seqs, int32_t n_seq, void *out,
                        int64_t out_stride, int32_t total_rows, void *stream) {
    if (!lin_geom_ok(geom)) return O1_ERR_UNSUPPORTED;
    const o1_lin_geom &g = *geom;
    if (n_seq < 0 || n_seq > LIN_MAX_SEQ || total_rows < 0) return O1_ERR_ARG;
    if (n_seq == 0) return O1_OK;
    if (!seqs || !seqs_ok(seqs, n_seq, n_slots, total_rows)) return O1_ERR_ARG;
    if (total_rows == 0) return O1_OK;
    if (!scratch || (uintptr_t)scratch % 256 || scratch_bytes < o1_lin_scratch_bytes(geom, 1, 1)) return O1_ERR_ARG;
    LinArgs a;
    const int rc = lin_args(a, state, n_slots, g, q, q_stride, k, k_stride, v, v_stride, log_decay, out, out_stride,
                            total_rows, o1_span(scratch, scratch_bytes));
    if (rc != O1_OK) return rc;
    cudaStream_t st = (cudaStream_t)stream;
    a.wait_cycles = o1_wait_limit();
    const int short_rows = row_max(g, seqs, n_seq, scratch_bytes);
    int64_t tiles_all = 0;
    for (int i = 0; i < n_seq; ++i)
        if (seqs[i].rows > short_rows) tiles_all += (seqs[i].rows - 1) / LIN_CHUNK + 1;
    a.seg = seg_rows(tiles_all * a.nh * ((g.dv + 127) / 128));
    LinTable rows;
    LinWorkTable work;
    int n = 0, segs = 0, tiles = 0, prows = 0;
    bool launched = true, first = true;
    work.n = 0;
    auto flush_rows = [&]() {
        if (n) rows_launch(a, g.dtype, &rows, n, st), first = false;
        n = 0;
    };
    auto flush_chunks = [&]() {
        if (work.n && !lin_launch_pass(a, g.dtype, work, segs, tiles, prows, scratch, first, st)) launched = false;
        first = first && !work.n;
        work.n = segs = tiles = prows = 0;
    };
    auto up = [](int64_t x, int m) { return (int)((x + m - 1) / m); };
    // whether the pass takes r more rows of a sequence
    auto fits = [&](int64_t r) {
        const int64_t p = prows + 16 * (int64_t)up(r, 16), n = segs + up(r, a.seg);
        return pass_within(g, n, p) && lin_pass_bytes(g, n, p) <= scratch_bytes;
    };
    for (int i = 0; i < n_seq; ++i) {
        const o1_lin_seq &s = seqs[i];
        if (s.rows == 0) continue;
        if (s.rows <= short_rows) {
            rows.s[n++] = s;
            if (n == LIN_TABLE) flush_rows();
            continue;
        }
        for (int off = 0; off < s.rows;) {
            // the rest of the sequence, or as many whole segments, tiles, or
            // (in an empty pass) steps of 16 rows as fit
            int take = s.rows - off;
            for (const int m : {a.seg, LIN_CHUNK, 16}) {
                if (work.n == LIN_TABLE) break;
                if (fits(take)) break;
                int lo = 0, hi = take / m;
                while (lo < hi) {
                    const int mid = lo + (hi - lo + 1) / 2;
                    if (fits((int64_t)mid * m)) lo = mid;
                    else hi = mid - 1;
                }
                take = lo * m;
                if (take || work.n) break;
                if (m != 16) take = s.rows - off;
            }
            if (!take || work.n == LIN_TABLE) {
                if (!work.n) return O1_ERR_ARG;   // not reached: the least scratch holds 16 rows
                flush_chunks();
                continue;
            }
            work.w[work.n++] = {s.row0 + off, take, s.slot, segs, tiles, prows};
            segs += up(take, a.seg);
            tiles += up(take, LIN_CHUNK);
            prows += 16 * up(take, 16);
            off += take;
        }
    }
    flush_rows();
    flush_chunks();
    return cudaGetLastError() == cudaSuccess && launched ? O1_OK : O1_ERR_CUDA;
}

int o1_lin_token_attend(float *state, int32_t n_slots, const o1_lin_geom *geom, const void *q, int64_t q_stride,
                        const void *k, int64_t k_stride, const void *v, int64_t v_stride, const float *log_decay,
                        const int32_t *slots, void *out, int64_t out_stride, int32_t rows, void *stream) {
    if (!lin_geom_ok(geom)) return O1_ERR_UNSUPPORTED;
    const o1_lin_geom &g = *geom;
    if (rows < 0 || rows > 65536 || (uintptr_t)slots % 4) return O1_ERR_ARG;
    if (rows == 0) return O1_OK;
    LinArgs a;
    const int rc = lin_args(a, state, n_slots, g, q, q_stride, k, k_stride, v, v_stride, log_decay, out, out_stride,
                            rows, o1_span(slots, (size_t)rows * 4));
    if (rc != O1_OK) return rc;
    if (!slots && rows > n_slots) return O1_ERR_ARG;
    a.slots = slots;
    rows_launch(a, g.dtype, nullptr, rows, (cudaStream_t)stream);
    return cudaGetLastError() == cudaSuccess ? O1_OK : O1_ERR_CUDA;
}

int o1_lin_flags(uint32_t *flags, int32_t clear, void *stream) {
    if (!flags) return O1_ERR_ARG;
    return lin_flags(flags, clear, (cudaStream_t)stream);
}

}  // extern "C"
