// Linear attention with a decay per head: the row kernel (token batches,
// short sequences) and the C ABI of the linear layer. Per head h and row t
//   S = e^{g_h} S + k_t v_t^T,   out_t = scale q_t S.
#include <limits.h>
#include <math.h>

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
// Bound: HBM, by the state (8 d dv bytes a head and step). The columns
// of a CTA are chosen by the launcher so that a batch of one still spreads
// over the SMs.
template <typename T, int NI>
__device__ __forceinline__ void lin_rows(const LinArgs &a, int slot, int row0, int rows, int h, int col0) {
    __shared__ float4 red[2][ROW_THREADS / 32][32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int vl = a.cols >> 2;                      // lanes along the columns (a power of two, <= 32)
    const int c = tid & (vl - 1), dg = tid / vl, DG = ROW_THREADS / vl;
    const int col = col0 + 4 * c;
    const bool in = col < a.dv;
    const int g = h / a.hpg;
    // One step's decay as near + dec: 0 + e^g, or 1 + (e^g - 1) for slow
    // decays. e^g rounded to fp32 is off by up to 2^-25 every step, the same
    // way each time; over the 1 / |g| steps a slow state remembers that adds
    // up to 2^-25 / |g|, while expm1f's error is 2^-24 |g| a step.
    const float gd = a.decay[h];
    const float near = gd > -0.35f ? 1.f : 0.f, dec = gd > -0.35f ? expm1f(gd) : expf(gd);
    float *S = a.state + ((size_t)slot * a.nh + h) * a.d * a.dv;
    const T *q = (const T *)a.q + (size_t)row0 * a.qs + (size_t)h * a.d;
    const T *k = (const T *)a.k + (size_t)row0 * a.ks + (size_t)g * a.d;
    const T *v = (const T *)a.v + (size_t)row0 * a.vs + (size_t)g * a.dv;
    T *o = (T *)a.out + (size_t)row0 * a.os + (size_t)h * a.dv;
    float4 s[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int di = dg + DG * i;
        s[i] = in && di < a.d ? *(const float4 *)(S + (size_t)di * a.dv + col) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int r = 0; r < rows; ++r) {
        const float4 vv = in ? o1_ld4(v + (size_t)r * a.vs + col) : make_float4(0.f, 0.f, 0.f, 0.f);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int di = dg + DG * i;
            const float kk = di < a.d ? o1_ld1(k + (size_t)r * a.ks + di) : 0.f;
            const float qq = di < a.d ? o1_ld1(q + (size_t)r * a.qs + di) : 0.f;
            s[i].x = fmaf(s[i].x, near, fmaf(s[i].x, dec, kk * vv.x));
            s[i].y = fmaf(s[i].y, near, fmaf(s[i].y, dec, kk * vv.y));
            s[i].z = fmaf(s[i].z, near, fmaf(s[i].z, dec, kk * vv.z));
            s[i].w = fmaf(s[i].w, near, fmaf(s[i].w, dec, kk * vv.w));
            acc.x = fmaf(qq, s[i].x, acc.x);
            acc.y = fmaf(qq, s[i].y, acc.y);
            acc.z = fmaf(qq, s[i].z, acc.z);
            acc.w = fmaf(qq, s[i].w, acc.w);
        }
        for (int m = vl; m < 32; m <<= 1) {
            acc.x += __shfl_xor_sync(0xffffffffu, acc.x, m);
            acc.y += __shfl_xor_sync(0xffffffffu, acc.y, m);
            acc.z += __shfl_xor_sync(0xffffffffu, acc.z, m);
            acc.w += __shfl_xor_sync(0xffffffffu, acc.w, m);
        }
        // two buffers: row r + 2 writes this one after the barrier of row
        // r + 1, which its readers reach only when done
        if (lane < vl) red[r & 1][warp][lane] = acc;
        __syncthreads();
        if (tid < vl && in) {
            float4 t = red[r & 1][0][tid];
#pragma unroll
            for (int w = 1; w < ROW_THREADS / 32; ++w) {
                const float4 x = red[r & 1][w][tid];
                t.x += x.x;
                t.y += x.y;
                t.z += x.z;
                t.w += x.w;
            }
            o1_st4(o + (size_t)r * a.os + col,
                   make_float4(t.x * a.scale, t.y * a.scale, t.z * a.scale, t.w * a.scale));
        }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int di = dg + DG * i;
        if (in && di < a.d) *(float4 *)(S + (size_t)di * a.dv + col) = s[i];
    }
}

// Token batch: row r on slot slots[r]. A row whose slot an earlier row names
// is padding (two CTAs on one state would race), so every CTA looks through
// the earlier rows' slots.
template <typename T, int NI>
__global__ __launch_bounds__(ROW_THREADS) void k_lin_token(LinArgs a) {
    const int ns = (a.dv + a.cols - 1) / a.cols;
    const int r = blockIdx.x / ns, col0 = (blockIdx.x - r * ns) * a.cols;
    const int slot = a.slots ? a.slots[r] : r;
    if (slot < 0 || slot >= a.nslots) return;
    if (a.slots) {
        int dup = 0;
        for (int i = threadIdx.x; i < r; i += ROW_THREADS) dup |= a.slots[i] == slot;
        if (__syncthreads_or(dup)) return;
    }
    lin_rows<T, NI>(a, slot, r, 1, blockIdx.y, col0);
}

// Sequences of a table, a few rows each.
template <typename T, int NI>
__global__ __launch_bounds__(ROW_THREADS) void k_lin_rows(LinArgs a, const __grid_constant__ LinTable t) {
    const int ns = (a.dv + a.cols - 1) / a.cols;
    const int i = blockIdx.x / ns, col0 = (blockIdx.x - i * ns) * a.cols;
    lin_rows<T, NI>(a, t.s[i].slot, t.s[i].row0, t.s[i].rows, blockIdx.y, col0);
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

// Sequences of up to LIN_ROW_MAX rows take the row kernel, longer ones the
// chunk kernels.
constexpr int LIN_ROW_MAX = 32;
// Limits of a pass: its states are written, read, rewritten and read again and
// are kept to what stays in the L2 (a 32768-row prompt of 2 MB a state: 412 us
// in passes of 64 MB, 469 of 96, 472 of 128); its scratch as a whole, and its
// rows, so that counts fit 32 bits.
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
// tiles of the segment: a 4096-row fp32 prompt of 8 heads of 256 took 141 us
// with 256 rows, 152 with 128, 178 with 512. A call that does not fill the SMs
// is bound by the longest chain instead: 1077 fp16 rows of 3 heads 19.7 us with
// 128 rows, 22.1 with 256.
int seg_rows(int64_t tiles) { return tiles <= LIN_SMS ? LIN_CHUNK : 2 * LIN_CHUNK; }

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
    if (!state || (uintptr_t)state % 16 || n_slots < 1 || !log_decay || (uintptr_t)log_decay % 4) return O1_ERR_ARG;
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
    if (!lin_geom_ok(geom) || slots < 1) return 0;
    return slot_floats(*geom) * slots * 4;
}

size_t o1_lin_scratch_bytes(const o1_lin_geom *geom, int32_t rows, int32_t seqs) {
    if (!lin_geom_ok(geom) || rows < 1 || seqs < 1) return 0;
    // segments of LIN_CHUNK rows are the most states any split into segments takes
    const size_t all = lin_pass_bytes(*geom, (int64_t)rows / LIN_CHUNK + seqs, (int64_t)rows + 16 * (int64_t)seqs);
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
    int64_t tiles_all = 0;
    for (int i = 0; i < n_seq; ++i)
        if (seqs[i].rows > LIN_ROW_MAX) tiles_all += (seqs[i].rows - 1) / LIN_CHUNK + 1;
    a.seg = seg_rows(tiles_all * a.nh * ((g.dv + 127) / 128));
    LinTable rows;
    LinWorkTable work;
    int n = 0, segs = 0, tiles = 0, prows = 0;
    bool launched = true;
    work.n = 0;
    auto flush_rows = [&]() {
        if (n) rows_launch(a, g.dtype, &rows, n, st);
        n = 0;
    };
    auto flush_chunks = [&]() {
        if (work.n && !lin_launch_pass(a, g.dtype, work, segs, tiles, prows, scratch, st)) launched = false;
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
        if (s.rows <= LIN_ROW_MAX) {
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
