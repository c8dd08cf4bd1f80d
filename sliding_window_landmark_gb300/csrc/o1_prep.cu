// o1_head_prep: the norm of every query and key head and their rotation in
// one pass over the rows ("cortiq-engine 0.8.77 src/gpu_wgpu/dory.rs",
// dory_prep). Per head vector: sum of squares, one factor, the weight, the
// half-split rotation of its first `rot` values.
//
// Bound: HBM. Each value is read once and written once; the cosine and sine
// of a row's rot/2 angles are shared by all its heads, so a block takes
// whole rows and makes their table in shared memory first.
//
// Angles. p inv_j has to be known modulo 2 pi to fp32 accuracy for positions
// in the millions, and FP64 runs at a small fraction of the fp32 rate on this
// part. A turn is taken as 2^64: turns_j = inv_j / (2 pi) in fixed point (the
// 24-bit mantissa of inv_j times 1/(2 pi) to 128 bits, shifted), and
// p * turns_j modulo 2^64 is the angle's fraction of a turn, exact but for
// p / 2^64 turns of truncation. sincospif takes it from there.
#include <math.h>

#include "o1_rows.cuh"

namespace {

constexpr int PREP_THREADS = 256;
constexpr int PREP_ROWS = 4;   // rows of a block

struct PrepArgs {
    const void *q, *k;
    void *qo, *ko;
    const float *qw, *kw, *inv;
    const int64_t *pos;
    int64_t pos0;
    size_t qs, ks, qos, kos;   // row strides, elements
    int rows, hq, hk, d, rot, norm;
    float eps;
};

// inv / (2 pi) in units of 2^-64 turns, modulo one turn; 0 <= inv < 2^24.
// 1/(2 pi) = 0.159154943..., its first 128 binary digits:
__device__ __forceinline__ uint64_t turns_of(float inv) {
    const uint64_t c_hi = 0x28BE60DB9391054Aull, c_lo = 0x7F09D5F47D4D3770ull;
    const uint32_t bits = __float_as_uint(inv);
    const int e = (int)(bits >> 23) & 0xff;
    const uint64_t m = e ? ((bits & 0x7fffffu) | 0x800000u) : (bits & 0x7fffffu);
    // inv = m 2^(x - 150), x = max(e, 1): the product m * c is 152 bits,
    // t2 (24 bits) : t1 : t0; wanted is (m c) >> (64 + s), s = 150 - x
    const uint64_t t0h = __umul64hi(m, c_lo);
    const uint64_t t1 = m * c_hi + t0h;
    const uint64_t t2 = __umul64hi(m, c_hi) + (t1 < t0h ? 1 : 0);
    const int s = 150 - (e ? e : 1);
    if (s <= 0) return t1;                     // inv in [2^23, 2^24)
    if (s < 64) return (t1 >> s) | (t2 << (64 - s));
    return s < 128 ? t2 >> (s - 64) : 0;
}

template <typename Tin, typename Tout>
__global__ __launch_bounds__(PREP_THREADS) void k_prep(PrepArgs a) {
    __shared__ float2 cs[PREP_ROWS][O1_MAX_D / 2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r0 = blockIdx.x * PREP_ROWS, nr = min(PREP_ROWS, a.rows - r0);
    const int half = a.rot >> 1, nh = a.hq + a.hk;
    for (int i = tid; i < nr * half; i += PREP_THREADS) {
        const int r = i / half, j = i - r * half;
        const int64_t p = a.pos ? a.pos[r0 + r] : a.pos0 + r0 + r;
        const int64_t frac = (int64_t)(turns_of(a.inv[j]) * (uint64_t)p);   // in [-1/2, 1/2) turn
        float s, c;
        sincospif((float)frac * 0x1p-63f, &s, &c);
        cs[r][j] = make_float2(c, s);
    }
    __syncthreads();
    for (int it = warp; it < nr * nh; it += PREP_THREADS / 32) {
        const int r = it / nh, h = it - r * nh;
        const bool isq = h < a.hq;
        const Tin *x = isq ? (const Tin *)a.q + (size_t)(r0 + r) * a.qs + (size_t)h * a.d
                           : (const Tin *)a.k + (size_t)(r0 + r) * a.ks + (size_t)(h - a.hq) * a.d;
        Tout *o = isq ? (Tout *)a.qo + (size_t)(r0 + r) * a.qos + (size_t)h * a.d
                      : (Tout *)a.ko + (size_t)(r0 + r) * a.kos + (size_t)(h - a.hq) * a.d;
        const float *w = isq ? a.qw : a.kw;
        float4 v[2], u[2];   // values 4 lane + 128 i and their rotation partners
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = 4 * lane + 128 * i;
            v[i] = u[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (e >= a.d) continue;
            v[i] = o1_ld4(x + e);
            if (e < a.rot) u[i] = o1_ld4(x + (e < half ? e + half : e - half));
            ss += v[i].x * v[i].x + v[i].y * v[i].y + v[i].z * v[i].z + v[i].w * v[i].w;
        }
        float f = 1.f;
        if (a.norm != O1_NORM_NONE) {
            ss = warp_sum(ss);
            if (a.norm == O1_NORM_RMS) ss /= (float)a.d;
            ss += a.eps;
            f = ss > 0.f ? rsqrtf(ss) : 0.f;
        }
        __syncwarp();   // in place: every lane's loads of this head come before any store
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = 4 * lane + 128 * i;
            if (e >= a.d) continue;
            float4 wv = make_float4(1.f, 1.f, 1.f, 1.f);
            if (w) wv = *(const float4 *)(w + e);
            float4 y = make_float4(v[i].x * f * wv.x, v[i].y * f * wv.y, v[i].z * f * wv.z, v[i].w * f * wv.w);
            if (e < a.rot) {
                const bool lo = e < half;
                const int pe = lo ? e + half : e - half, j = lo ? e : pe;
                float4 pw = make_float4(1.f, 1.f, 1.f, 1.f);
                if (w) pw = *(const float4 *)(w + pe);
                const float sg = lo ? -1.f : 1.f;
                const float2 c0 = cs[r][j], c1 = cs[r][j + 1], c2 = cs[r][j + 2], c3 = cs[r][j + 3];
                y.x = y.x * c0.x + sg * (u[i].x * f * pw.x) * c0.y;
                y.y = y.y * c1.x + sg * (u[i].y * f * pw.y) * c1.y;
                y.z = y.z * c2.x + sg * (u[i].z * f * pw.z) * c2.y;
                y.w = y.w * c3.x + sg * (u[i].w * f * pw.w) * c3.y;
            }
            o1_st4(o + e, y);
        }
    }
}

template <typename Tin, typename Tout>
void prep_launch(const PrepArgs &a, cudaStream_t st) {
    k_prep<Tin, Tout><<<(a.rows - 1) / PREP_ROWS + 1, PREP_THREADS, 0, st>>>(a);
}

bool prep_geom_ok(const o1_prep_geom *g) {
    if (!g) return false;
    if (g->q_heads < 0 || g->q_heads > 4096 || g->k_heads < 0 || g->k_heads > 4096) return false;
    if (g->q_heads + g->k_heads < 1) return false;
    if (g->d < 8 || g->d > O1_MAX_D || g->d % 8) return false;
    if (g->rot < 0 || g->rot > g->d || g->rot % 8) return false;
    if (g->norm < O1_NORM_NONE || g->norm > O1_NORM_UNIT) return false;
    if (!o1_dtype_ok(g->in_dtype)) return false;
    if (g->out_dtype != O1_F32 && g->out_dtype != g->in_dtype) return false;
    return isfinite(g->eps) && g->eps >= 0.f;
}

}  // namespace

extern "C" int o1_head_prep(const o1_prep_geom *geom, const void *q, int64_t q_stride, const void *k,
                            int64_t k_stride, const float *q_weight, const float *k_weight, const float *inv_freq,
                            const int64_t *pos, int64_t pos0, int32_t rows, void *q_out, int64_t q_out_stride,
                            void *k_out, int64_t k_out_stride, void *stream) {
    if (!prep_geom_ok(geom)) return O1_ERR_UNSUPPORTED;
    if (rows < 0) return O1_ERR_ARG;
    if (rows == 0) return O1_OK;
    const o1_prep_geom &g = *geom;
    if (g.rot && !inv_freq) return O1_ERR_ARG;
    if ((uintptr_t)q_weight % 16 || (uintptr_t)k_weight % 16 || (uintptr_t)inv_freq % 4 || (uintptr_t)pos % 8)
        return O1_ERR_ARG;
    const O1Span in[2] = {o1_row_span(g.q_heads ? q : nullptr, g.in_dtype, g.q_heads, g.d, q_stride, rows),
                          o1_row_span(g.k_heads ? k : nullptr, g.in_dtype, g.k_heads, g.d, k_stride, rows)};
    const O1Span out[2] = {o1_row_span(g.q_heads ? q_out : nullptr, g.out_dtype, g.q_heads, g.d, q_out_stride, rows),
                           o1_row_span(g.k_heads ? k_out : nullptr, g.out_dtype, g.k_heads, g.d, k_out_stride, rows)};
    const O1Span side[4] = {o1_span(g.q_heads ? q_weight : nullptr, (size_t)g.d * 4),
                            o1_span(g.k_heads ? k_weight : nullptr, (size_t)g.d * 4),
                            o1_span(g.rot ? inv_freq : nullptr, (size_t)g.rot * 2), o1_span(pos, (size_t)rows * 8)};
    const int heads[2] = {g.q_heads, g.k_heads};
    for (int i = 0; i < 2; ++i) {
        if (!heads[i]) continue;
        if (!o1_rows_ok(in[i]) || !o1_rows_ok(out[i])) return O1_ERR_ARG;
        const bool inplace = in[i].p == out[i].p && in[i].stride == out[i].stride && g.in_dtype == g.out_dtype;
        if (!inplace && o1_spans_overlap(in[i], out[i])) return O1_ERR_ARG;
        if (o1_spans_overlap(in[1 - i], out[i])) return O1_ERR_ARG;
        for (const O1Span &s : side)
            if (o1_spans_overlap(s, out[i])) return O1_ERR_ARG;
    }
    if (o1_spans_overlap(out[0], out[1])) return O1_ERR_ARG;
    PrepArgs a;
    a.q = q; a.k = k; a.qo = q_out; a.ko = k_out;
    a.qw = q_weight; a.kw = k_weight; a.inv = inv_freq; a.pos = pos; a.pos0 = pos0;
    a.qs = (size_t)q_stride; a.ks = (size_t)k_stride; a.qos = (size_t)q_out_stride; a.kos = (size_t)k_out_stride;
    a.rows = rows; a.hq = g.q_heads; a.hk = g.k_heads; a.d = g.d; a.rot = g.rot; a.norm = g.norm; a.eps = g.eps;
    cudaStream_t st = (cudaStream_t)stream;
    if (g.in_dtype == O1_F32) prep_launch<float, float>(a, st);
    else if (g.in_dtype == O1_BF16 && g.out_dtype == O1_F32) prep_launch<__nv_bfloat16, float>(a, st);
    else if (g.in_dtype == O1_BF16) prep_launch<__nv_bfloat16, __nv_bfloat16>(a, st);
    else if (g.out_dtype == O1_F32) prep_launch<__half, float>(a, st);
    else prep_launch<__half, __half>(a, st);
    return cudaGetLastError() == cudaSuccess ? O1_OK : O1_ERR_CUDA;
}
