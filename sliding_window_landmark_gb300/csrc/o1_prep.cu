// o1_head_prep: the norm of every query and key head and their rotation in
// one pass over the rows ("cortiq-engine 0.8.77 src/gpu_wgpu/dory.rs",
// dory_prep). Per head vector: sum of squares, one factor, the weight, the
// half-split rotation of its first `rot` values.
//
// Bound: HBM; each value is read once and written once. What stands against it
// is the instruction count (a kernel with a lane on 8 consecutive values and
// rotation partners read again took 176 us for 32749 bf16 rows of 20 heads of
// 128, whose bytes take 50), so a lane holds both values of four rotation
// pairs: 4 values from the head's lower half and the 4 half a rotation further
// on (past the rotated part: 8 in a row), and works on pairs in packed fp32.
// 32 / lanes heads run side by side. A warp takes rows, or parts of a row's
// heads, with the row's cosines times the weights in registers; the loads of
// two rounds of heads go out before the cosines are made. The batch above: 65
// us, 5.2 TB/s, with 1450 instructions a row issued at 0.6 of the rate (four
// rounds in flight, or the next row's loads ahead of the stores, at 64
// registers 72 to 76; three blocks an SM with more registers 65 to 72); 4096
// fp32 rows of 10 heads of 256: 17 us, where the pipelined form takes 20.
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

constexpr int PREP_WARPS = 8;

struct PrepArgs {
    const void *q, *k;
    void *qo, *ko;
    const float *qw, *kw, *inv;
    const int64_t *pos;
    int64_t pos0;
    size_t qs, ks, qos, kos;   // row strides, elements
    int rows, hq, hk, d, rot, norm;
    int parts, per;   // warps of a row, and heads of one
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

// Two fp32 values in one register pair: the packed operations take one issue
// for both.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void f2_get(F2 x, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v)); }
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

template <typename T>
struct Raw4 {
    using type = uint2;
};
template <>
struct Raw4<float> {
    using type = float4;
};

// Sum of a head's squares over its LPV lanes.
template <int LPV>
__device__ __forceinline__ float head_squares(const F2 (&xl)[2], const F2 (&xh)[2], bool on) {
    const F2 s2 = f2_fma(xh[1], xh[1], f2_fma(xh[0], xh[0], f2_fma(xl[1], xl[1], f2_mul(xl[0], xl[0]))));
    float ss, s_odd;
    f2_get(s2, ss, s_odd);
    ss = on ? ss + s_odd : 0.f;
#pragma unroll
    for (int m = 1; m < LPV; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    return ss;
}
// A mean or sum of squares from here on has lost at most d 2^-150, 2^-52 of it,
// to squares below fp32's range; with an epsilon that large none can fall
// below. Below it (values under 2^-41) a head is squared times 2^100: the
// smallest fp32 value becomes 2^-49, and the sum of 256 stays under 2^118.
constexpr float TINY = 0x1p-90f;

// LPV lanes of 8 values a head (a power of two, 8 LPV >= d); SMALL: the epsilon
// is below TINY (a kernel of its own: the batch above 65.4 us, 65.9 with the
// question in every head)
template <typename Tin, typename Tout, int LPV, bool SMALL>
__global__ __launch_bounds__(32 * PREP_WARPS, 4) void k_prep(PrepArgs a) {
    using R = typename Raw4<Tin>::type;
    constexpr int SIDE = 32 / LPV, U = 2;   // heads side by side, and rounds of them in flight
    __shared__ float2 table[PREP_WARPS][O1_MAX_D / 2];
    __shared__ __align__(16) float sw[2][O1_MAX_D];   // weights of q and k
    __shared__ uint64_t turns[O1_MAX_D / 2];          // of one position step
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slot = lane % LPV, side = lane / LPV;
    const int half = a.rot >> 1, pairs = a.rot >> 3;
    const bool on = 8 * slot < a.d, rotates = slot < pairs;
    const int lo = on ? rotates ? 4 * slot : 8 * slot : 0, hi = on ? rotates ? lo + half : lo + 4 : 0;
    float2 *cs = table[warp];
    for (int j = threadIdx.x; j < half; j += 32 * PREP_WARPS) turns[j] = turns_of(a.inv[j]);
    for (int i = threadIdx.x; i < 2 * a.d; i += 32 * PREP_WARPS) {
        const int t = i >= a.d, c = i - t * a.d;
        const float *p = t ? a.kw : a.qw;
        sw[t][c] = p ? p[c] : 1.f;
    }
    __syncthreads();
    const float inv_d = a.norm == O1_NORM_RMS ? 1.f / (float)a.d : 1.f;
    const int64_t items = (int64_t)a.rows * a.parts;
    for (int64_t it = (int64_t)blockIdx.x * PREP_WARPS + warp; it < items; it += (int64_t)gridDim.x * PREP_WARPS) {
        const int r = (int)(it / a.parts), part = (int)(it - (int64_t)r * a.parts);
        const int64_t pos = a.pos ? a.pos[r] : a.pos0 + r;
        const int h_end = min(a.hq + a.hk, (part + 1) * a.per);
        bool made = false;
        for (int h0 = part * a.per; h0 < h_end;) {
            // the part's heads of q, then those of k
            const bool isq = h0 < a.hq;
            const int h1 = isq ? min(h_end, a.hq) : h_end;
            const Tin *x = isq ? (const Tin *)a.q + (size_t)r * a.qs : (const Tin *)a.k + (size_t)r * a.ks - (size_t)a.hq * a.d;
            Tout *o = isq ? (Tout *)a.qo + (size_t)r * a.qos : (Tout *)a.ko + (size_t)r * a.kos - (size_t)a.hq * a.d;
            F2 c0[2], c1[2], s0[2], s1[2];   // z_lo = c0 x_lo + s0 x_hi, z_hi = c1 x_hi + s1 x_lo
            bool have = false;
            for (int h = h0; h < h1; h += SIDE * U) {
                R vl[U], vh[U];
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int hh = h + SIDE * k + side;
                    const Tin *p = x + (size_t)(hh < h1 ? hh : h) * a.d;
                    vl[k] = *(const R *)(p + lo);
                    vh[k] = *(const R *)(p + hi);
                }
                if (!made) {
                    __syncwarp();
                    for (int j = lane; j < half; j += 32) {
                        // the angle's fraction of a turn, [-1/2, 1/2), to 2^-32
                        const int frac = (int)(uint32_t)((turns[j] * (uint64_t)pos) >> 32);
                        float s, c;
                        sincospif((float)frac * 0x1p-31f, &s, &c);
                        cs[j] = make_float2(c, s);
                    }
                    __syncwarp();
                    made = true;
                }
                if (!have) {
                    const float4 wl = *(const float4 *)&sw[isq ? 0 : 1][lo], wh = *(const float4 *)&sw[isq ? 0 : 1][hi];
                    float2 t[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) t[i] = rotates ? cs[lo + i] : make_float2(1.f, 0.f);
                    c0[0] = f2(wl.x * t[0].x, wl.y * t[1].x);
                    c0[1] = f2(wl.z * t[2].x, wl.w * t[3].x);
                    s0[0] = f2(-wh.x * t[0].y, -wh.y * t[1].y);
                    s0[1] = f2(-wh.z * t[2].y, -wh.w * t[3].y);
                    c1[0] = f2(wh.x * t[0].x, wh.y * t[1].x);
                    c1[1] = f2(wh.z * t[2].x, wh.w * t[3].x);
                    s1[0] = f2(wl.x * t[0].y, wl.y * t[1].y);
                    s1[1] = f2(wl.z * t[2].y, wl.w * t[3].y);
                    have = true;
                }
                __syncwarp();   // in place: every lane's loads of these heads come before any store
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const int hh = h + SIDE * k + side;
                    const float4 l = o1_ld4((const Tin *)&vl[k]), g = o1_ld4((const Tin *)&vh[k]);
                    F2 xl[2] = {f2(l.x, l.y), f2(l.z, l.w)}, xh[2] = {f2(g.x, g.y), f2(g.z, g.w)};
                    float f = 1.f;
                    if (a.norm != O1_NORM_NONE) {
                        float ss = fmaf(head_squares<LPV>(xl, xh, on), inv_d, a.eps);
                        if (SMALL && __any_sync(0xffffffffu, ss < TINY)) {
                            // squares that leave fp32's range at the bottom: such heads times 2^100
                            const float up = ss < TINY ? 0x1p100f : 1.f;
                            const F2 u2 = f2(up, up);
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                xl[i] = f2_mul(u2, xl[i]);
                                xh[i] = f2_mul(u2, xh[i]);
                            }
                            ss = fmaf(head_squares<LPV>(xl, xh, on), inv_d, a.eps * up * up);
                        }
                        f = ss == 0.f ? 0.f : rsqrtf(ss);   // a NaN stays one
                    }
                    const F2 ff = f2(f, f);
                    float yl[4], yh[4];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const F2 ul = f2_mul(ff, xl[i]), uh = f2_mul(ff, xh[i]);
                        F2 zl = f2_mul(c0[i], ul), zh = f2_mul(c1[i], uh);
                        if (rotates) {
                            zl = f2_fma(s0[i], uh, zl);
                            zh = f2_fma(s1[i], ul, zh);
                        }
                        f2_get(zl, yl[2 * i], yl[2 * i + 1]);
                        f2_get(zh, yh[2 * i], yh[2 * i + 1]);
                    }
                    if (on && hh < h1) {
                        Tout *p = o + (size_t)hh * a.d;
                        o1_st4(p + lo, make_float4(yl[0], yl[1], yl[2], yl[3]));
                        o1_st4(p + hi, make_float4(yh[0], yh[1], yh[2], yh[3]));
                    }
                }
            }
            h0 = h1;
        }
    }
}

template <typename Tin, typename Tout, int LPV>
void prep_launch_l(PrepArgs a, cudaStream_t st) {
    // Warps of a row: one, or more while the rows leave SMs idle (down to the
    // heads that a warp has in flight).
    constexpr int UNIT = (32 / LPV) * 2, SMS = 152;
    const int nh = a.hq + a.hk, most = (nh + UNIT - 1) / UNIT, want = (SMS * 16 - 1) / a.rows + 1;
    a.parts = want < most ? want : most;
    a.per = (most + a.parts - 1) / a.parts * UNIT;
    a.parts = (nh + a.per - 1) / a.per;
    // At most the blocks that run at once (four an SM): a warp then takes rows
    // in turn, and none of a second wave's SMs idle (the batch above: 65 us;
    // 1.7 waves 68, a block for every 8 rows 69, 1.25 waves 80).
    const int64_t blocks = ((int64_t)a.rows * a.parts + PREP_WARPS - 1) / PREP_WARPS, most_blocks = 4 * SMS;
    const int64_t grid = blocks < most_blocks ? blocks : most_blocks;
    if (a.eps < TINY && a.norm != O1_NORM_NONE) k_prep<Tin, Tout, LPV, true><<<(unsigned)grid, 32 * PREP_WARPS, 0, st>>>(a);
    else k_prep<Tin, Tout, LPV, false><<<(unsigned)grid, 32 * PREP_WARPS, 0, st>>>(a);
}
template <typename Tin, typename Tout>
void prep_launch(const PrepArgs &a, cudaStream_t st) {
    if (a.d <= 32) prep_launch_l<Tin, Tout, 4>(a, st);
    else if (a.d <= 64) prep_launch_l<Tin, Tout, 8>(a, st);
    else if (a.d <= 128) prep_launch_l<Tin, Tout, 16>(a, st);
    else prep_launch_l<Tin, Tout, 32>(a, st);
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
    PrepArgs a = {};
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
