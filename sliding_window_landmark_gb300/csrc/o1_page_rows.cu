// Attention over the paged cache for few rows a group: decode rows, and chunks
// of few query vectors. The query heads of a group share its keys, so up to 16
// query vectors (rows of the sequence times heads of the group) go against each
// key with one mma.sync m16n8k16: the keys and values are read once, and the
// bound is HBM.
//
// A warp takes 16 of a tile's keys and keeps a softmax and an accumulator of
// its own, so that nothing waits for another warp until the segment's end. Its
// keys and values, 16 rows of a page and so contiguous, come by 16-byte
// asynchronous copies, 512 bytes in a row an instruction, into a ring of items
// of its own (16 keys, or 16 values). (A lane copying just the bytes that it
// will use needs no exchange, but an instruction then touches 8 or 16 rows: 1024
// bf16 heads of 9000 positions took 970 us.) The order of a contraction is free:
// the lane that holds key n's contraction indices 2q, 2q + 1, 2q + 8, 2q + 9 of
// every k16 step (q = lane % 4) takes them from 16 consecutive bytes of the row,
// and the queries are laid out to match; likewise a lane takes 16 consecutive
// bytes of the value columns, column j of it belonging to the j-th n8 tile. The
// pieces of 16 bytes are permuted within 128 by their key, so that neither read
// hits a bank twice.
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "o1_page.cuh"

namespace {

constexpr int RW = 4, RT = 32 * RW;   // warps and threads of a block
constexpr int RV = PG_ROWS_V;         // query vectors of a unit
constexpr int TILE = 16 * RW;         // keys of a tile
// Two blocks an SM leave a thread 255 registers (three, with 168, took 3 % longer).
constexpr int PER_SM = 2, BLOCKS = 152 * PER_SM;
// A segment of a decode batch costs as much as five tiles of keys: 61 bf16 rows of
// 1 to 32768 positions over e4m3 took 113 us with START = 1, 88 with 2, 75 with 3,
// 68 with 4, 64 with 5, 65 with 6, 66 with 8. A single fp32 row at 8191: 31 us with
// LEAST = 1 (its parts' sum takes longer), 23 with 2, 27 with 4, 31 with 6.
struct Plan {
    static constexpr int V = RV, K = TILE, START = 5, LEAST = 2;
};

// Rows of type T over a cache of type C: the MMA's type M, and the terms that q
// and the weights are split into (a weight at most 2^8, in fp16 2^15): 16-bit rows
// over their own type need one, fp32 rows three, which hold fp32.
// 16-bit rows over e4m3 run in fp16, which holds the codes: a pair of codes is
// one conversion (bf16 takes four). fp16's short range is met by powers of two:
// a query vector is taken times the one that brings its largest value into [1,
// 2), and the weights of the values, which carry the values' powers of two, from
// a reference of their own, the maximum of score and power together.
template <typename T, typename C>
struct Types {
    using M = T;
    static constexpr int TERMS = 1;
    static constexpr bool CODES = false;   // codes under powers of two in fp16
};
template <>
struct Types<float, __nv_bfloat16> {
    using M = __nv_bfloat16;
    static constexpr int TERMS = 3;
    static constexpr bool CODES = false;
};
template <>
struct Types<float, uint8_t> {
    using M = __nv_bfloat16;
    static constexpr int TERMS = 3;
    static constexpr bool CODES = false;
};
template <typename T>
struct Types<T, uint8_t> {
    using M = __half;
    static constexpr int TERMS = 1;
    static constexpr bool CODES = true;
};

// Sizes for widths of up to 64 N values.
template <typename C, int N, int TERMS>
struct Sizes {
    static constexpr int CB = sizeof(C), VL = 16 / CB;   // values of a lane's 16 bytes
    static constexpr int KB = N * CB;                    // 64-byte blocks of a key
    static constexpr int VB = (N * CB + 1) / 2;          // 128-byte blocks of a value row
    static constexpr int STEPS = N * 4;                  // k16 steps of a key
    static constexpr int ITEM = (2 * KB > 4 * VB ? 2 * KB : 4 * VB) * 512;
    static constexpr int QUERIES = TERMS * STEPS * 512;  // bytes of the queries
    // items of a warp's ring: what PER_SM blocks an SM hold beside the queries (wide
    // fp32 rows over 16 bits: one in use and one in flight; 64 rows of 2 groups of 4
    // heads of 256 at 8191 took 177 us, and 299 with three items and one block an SM;
    // over e4m3 194 with five, 294 with six and one block)
    static constexpr int RING = N == 4 ? (CB == 2 ? (TERMS == 3 ? 2 : 3) : TERMS == 3 ? 5 : 6) : N == 2 && CB == 2 ? 6 : 8;
    static constexpr int RESULTS = RV * (64 * N + 4) * 4;   // a warp's, in its ring
    static constexpr int WARP = RING * ITEM > RESULTS ? RING * ITEM : RESULTS, SMEM = RW * WARP + QUERIES;
    // beside it: the block's static part, and what the SM keeps for itself a block
    static_assert(PER_SM * (SMEM + 768 + (CB == 1 ? RW * RING * 32 : 0) + 1024) <= 228 * 1024, "one wave of blocks");
};

__device__ __forceinline__ uint32_t pack_m(const __nv_bfloat16 *, float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *(const uint32_t *)&h;
}
__device__ __forceinline__ uint32_t pack_m(const __half *, float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *(const uint32_t *)&h;
}
__device__ __forceinline__ float2 unpack_m(const __nv_bfloat16 *, uint32_t w) {
    return __bfloat1622float2(*(const __nv_bfloat162 *)&w);
}
__device__ __forceinline__ float2 unpack_m(const __half *, uint32_t w) { return __half22float2(*(const __half2 *)&w); }

// (a, b) as TERMS packed pairs, the first the nearest, each next the nearest to
// what is left (the subtractions are exact)
template <typename M, int TERMS>
__device__ __forceinline__ void split_m(float a, float b, uint32_t (&w)[TERMS]) {
#pragma unroll
    for (int t = 0; t < TERMS; ++t) {
        w[t] = pack_m((const M *)nullptr, a, b);
        if (t + 1 < TERMS) {
            const float2 f = unpack_m((const M *)nullptr, w[t]);
            a -= f.x;
            b -= f.y;
        }
    }
}

__device__ __forceinline__ void mma16(const __nv_bfloat16 *, float (&c)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16(const __half *, float (&c)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// two e4m3 codes (low half of w, or its high half) as a pair of M: exact
__device__ __forceinline__ uint32_t of_e4m3(const __half *, uint32_t w, int half) {
    const uint16_t two = (uint16_t)(half ? w >> 16 : w);
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
    return h;
}
__device__ __forceinline__ uint32_t of_e4m3(const __nv_bfloat16 *m, uint32_t w, int half) {
    const uint32_t h = of_e4m3((const __half *)nullptr, w, half);
    const float2 f = __half22float2(*(const __half2 *)&h);
    return pack_m(m, f.x, f.y);
}

// 16 bytes, or zeros where !on
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool on) {
    const int n = on ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
template <int O>
__device__ __forceinline__ void copy16_at(uint32_t dst, const void *src) {   // dst + O, src + O
    asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %2], 16;" ::"r"(dst), "l"(src), "n"(O) : "memory");
}
// What the 16-byte pieces of a key's row are permuted by (piece p of each 128
// bytes lies at p ^ turn). 8 lanes that read at once read 4 pieces of keys 2i and
// 2i + 1, which differ in bit 2 of it, or 2 pieces of values 0, 2, 4, 6 or 1, 3,
// 5, 7 (mod 8), which differ in bits 1 and 2.
__device__ __forceinline__ constexpr int turn(int k) { return ((k >> 2 ^ k) & 1) << 2 | (k & 2); }
// (rows of 128, 256 and 512 bytes; others lie as they come)
__device__ __forceinline__ bool turned(int width) { return width >= 128 && !(width & (width - 1)); }
// A loop of constants 0 .. N - 1.
template <int N, typename F>
__device__ __forceinline__ void each(F f) {
    if constexpr (N > 0) {
        each<N - 1>(f);
        f(std::integral_constant<int, N - 1>());
    }
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename T, typename C, int N>
__global__ __launch_bounds__(RT, PER_SM) void k_pg_rows(PgArgs a, const __grid_constant__ PgTable tab, int units) {
    using Ty = Types<T, C>;
    using M = typename Ty::M;
    constexpr int TERMS = Ty::TERMS;
    constexpr bool CODES = Ty::CODES;
    using Z = Sizes<C, N, TERMS>;
    constexpr int CB = Z::CB, VL = Z::VL, KB = Z::KB, VB = Z::VB, STEPS = Z::STEPS, RING = Z::RING, ITEM = Z::ITEM;
    constexpr bool E4 = CB == 1;
    constexpr bool Q_REGS = TERMS == 1 && N <= 2;   // the queries in registers
    // of the sum's weights, and of the values' (the same ones unless CODES)
    constexpr PgReference REF(std::is_same<M, __half>::value && !CODES), REF_V(std::is_same<M, __half>::value);
    extern __shared__ __align__(128) unsigned char sm[];
    __shared__ long long s_share[RW + 2];
    __shared__ float s_m[RW][RV], s_l[RW][RV];
    __shared__ int s_qe[RV];
    __shared__ __align__(16) uint8_t s_exp[E4 ? RW * RING * 32 : 16];   // of an item of keys: theirs, then the values'
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, qd = lane & 3, row = lane >> 2;
    unsigned char *ring = sm + (size_t)warp * Z::WARP;
    const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
    uint32_t *sq = (uint32_t *)(sm + (size_t)RW * Z::WARP);   // [term][step][lane][4]

    PgShare share = pg_share<Plan, RT>(a, tab, units, s_share);
    const PgParts parts = pg_parts(a.part, BLOCKS, RV);
    if (tid == 0) parts.head[blockIdx.x].last = -1;
    const float sc2 = a.scale * 1.4426950408889634f;
    const int kb_n = (a.d * CB + 63) >> 6, vb_n = (a.dv * CB + 127) >> 7;
    const bool k_whole = (a.d * CB & 63) == 0;
    const int kw = a.d * CB, vw = a.dv * CB;   // bytes of a cached row
    // this lane's pieces of an item: of key `row` (block b: even and odd ones), of
    // values 2 qd and 2 qd + 1; 8 rows further on the same
    const int k_turn = turned(kw) ? turn(row) : 0, v_turn = turned(vw) ? turn(2 * qd) : 0, v_turn1 = turned(vw) ? turn(2 * qd + 1) : 0;
    const int k_even = row * kw + 16 * (qd ^ k_turn), k_odd = row * kw + 16 * ((4 + qd) ^ k_turn);
    const int v_even = 2 * qd * vw + 16 * (row ^ v_turn), v_odd = (2 * qd + 1) * vw + 16 * (row ^ v_turn1);
    bool first_seg = true;
    PgSegment seg;
    while (pg_next<Plan>(a, tab, units, share, seg)) {
        const PgUnit &x = seg.x;
        const int g = seg.g;
        __syncthreads();   // the segment before is done with shared memory
        if (CODES) {   // the exponents of the query vectors' largest values, eight threads a vector
            const int v = tid >> 3;
            float top = 0.f;
            if (v < x.nv) {
                const T *q = (const T *)a.q + pg_vec_at(a, x.row0, x.vec0 + v, g, a.qs, a.d);
                for (int c = 4 * (tid & 7); c < a.d; c += 32) {
                    const float4 f = o1_ld4(q + c);
                    top = fmaxf(top, fmaxf(fmaxf(fabsf(f.x), fabsf(f.y)), fmaxf(fabsf(f.z), fabsf(f.w))));
                }
            }
#pragma unroll
            for (int k = 1; k < 8; k <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
            // 2^-e and 2^e are normal numbers; an exponent below that range loses nothing but zeros
            if ((tid & 7) == 0) s_qe[v] = min(max((int)(__float_as_uint(top) >> 23) - 127, -126), 126);
            __syncthreads();
        }
        // ---- queries, in the MMA's A layout of this lane order
        for (int i = tid; i < kb_n * (VL / 4) * 32; i += RT) {
            const int st = i >> 5, ln = i & 31, b = st / (VL / 4), s = st - b * (VL / 4);
            const int c = 4 * VL * b + VL * (ln & 3) + 4 * s;   // 4 consecutive values: k indices 2q, 2q + 1, 2q + 8, 2q + 9
            uint32_t w[4][TERMS];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int v = (ln >> 2) + 8 * h;
                float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                if (v < x.nv && c < a.d) f = o1_ld4((const T *)a.q + pg_vec_at(a, x.row0, x.vec0 + v, g, a.qs, a.d) + c);
                if (CODES) {
                    const float e = pg_scale((uint32_t)(127 - s_qe[v]));
                    f = make_float4(f.x * e, f.y * e, f.z * e, f.w * e);
                }
                split_m<M, TERMS>(f.x, f.y, w[h]);
                split_m<M, TERMS>(f.z, f.w, w[2 + h]);
            }
#pragma unroll
            for (int t = 0; t < TERMS; ++t) *(uint4 *)(sq + ((t * STEPS + st) * 32 + ln) * 4) = make_uint4(w[0][t], w[1][t], w[2][t], w[3][t]);
        }
        __syncthreads();
        uint4 qr[Q_REGS ? STEPS : 1];
        if (Q_REGS) {
#pragma unroll
            for (int st = 0; st < (Q_REGS ? STEPS : 1); ++st) qr[st] = *(const uint4 *)(sq + (st * 32 + lane) * 4);
        }

        // ---- this warp's blocks of 16 keys: blk0, blk0 + RW, ...
        const int blk0 = (x.lo / TILE + seg.t0) * RW + warp, nb = seg.t1 - seg.t0;
        int pos[2], low[2];   // of this lane's two vectors: last and first position attended
        float sc[2];          // what a score of theirs is taken times
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            pos[h] = x.pos(a, min(row + 8 * h, x.nv - 1));   // past the last: zeros, not written
            low[h] = a.window ? pos[h] - a.window + 1 : 0;
            sc[h] = CODES ? sc2 * pg_scale((uint32_t)(s_qe[row + 8 * h] + 127)) : sc2;
        }
        const int plain_lo = a.window ? max(0, x.hi - a.window + 1) : 0, plain_hi = x.pos(a, 0);
        // m, l: the softmax's reference and sum; mv: the reference of the values' weights
        float acc[VB * VL][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, mv[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < VB * VL; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
        // pages of the next 32 blocks, a lane each, and of the 32 after them
        auto page_of = [&](int i) {
            const int p = (blk0 + RW * i) * 16;
            return i < nb && p <= x.hi ? pg_page(a, x.slot, p) : -1;
        };
        int pages = page_of(lane), pages_next = page_of(32 + lane);
        uint32_t present = 0;   // bit i % 32: block i has a page
        int put = 0, put_slot = 0, get_slot = 0;   // next item to issue: block put / 2, keys then values
        int rowid = 0;          // of the block's first position in the pools
        bool inside = false;    // all of the block's positions are attended by some vector, and on a page
        // 16 rows of `width` bytes from row `rowid` of a pool. Where not all of
        // them are attended, the others are zeros.
        auto copy_rows = [&](const void *pool, int width, int i) {
            const uint32_t dst = ring_at + put_slot * ITEM;
            const char *src = (const char *)pool + (size_t)(uint32_t)rowid * width + 16 * lane;
            const bool sw = turned(width);
            constexpr int MOST = ITEM / 512;
            if (inside && sw) {
                // 512 bytes: half a key, one, two or four; piece p of key k goes
                // to p ^ turn(k), of which the lane's part stands in `at` and
                // the instruction's is a constant
                const int log = 31 - __clz(width);   // 7 to 9
                const uint32_t at = dst + ((16 * lane) ^ (log == 7 ? 16 * turn(lane >> 3) : log == 8 ? 16 * turn(lane >> 4) : 0));
                each<MOST>([&](auto n) {
                    if (n * 512 < 16 * width) {
                        const uint32_t x = log == 7 ? 16 * turn(4 * n) : log == 8 ? 16 * turn(2 * n) : 16 * turn(n);
                        copy16_at<n * 512>(at ^ x, src);
                    }
                });
            } else if (inside) {
                each<MOST>([&](auto n) {
                    if (n * 512 + 16 * lane < 16 * width) copy16_at<n * 512>(dst + 16 * lane, src);
                });
            } else {
                const int p0 = (blk0 + RW * i) * 16;
                const bool page = present >> (i & 31) & 1;
#pragma unroll 1
                for (int o = 16 * lane; o < 16 * width; o += 512) {
                    const int key = o / width, p = p0 + key;
                    const bool on = page && p >= x.lo && p <= x.hi;
                    copy16(dst + (o ^ (sw ? 16 * turn(key) : 0)), on ? src + (o - 16 * lane) : pool, on);
                }
            }
        };
        auto issue_keys = [&]() {
            const int i = put >> 1;
            if (i < nb) {
                const int p0 = (blk0 + RW * i) * 16;
                const int page = __shfl_sync(0xffffffffu, pages, i & 31);
                present = (present & ~(1u << (i & 31))) | (page >= 0 ? 1u : 0u) << (i & 31);
                rowid = ((max(page, 0) * a.G + g) << a.lpage) + (p0 & ((1 << a.lpage) - 1));
                inside = page >= 0 && p0 >= x.lo && p0 + 15 <= x.hi;
                copy_rows(a.k, kw, i);
                if (E4 && lane < 2) {   // the 16 exponents of the keys, and of the values
                    const uint8_t *e = lane ? a.ve : a.ke;
                    copy16((uint32_t)__cvta_generic_to_shared(&s_exp[(warp * RING + put_slot) * 32 + 16 * lane]),
                           page >= 0 ? e + (size_t)(uint32_t)rowid : e, page >= 0);
                }
            }
            copy_commit();
            ++put;
            put_slot = put_slot + 1 == RING ? 0 : put_slot + 1;
        };
        auto issue_values = [&]() {   // of the block whose keys were issued last
            const int i = put >> 1;
            if (i < nb) {
                copy_rows(a.v, vw, i);
                if ((i & 31) == 31) {
                    pages = pages_next;
                    pages_next = page_of(i + 33 + lane);
                }
            }
            copy_commit();
            ++put;
            put_slot = put_slot + 1 == RING ? 0 : put_slot + 1;
        };
        // items alternate: the one RING - 1 further on, keys or values
        auto issue_at = [&](bool keys) {
            if (keys) issue_keys();
            else issue_values();
        };
        // the item to use next: all but the last RING - 1 groups of every lane are here
        auto item = [&]() -> const unsigned char * {
            copy_wait<RING - 1>();
            __syncwarp();
            return ring + get_slot * ITEM;
        };
        auto done = [&]() {
            __syncwarp();
            get_slot = get_slot + 1 == RING ? 0 : get_slot + 1;
        };
#pragma unroll 1
        for (int i = 0; i < RING - 1; ++i) issue_at(!(i & 1));
#pragma unroll 1
        for (int i = 0; i < nb; ++i) {
            issue_at((RING - 1) % 2 == 0);
            const unsigned char *it = item();
            // ---- scores
            // the lower terms of q in a sum of their own: the MMA truncates at each
            // accumulation, and three times as many of the full sum showed (d = 256:
            // fp32 outputs 1.2e-6 off in the 2-norm)
            float s[2][4] = {}, low_s[2][4] = {};
#pragma unroll
            for (int b = 0; b < KB; ++b)
                if (b < kb_n) {
                    uint4 kw4[2];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        kw4[n] = *(const uint4 *)(it + (b & 1 ? k_odd : k_even) + (b >> 1) * 128 + n * 8 * kw);
                        if (!k_whole && b == kb_n - 1 && 4 * VL * b + VL * qd >= a.d) kw4[n] = make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int st = 0; st < VL / 4; ++st) {
                        uint32_t b0[2], b1[2];
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            if (E4) {
                                const uint32_t w = st == 0 ? kw4[n].x : st == 1 ? kw4[n].y : st == 2 ? kw4[n].z : kw4[n].w;
                                b0[n] = of_e4m3((const M *)nullptr, w, 0);
                                b1[n] = of_e4m3((const M *)nullptr, w, 1);
                            } else {
                                b0[n] = st == 0 ? kw4[n].x : kw4[n].z;
                                b1[n] = st == 0 ? kw4[n].y : kw4[n].w;
                            }
                        }
#pragma unroll
                        for (int t = TERMS - 1; t >= 0; --t) {
                            const int step = b * (VL / 4) + st;
                            const uint4 qa = Q_REGS ? qr[Q_REGS ? step : 0] : *(const uint4 *)(sq + ((t * STEPS + step) * 32 + lane) * 4);
#pragma unroll
                            for (int n = 0; n < 2; ++n) mma16((const M *)nullptr, t ? low_s[n] : s[n], qa, b0[n], b1[n]);
                        }
                    }
                }
            const int p0 = (blk0 + RW * i) * 16;
            uint32_t eb[2][2];   // this lane's columns' bytes, keys' and values': column c of tile n in byte c
            if (E4) {
                const uint8_t *e = &s_exp[(warp * RING + get_slot) * 32 + 2 * qd];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) eb[kv][n] = *(const uint16_t *)(e + 16 * kv + 8 * n);
            }
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[n][j] = (TERMS > 1 ? s[n][j] + low_s[n][j] : s[n][j]) * sc[j >> 1];
                    if (E4) s[n][j] *= pg_scale(eb[0][n] >> (8 * (j & 1)) & 0xff);
                }
            const bool there = present >> (i & 31) & 1;
            if (!(there && p0 >= plain_lo && p0 + 15 <= plain_hi)) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int p = p0 + 8 * n + 2 * qd + (j & 1);
                        if (!there || p > pos[j >> 1] || p < low[j >> 1]) s[n][j] = -INFINITY;
                    }
            }
            done();
            issue_at((RING - 1) % 2 == 1);
            // ---- softmax: a reference near the running maximum
            float top[2], topv[2], sv[2][4];
            if (CODES) {   // score and the value's power of two together (-inf stays)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sv[n][j] = s[n][j] + (float)((int)(eb[1][n] >> (8 * (j & 1)) & 0xff) - 127);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                top[h] = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
                top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
                top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
                topv[h] = top[h];
                if (CODES) {
                    topv[h] = fmaxf(fmaxf(sv[0][2 * h], sv[0][2 * h + 1]), fmaxf(sv[1][2 * h], sv[1][2 * h + 1]));
                    topv[h] = fmaxf(topv[h], __shfl_xor_sync(0xffffffffu, topv[h], 1));
                    topv[h] = fmaxf(topv[h], __shfl_xor_sync(0xffffffffu, topv[h], 2));
                }
            }
            if (__any_sync(0xffffffffu, top[0] > m[0] + REF.above || top[1] > m[1] + REF.above ||
                                            (CODES && (topv[0] > mv[0] + REF_V.above || topv[1] > mv[1] + REF_V.above)))) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float mn = fmaxf(m[h], top[h] - REF.below), r = m[h] > -INFINITY ? ex2(m[h] - mn) : 0.f;
                    m[h] = mn;
                    l[h] *= r;
                    float rv = r;
                    if (CODES) {
                        const float mvn = fmaxf(mv[h], topv[h] - REF_V.below);
                        rv = mv[h] > -INFINITY ? ex2(mv[h] - mvn) : 0.f;
                        mv[h] = mvn;
                    }
#pragma unroll
                    for (int j = 0; j < VB * VL; ++j) {
                        acc[j][2 * h] *= rv;
                        acc[j][2 * h + 1] *= rv;
                    }
                }
            }
            const float ref[2] = {m[0] > -INFINITY ? m[0] : 0.f, m[1] > -INFINITY ? m[1] : 0.f};
            const float refv[2] = {mv[0] > -INFINITY ? mv[0] : 0.f, mv[1] > -INFINITY ? mv[1] : 0.f};
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[n][j] = ex2(s[n][j] - ref[j >> 1]);
                    l[j >> 1] += s[n][j];
                    if (CODES) s[n][j] = ex2(sv[n][j] - refv[j >> 1]);
                    // fp32 rows: the value's power of two (a masked position's byte may be any)
                    else if (E4) s[n][j] = s[n][j] > 0.f ? s[n][j] * pg_scale(eb[1][n] >> (8 * (j & 1)) & 0xff) : 0.f;
                }
            // ---- weighted values
            it = item();
            uint32_t w[4][TERMS];
            split_m<M, TERMS>(s[0][0], s[0][1], w[0]);
            split_m<M, TERMS>(s[0][2], s[0][3], w[1]);
            split_m<M, TERMS>(s[1][0], s[1][1], w[2]);
            split_m<M, TERMS>(s[1][2], s[1][3], w[3]);
#pragma unroll
            for (int b = 0; b < VB; ++b)
                if (b < vb_n) {
                    uint32_t vr[4][4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) *(uint4 *)vr[r] = *(const uint4 *)(it + (r & 1 ? v_odd : v_even) + b * 128 + (r >> 1) * 8 * vw);
#pragma unroll
                    for (int j4 = 0; j4 < 4; ++j4) {
                        uint32_t b0[VL / 4], b1[VL / 4];   // of the columns in word j4
                        if (E4) {
                            const uint32_t lo = __byte_perm(vr[0][j4], vr[1][j4], 0x5140), hi = __byte_perm(vr[0][j4], vr[1][j4], 0x7362);
                            const uint32_t lo8 = __byte_perm(vr[2][j4], vr[3][j4], 0x5140), hi8 = __byte_perm(vr[2][j4], vr[3][j4], 0x7362);
#pragma unroll
                            for (int c = 0; c < VL / 4; ++c) {
                                b0[c] = of_e4m3((const M *)nullptr, c < 2 ? lo : hi, c & 1);
                                b1[c] = of_e4m3((const M *)nullptr, c < 2 ? lo8 : hi8, c & 1);
                            }
                        } else {
#pragma unroll
                            for (int c = 0; c < VL / 4; ++c) {
                                b0[c] = __byte_perm(vr[0][j4], vr[1][j4], c ? 0x7632 : 0x5410);
                                b1[c] = __byte_perm(vr[2][j4], vr[3][j4], c ? 0x7632 : 0x5410);
                            }
                        }
#pragma unroll
                        for (int c = 0; c < VL / 4; ++c) {
                            float (&o)[4] = acc[b * VL + j4 * (VL / 4) + c];
                            if (TERMS == 3) {
                                // a sum of its own, added with rounding: the MMA's own accumulation truncates
                                // each time, the same way, which over a long cache adds up
                                float y[4] = {};
#pragma unroll
                                for (int t = TERMS - 1; t >= 0; --t)
                                    mma16((const M *)nullptr, y, make_uint4(w[0][t], w[1][t], w[2][t], w[3][t]), b0[c], b1[c]);
#pragma unroll
                                for (int i2 = 0; i2 < 4; ++i2) o[i2] += y[i2];
                            } else {
                                mma16((const M *)nullptr, o, make_uint4(w[0][0], w[1][0], w[2][0], w[3][0]), b0[c], b1[c]);
                            }
                        }
                    }
                }
            done();
        }
        copy_wait<0>();

        // ---- the four warps' results under one reference
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            if (qd == 0) s_m[warp][row + 8 * h] = m[h], s_l[warp][row + 8 * h] = l[h];
        }
        __syncthreads();
        float big[2], fac[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            big[h] = -INFINITY;
            for (int w = 0; w < RW; ++w) big[h] = fmaxf(big[h], s_m[w][row + 8 * h]);
            const float from = CODES ? mv[h] : m[h];   // what the sums are relative to
            fac[h] = from > -INFINITY ? ex2(from - big[h]) : 0.f;
        }
        const int ld = a.dv + 4;
        float *so = (float *)ring;   // [RV][ld]: within this warp's ring
#pragma unroll
        for (int b = 0; b < VB; ++b)
            if (b < vb_n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {   // C column 2 qd + (j & 1) of vector row + 8 (j / 2)
                    const int c0 = 8 * VL * b + VL * (2 * qd + (j & 1));
                    if (c0 >= a.dv) continue;
#pragma unroll
                    for (int i = 0; i < VL; i += 4)
                        *(float4 *)(so + (row + 8 * (j >> 1)) * ld + c0 + i) =
                            make_float4(acc[b * VL + i][j] * fac[j >> 1], acc[b * VL + i + 1][j] * fac[j >> 1],
                                        acc[b * VL + i + 2][j] * fac[j >> 1], acc[b * VL + i + 3][j] * fac[j >> 1]);
                }
        __syncthreads();
        const bool whole = seg.whole();
        const size_t ps = seg.part();
        for (int i = tid; i < x.nv * (a.dv >> 2); i += RT) {
            const int v = i / (a.dv >> 2), c = 4 * (i - v * (a.dv >> 2));
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            float sum = 0.f, mx = -INFINITY;
            for (int w = 0; w < RW; ++w) mx = fmaxf(mx, s_m[w][v]);
            for (int w = 0; w < RW; ++w) {
                const float4 y = *(const float4 *)((const float *)(sm + (size_t)w * Z::WARP) + v * ld + c);
                o.x += y.x; o.y += y.y; o.z += y.z; o.w += y.w;
                sum += s_m[w][v] > -INFINITY ? s_l[w][v] * ex2(s_m[w][v] - mx) : 0.f;
            }
            if (whole) {
                const float r = sum == 0.f ? 0.f : 1.f / sum;   // a NaN stays one
                o1_st4((T *)a.out + pg_vec_at(a, x.row0, x.vec0 + v, g, a.os, a.dv) + c, make_float4(o.x * r, o.y * r, o.z * r, o.w * r));
            } else {
                *pg_val(parts, ps, RV, a.dv, v, c) = o;
                if (c == 0) *(float2 *)(parts.stat + (ps * RV + v) * 2) = make_float2(mx, sum);
            }
        }
        if (tid == 0 && first_seg) pg_head<Plan>(&parts.head[blockIdx.x], share, seg);
        first_seg = false;
    }
}

// The partial results of a unit that borders cut, added up by the blocks of the
// first border inside it, eight parts (four) in flight: what it takes is the
// latency of three loads one behind the other.
constexpr int JOIN = 256, JOIN_MANY = 128;   // threads, of few and of many vectors
struct Sum {
    float m, l;
    float4 o;
    __device__ __forceinline__ void add(float2 st, float4 y) {
        const float mn = fmaxf(m, st.x);
        const float f = m > -INFINITY ? exp2f(m - mn) : 0.f, h = st.x > -INFINITY ? exp2f(st.x - mn) : 0.f;
        m = mn;
        l = l * f + st.y * h;
        o.x = o.x * f + y.x * h;
        o.y = o.y * f + y.y * h;
        o.z = o.z * f + y.z * h;
        o.w = o.w * f + y.w * h;
    }
    __device__ __forceinline__ float4 result() const {
        const float r = l == 0.f ? 0.f : 1.f / l;   // a NaN stays one
        return make_float4(o.x * r, o.y * r, o.z * r, o.w * r);
    }
};
// Parts first, first + STEP, ... of columns c .. c + 3 of a vector.
template <int U, int STEP>
__device__ __forceinline__ Sum join_parts(const PgParts &parts, int border, int last, int first, int vecs, int dv, int v, int c) {
    Sum s = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int i0 = border - 1 + first; i0 <= last; i0 += U * STEP) {
        float2 st[U];
        float4 y[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * STEP;
            const size_t ps = i == border - 1 ? 2 * (size_t)i + 1 : 2 * (size_t)i;
            if (i <= last) st[u] = *(const float2 *)(parts.stat + (ps * vecs + v) * 2), y[u] = *pg_val(parts, ps, vecs, dv, v, c);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * STEP <= last) s.add(st[u], y[u]);
    }
    return s;
}
// Few vectors, maybe many parts: a vector a block, TPV threads its columns, the
// parts dealt to JOIN / TPV groups of them.
template <typename T, int TPV>
__global__ __launch_bounds__(JOIN) void k_pg_join_few(PgArgs a, int room, int vecs) {
    constexpr int GROUPS = JOIN / TPV;
    __shared__ Sum part[JOIN];
    o1_chain_wait();
    const int border = blockIdx.x + 1, grp = threadIdx.x / TPV, c = 4 * (threadIdx.x % TPV), v = blockIdx.y;
    const PgParts parts = pg_parts(a.part, room, vecs);
    const PgHead h = parts.head[border];
    if (h.last < 0 || v >= h.nv) return;
    Sum s = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    if (c < a.dv) s = join_parts<8, GROUPS>(parts, border, h.last, grp, vecs, a.dv, v, c);
    part[threadIdx.x] = s;
    __syncthreads();
    if (grp || c >= a.dv) return;
    for (int g = 1; g < GROUPS; ++g) {
        const Sum &o = part[g * TPV + threadIdx.x];
        s.add(make_float2(o.m, o.l), o.o);
    }
    o1_st4((T *)a.out + pg_vec_at(a, h.row0, h.vec0 + v, h.g, a.os, a.dv) + c, s.result());
}
// Many vectors: a block takes 32 vectors and 16 columns, a lane a vector and a warp
// 4 columns; the rows go out through shared memory. (A block that took all
// columns of its vectors left the sum of a few units' many parts to few of them:
// 64 bf16 rows behind 16000, 4 groups of 4 heads of 128, 53 us; 35 with 32 columns,
// 33 with 16, 37 with 8.)
template <typename T>
__global__ __launch_bounds__(JOIN_MANY) void k_pg_join(PgArgs a, int room, int vecs) {
    constexpr int W = JOIN_MANY / 32;
    __shared__ float4 rows[32][W + 1];
    o1_chain_wait();
    const int border = blockIdx.x + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, v0 = 32 * blockIdx.y, v = v0 + lane;
    const PgParts parts = pg_parts(a.part, room, vecs);
    const PgHead h = parts.head[border];
    if (h.last < 0 || v0 >= h.nv) return;
    const int r = threadIdx.x / W, k = threadIdx.x % W;
    const int c0 = 4 * W * blockIdx.z, c = c0 + 4 * warp;
    if (v < h.nv && c < a.dv) rows[lane][warp] = join_parts<8, 1>(parts, border, h.last, 0, vecs, a.dv, v, c).result();
    __syncthreads();
    if (v0 + r < h.nv && c0 + 4 * k < a.dv)
        o1_st4((T *)a.out + pg_vec_at(a, h.row0, h.vec0 + v0 + r, h.g, a.os, a.dv) + c0 + 4 * k, rows[r][k]);
}
template <typename T>
void join_launch(const PgArgs &a, int blocks, int room, int vecs, int most, cudaStream_t st) {
    const dim3 few(blocks - 1, most), many(blocks - 1, (vecs + 31) / 32, (a.dv + JOIN_MANY / 8 - 1) / (JOIN_MANY / 8));
    if (vecs > PG_ROWS_V) o1_launch_chained(true, k_pg_join<T>, many, dim3(JOIN_MANY), 0, st, a, room, vecs);
    else if (a.dv <= 64) o1_launch_chained(true, k_pg_join_few<T, 16>, few, dim3(JOIN), 0, st, a, room, vecs);
    else if (a.dv <= 128) o1_launch_chained(true, k_pg_join_few<T, 32>, few, dim3(JOIN), 0, st, a, room, vecs);
    else o1_launch_chained(true, k_pg_join_few<T, 64>, few, dim3(JOIN), 0, st, a, room, vecs);
}

template <typename T, typename C, int N>
cudaError_t rows_launch_n(const PgArgs &a, int dtype, const PgTable *tab, int units, int most, int64_t cost, cudaStream_t st) {
    using Z = Sizes<C, N, Types<T, C>::TERMS>;
    static_assert(sizeof(PgHead) == 32, "headers of 8 words");
    static unsigned long long done = 0;
    unsigned long long bit = 0;
    auto *k = k_pg_rows<T, C, N>;
    if (o1_attrs_needed(&done, &bit)) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Z::SMEM);
        if (e != cudaSuccess) return e;
        o1_attrs_done(&done, bit);
    }
    PgTable none;
    none.n = 0;
    const int blocks = (int)std::min<int64_t>(BLOCKS, std::max<int64_t>(1, cost / Plan::LEAST));
    k<<<blocks, RT, Z::SMEM, st>>>(a, tab ? *tab : none, units);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess && blocks > 1 ? pg_launch_join(a, dtype, blocks, BLOCKS, RV, most, st) : e;
}
template <typename T, typename C>
cudaError_t rows_launch_c(const PgArgs &a, int dtype, const PgTable *tab, int units, int most, int64_t cost, cudaStream_t st) {
    const int w = a.d > a.dv ? a.d : a.dv;
    if (w <= 64) return rows_launch_n<T, C, 1>(a, dtype, tab, units, most, cost, st);
    if (w <= 128) return rows_launch_n<T, C, 2>(a, dtype, tab, units, most, cost, st);
    return rows_launch_n<T, C, 4>(a, dtype, tab, units, most, cost, st);
}

}  // namespace

size_t pg_rows_scratch(int dv) { return pg_parts_bytes(BLOCKS, RV, dv); }

cudaError_t pg_launch_join(const PgArgs &a, int dtype, int blocks, int room, int vecs, int most, cudaStream_t st) {
    if (dtype == O1_F32) join_launch<float>(a, blocks, room, vecs, most, st);
    else if (dtype == O1_BF16) join_launch<__nv_bfloat16>(a, blocks, room, vecs, most, st);
    else join_launch<__half>(a, blocks, room, vecs, most, st);
    return cudaGetLastError();
}

cudaError_t pg_launch_rows(const PgArgs &a, int dtype, int cache_dtype, const PgTable *tab, cudaStream_t st) {
    const int units = tab ? tab->total : a.rows;
    int most = tab ? 1 : a.hpg;   // vectors of a unit
    if (tab)
        for (int i = 0; i < tab->n && most < RV; ++i) most = (int)std::max<int64_t>(most, std::min<int64_t>(RV, (int64_t)tab->s[i].rows * a.hpg));
    // What the call can cost (pg_share): no more blocks than get a share of it.
    // (Those without one are not free: one row at 8191 of the heads above, where 133 of
    // 304 blocks have a share, took 19.7 us with all of them and 18.4 without; over
    // e4m3 21.7 and 19.2.)
    auto cost_of = [&](int64_t n, int lo, int hi) { return n * (hi / TILE - lo / TILE + 1 + Plan::START) * a.G; };
    int64_t cost = 0;
    if (tab) {
        for (int i = 0; i < tab->n; ++i) {
            const PgSeq &s = tab->s[i];
            cost += cost_of((i + 1 < tab->n ? tab->s[i + 1].before : tab->total) - s.before, a.window ? std::max(0, s.pos0 - a.window + 1) : 0,
                            s.pos0 + s.rows - 1);
        }
    } else {
        const int64_t len = (int64_t)a.width << a.lpage;   // the window anywhere in it: a tile more
        cost = cost_of(units, 0, (int)std::min<int64_t>(len - 1, a.window ? (int64_t)a.window - 1 + TILE : len - 1));
    }
    if (dtype == O1_F32 && cache_dtype == O1_BF16) return rows_launch_c<float, __nv_bfloat16>(a, dtype, tab, units, most, cost, st);
    if (dtype == O1_F32) return rows_launch_c<float, uint8_t>(a, dtype, tab, units, most, cost, st);
    if (dtype == O1_BF16 && cache_dtype == O1_BF16) return rows_launch_c<__nv_bfloat16, __nv_bfloat16>(a, dtype, tab, units, most, cost, st);
    if (dtype == O1_BF16) return rows_launch_c<__nv_bfloat16, uint8_t>(a, dtype, tab, units, most, cost, st);
    if (cache_dtype == O1_F16) return rows_launch_c<__half, __half>(a, dtype, tab, units, most, cost, st);
    return rows_launch_c<__half, uint8_t>(a, dtype, tab, units, most, cost, st);
}
