// Attention of many query vectors over the paged cache, on the tensor cores
// (tcgen05, accumulators in TMEM). The query heads of a group share its keys, so
// a tile is 128 query vectors (rows times heads of the group) against 128 keys:
//   S = Q K^T, P = e^{S - m}, O += P V
// with a running reference m a row near the row's maximum (O is rescaled only when
// the maximum passes it by 2^8; see PgReference), P written over S in TMEM.
//
// A block takes segments of units (o1_page.cuh), one block an SM:
//   warps 0-7   softmax: a thread a row; two query tiles (QT = 2: rows of up to
//               128 values), a warpgroup each, in turn on the tensor cores, or
//               one tile with two score buffers and a warpgroup on either half
//               of its keys (QT = 1)
//   warps 8-11  producers: queries, keys and values into shared memory, 128-byte
//               swizzled. 16-bit caches: the tiles that lie wholly in a sequence
//               and on pages in TMA boxes, the warps in turn; others by 16-byte
//               asynchronous copies (pages end anywhere on 16 positions; what no
//               row attends is zero-filled, not read). e4m3: codes, converted
//               to bf16 values under their row's power of two (exact)
//   warp 12     issues the MMAs (QT = 2: warps 12 and 13, a query tile each)
//   warp 14     e4m3: brings the codes
// Keys come as items of 128 keys x 128 columns, values as 128 keys x 128 columns
// or 64 x 256: 32 KB slots of one ring, in the order of use.
//
// Bound: rows of 128, the weights' formation. Two tiles of 128 x 128 scores take
// the tensor cores 2150 cycles and their softmax warps about 4000 (an element is
// one exponential and three other operations; they are formed by the tiles'
// warps half a turn apart, which took 9 % less than all at once). 8192 bf16 rows
// of 4 groups of 4 heads of 128, cache empty before: 256 us, 1070 TFLOP/s. Rows of
// 256 have twice the products to a weight, and the tensor cores are the bound:
// 4096 bf16 rows of 2 groups of 4 heads behind 12288: 317 us, 1520 TFLOP/s. (All
// times here are of replayed graphs; in a loop of calls these two take 256 and 338.)
// Producers: a slot's wait, its arrival and its copies are a chain of single
// instructions, and one warp that also formed the addresses there (453 us) was
// the bound of the latter. (Pairs of blocks that load each key tile once for
// both were no faster.) e4m3: the conversion, 2100 cycles a 16 KB item of codes; 2047
// bf16 rows and eight shorter sequences, 4 groups of 4 heads of 128: 79 us.
//
// Terms. As in o1_page_rows.cu: one for 16-bit rows over their own type and bf16
// over e4m3, two bf16 for fp16 over e4m3, three for fp32. For fp32 rows a tile's
// P V is an accumulation of its own, added to sums in registers with rounding:
// the MMA's accumulation truncates, the same way each time.
//
// Every wait is bounded; where one runs out the block raises a flag, writes NaN
// for what is left of its share, and ends once its copies and MMAs are over: the
// issuers wait for their MMAs, one thread at the end for the last copy of each
// barrier, as recorded where it was sent.
#include <math.h>

#include <type_traits>

#include "o1_page.cuh"
#include "o1_tc.cuh"

static __device__ uint32_t pg_device_flags;

namespace {

constexpr int KT = 128;                        // keys of a tile
constexpr int SM_WARPS = 8, PR_WARPS = 4;      // softmax and producer warps
constexpr int THREADS = 32 * (SM_WARPS + PR_WARPS + 4), SM_THREADS = 32 * SM_WARPS;
constexpr int SLOT = 32768, MAX_SLOTS = 6;
constexpr int BLOCKS = 152;
constexpr size_t SMEM = 225 * 1024;            // dynamic; static parts beside it

// A segment costs about two tiles beside its own (8192 bf16 rows: 306 us with
// START = 1, 259 with 2, 261 with 3, 263 with 4; the ragged e4m3 batch 90, 81, 82,
// 83), and a tile alone is worth a block: 300 and 77 fp16 rows of odd widths and a
// window took 21 us with LEAST = 1, 25 with 2, 28 with 4, 34 with 6.
template <int QT>
struct Plan {
    static constexpr int V = 128 * QT, K = KT, START = 2, LEAST = 1;
};

template <typename T, typename C>
struct Types {   // 16-bit rows over their own type
    using M = T;
    static constexpr int TERMS = 1;
};
template <>
struct Types<float, __nv_bfloat16> {
    using M = __nv_bfloat16;
    static constexpr int TERMS = 3;
};
template <>
struct Types<float, uint8_t> {
    using M = __nv_bfloat16;
    static constexpr int TERMS = 3;
};
template <>
struct Types<__nv_bfloat16, uint8_t> {
    using M = __nv_bfloat16;
    static constexpr int TERMS = 1;
};
template <>
struct Types<__half, uint8_t> {
    using M = __nv_bfloat16;
    static constexpr int TERMS = 2;
};

// Registers a thread. The block starts with 128, all of the SM's; each role's
// warpgroups then trade them: softmax (two warpgroups), producers, issuer.
constexpr int REGS = 128;
struct Regs {
    static constexpr int PRODUCER = 88, ISSUER = 72, SOFTMAX = 176;
    static_assert(2 * SOFTMAX + PRODUCER + ISSUER <= 4 * REGS, "no more than the block has");
};
template <int N>
__device__ __forceinline__ void regs_more() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_less() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// TMEM columns. QT = 2: scores of the two tiles at 0 and 128, outputs at 256 and
// 384. QT = 1: two score buffers, outputs behind them; a third term of P has 64
// columns more a buffer.
template <int TERMS>
struct Cols {
    static constexpr uint32_t STRIDE = TERMS == 3 ? 192 : 128, OUT = 2 * STRIDE;
    static __device__ __forceinline__ uint32_t score(int b) { return STRIDE * b; }
    static __device__ __forceinline__ uint32_t out(int tile) { return OUT + 128 * tile; }
    // A operand of 16 keys (step k of 8), term t. P lies over the scores of the
    // same keys: 64 keys' first 32 columns or, of several terms, 32 keys' first
    // and second 16; third terms behind the scores
    static __device__ __forceinline__ uint32_t p(int k, int t) {
        return TERMS == 1 ? 64 * (k >> 2) + 8 * (k & 3) : t < 2 ? 32 * (k >> 1) + 16 * t + 8 * (k & 1) : 128 + 8 * k;
    }
};

template <typename M>
__device__ __forceinline__ uint32_t idesc(int m, int n, int mn_b) {
    return (1u << 4) | (std::is_same<M, __nv_bfloat16>::value ? (1u << 7) | (1u << 10) : 0u) | ((uint32_t)mn_b << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
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
// (a, b) as packed M pair, and what it leaves of them
template <typename M>
__device__ __forceinline__ uint32_t take_m(float &a, float &b) {
    const uint32_t w = pack_m((const M *)nullptr, a, b);
    const float2 f = unpack_m((const M *)nullptr, w);
    a -= f.x;
    b -= f.y;
    return w;
}

// 16 bytes into shared memory, zeros where !on
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool on) {
    const int n = on ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void st16(uint32_t dst, const uint4 &v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void tma_2d_at(uint32_t dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"((uint64_t)map), "r"(x), "r"(y), "r"(su32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_3d_at(uint32_t dst, const CUtensorMap *map, int x, int y, int w, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"((uint64_t)map), "r"(x), "r"(y), "r"(w), "r"(su32(bar))
        : "memory");
}
// `bytes` (a multiple of 16) from a 16-byte boundary to another.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, int bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes),
                 "r"(su32(bar))
                 : "memory");
}
__device__ __forceinline__ uint4 ld16(uint32_t src) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(src) : "memory");
    return v;
}
// Byte of 16-byte piece p (0 to 7) of row r in a panel of 128-byte rows.
__device__ __forceinline__ uint32_t piece(int r, int p) { return (uint32_t)(128 * r + 16 * (p ^ (r & 7))); }

// 8 e4m3 codes as bf16 pairs times a power of two (a bf16 pair)
__device__ __forceinline__ uint4 bf16_of_e4m3(uint2 c, __nv_bfloat162 f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint16_t two = (uint16_t)((i < 2 ? c.x : c.y) >> (16 * (i & 1)));
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
        const float2 x = __half22float2(*(const __half2 *)&h);
        const __nv_bfloat162 y = __hmul2(__floats2bfloat162_rn(x.x, x.y), f);
        w[i] = *(const uint32_t *)&y;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Two fp32 values in a register pair: packed operations take one issue for both.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void f2_get(F2 x, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v)); }
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ float max3(float a, uint32_t b, uint32_t c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
    return r;
}

struct Shared {
    uint64_t full[MAX_SLOTS], empty[MAX_SLOTS];
    uint64_t raw_full[2], raw_empty[2];   // e4m3: items of codes to be converted
    uint64_t q_full, q_free;
    uint64_t s_full[2], p_full[4], pv_half[2], pv_done[2], o_free[2], fin;   // p_full: QT = 2, halves of keys of either tile
    long long share[THREADS / 32 + 2];
    uint64_t turn[2][4];   // QT = 2: the two tiles' warps of a scheduler form weights in turn
    alignas(16) uint8_t raw_exps[2][KT];  // their exponents
    uint32_t raw_there[2];                // their runs of 16 positions that have a page, a bit each
    // for the block's end after a wait that ran out: where TMA writes or wrote
    // last, 1 and the phase that this completes (0: nowhere): slots, queries, codes
    uint32_t sent[MAX_SLOTS], sent_q, sent_raw[2];
    uint32_t tslot;
    int abort;
    float half[2][128];   // QT = 1: the warpgroups' maxima, then sums
};
static_assert(sizeof(Shared) <= 2048, "static and dynamic shared memory in 227 KB");
// Announces `bytes` of TMA at a barrier, whose phase they complete.
__device__ __forceinline__ void expect_tx(uint64_t *bar, uint32_t &sent, uint32_t phase, int bytes) {
    sent = 1 + phase;
    mbar_expect_tx(bar, bytes);
}
// Waits until what TMA was last told to write is written.
__device__ __forceinline__ void drain(uint64_t *bar, uint32_t sent) {
    if (sent) mbar_drain(bar, sent - 1);
}

// Sizes of a call, the same in every role.
struct Shape {
    int nqc;       // 64-column blocks of Q and K
    int ksteps;    // k16 steps of a score
    int k_items;   // items of a key tile (128 columns each)
    int v_keys;    // keys of a value item
    int v_items;
    int nv;        // value columns, rounded to 16
    int nslot;
    int raw;       // bytes of the queries, behind which codes to be converted lie, and then the ring
};
constexpr int RAW_ITEM = 16384, RAW_BYTES = 2 * RAW_ITEM;
template <int QT, int TERMS, bool E4>
__device__ __forceinline__ Shape shape_of(int d, int dv) {
    Shape s;
    s.nqc = (d + 63) / 64;
    s.ksteps = (d + 15) / 16;
    s.k_items = (d + 127) / 128;
    s.v_keys = dv > 128 ? 64 : 128;
    s.v_items = dv > 128 ? 2 : 1;
    s.nv = (dv + 15) / 16 * 16;
    s.raw = TERMS * QT * s.nqc * 16384;
    s.nslot = min(MAX_SLOTS, (int)((SMEM - 1024 - s.raw - (E4 ? RAW_BYTES : 0)) / SLOT));   // 3 at least (fp16 over e4m3, d > 128: 2)
    return s;
}

// A ring position.
struct Ring {
    int slot;
    uint32_t phase;
    __device__ __forceinline__ void next(int n) {
        if (++slot == n) slot = 0, phase ^= 1;
    }
};

__device__ __forceinline__ void sm_sync() { asm volatile("bar.sync 1, %0;" ::"n"(SM_THREADS) : "memory"); }
// the softmax warps' barrier that says whether any thread had `p`
__device__ __forceinline__ bool sm_or(bool p) {
    int r;
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.s32 p, %1, 0;\nbar.red.or.pred q, 1, %2, p;\nselp.s32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"((int)p), "n"(SM_THREADS)
        : "memory");
    return r != 0;
}

// ---------------------------------------------------------------- producers

template <typename T, typename C, int QT>
struct Producer {
    using M = typename Types<T, C>::M;
    static constexpr int TERMS = Types<T, C>::TERMS;
    static constexpr bool E4 = sizeof(C) == 1, Q_COPY = TERMS == 1 && sizeof(T) == 2;
    const PgArgs &a;
    Shared &sh;
    const Shape &z;
    uint32_t q0, ring0;   // shared addresses
    int lane, r4, l8;     // r4: this thread's row of each 16, l8: its place among the 8 threads of a row
    const CUtensorMap *mq, *mk, *mv;   // for TMA: queries (null: not in boxes), and the pools of a 16-bit cache
    int qrows;            // rows of a query box
    int wid;              // this warp among the producers
    Ring put;             // slot of the next item
    bool ok;

    // 16-bit caches: the warps take the items that come in boxes in turn, each
    // waiting for its own (`met`: its waits were met so far); where all four copy,
    // the first waits, a barrier before says whether any wait ran out (`ok`), and
    // one after lets the first announce. e4m3: every warp waits and arrives for
    // itself.
    bool met;
    uint32_t items;       // items so far
    uint32_t qp;          // phase of q_free
    __device__ __forceinline__ bool master() const { return wid == 0; }
    __device__ __forceinline__ void sync() { asm volatile("bar.sync 2, %0;" ::"n"(32 * PR_WARPS) : "memory"); }
    __device__ __forceinline__ bool any_of(bool p) {   // of the producers' threads
        int r;
        asm volatile(
            "{\n.reg .pred p, q;\nsetp.ne.s32 p, %1, 0;\nbar.red.or.pred q, 2, %2, p;\nselp.s32 %0, 1, 0, q;\n}\n"
            : "=r"(r)
            : "r"((int)p), "n"(32 * PR_WARPS)
            : "memory");
        return r != 0;
    }
    __device__ __forceinline__ void agree() { ok = !any_of(!met); }
    __device__ __forceinline__ void wait_for(uint64_t *bar, uint32_t parity) { met = met && warp_wait(bar, parity, &sh.abort, a.wait_cycles); }
    // all warps' copies are in shared memory
    __device__ __forceinline__ void announce(uint64_t *bar) {
        copy_commit();
        copy_wait<0>();
        fence_async_smem();
        if (E4) __syncwarp();
        else sync();
        if (lane == 0 && (E4 || master())) mbar_arrive(bar);
    }

    // The query tiles: row v of the unit's vectors, its values as terms. Where
    // a group's heads are a power of two, a tile's vectors are whole rows of heads
    // and come as boxes (rows past the sequence's are not used).
    __device__ __forceinline__ void queries(const PgSegment &s) {
        const int tiles = QT == 2 && s.x.nv > 128 ? 2 : 1, pieces = 2 * z.ksteps;   // 16-byte pieces of a row
        if (Q_COPY && mq) {
            const int n = z.nqc * tiles;
            if (master() && (E4 ? ok : met)) {
                if (lane == 0) expect_tx(&sh.q_full, sh.sent_q, qp, 16384 * n);
                __syncwarp();
                if (lane < n) {
                    const int tile = lane / z.nqc, c = lane - tile * z.nqc;
                    tma_3d_at(q0 + 16384 * lane, mq, 64 * c, s.g * a.hpg, s.x.row0 + s.x.vec0 / a.hpg + tile * qrows, &sh.q_full);
                }
                __syncwarp();
            }
            return;
        }
        if (!E4) {
            agree();
            if (!ok) return;
        }
        constexpr int U = TERMS == 1 ? 4 : 2;   // rows in flight
#pragma unroll 1
        for (int r0 = 0; r0 < 128 * tiles; r0 += 16 * U) {
            const T *src[U];
            bool in[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int v = r0 + 16 * u + r4;
                in[u] = v < s.x.nv;
                src[u] = (const T *)a.q + (in[u] ? pg_vec_at(a, s.x.row0, s.x.vec0 + v, s.g, a.qs, a.d) : 0) + 8 * l8;
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int p = 8 * c + l8;
                if (8 * c >= pieces) break;
                if constexpr (Q_COPY) {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int v = r0 + 16 * u + r4;
                        const bool on = in[u] && 8 * p < a.d;
                        if (p < pieces)
                            copy16(q0 + (uint32_t)((v >> 7) * z.nqc + c) * 16384 + piece(v & 127, l8), on ? (const void *)(src[u] + 64 * c) : a.q, on);
                    }
                } else {
                    float4 f[U][2];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        f[u][0] = f[u][1] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (in[u] && 8 * p < a.d) f[u][0] = o1_ld4(src[u] + 64 * c), f[u][1] = o1_ld4(src[u] + 64 * c + 4);
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int v = r0 + 16 * u + r4;
                        float x[8] = {f[u][0].x, f[u][0].y, f[u][0].z, f[u][0].w, f[u][1].x, f[u][1].y, f[u][1].z, f[u][1].w};
#pragma unroll
                        for (int t = 0; t < TERMS; ++t) {
                            uint32_t w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) w[i] = take_m<M>(x[2 * i], x[2 * i + 1]);
                            if (p < pieces)
                                st16(q0 + (uint32_t)((t * QT + (v >> 7)) * z.nqc + c) * 16384 + piece(v & 127, l8),
                                     make_uint4(w[0], w[1], w[2], w[3]));
                        }
                    }
                }
            }
        }
        announce(&sh.q_full);
    }

    // The table's entries for a tile's eight runs of 16 positions, run i in lanes
    // i, i + 8, ...; and an entry's page, or -1. They are apart, for an entry is
    // looked up a tile ahead and would be waited for where it is first compared.
    __device__ __forceinline__ int entries(const PgSegment &s, int j) const {
        const int p = (s.x.lo / KT + j) * KT + 16 * (lane & 7);
        return j < s.t1 && p <= s.x.last && p + 15 >= s.x.first ? a.table[(size_t)s.x.slot * a.width + (p >> a.lpage)] : -1;
    }
    __device__ __forceinline__ int page_of(int entry) const { return entry >= 0 && entry < a.n_pages ? entry : -1; }

    // An item of the tile: keys (128 columns) or values (v_keys rows). 16 rows
    // at a time; a thread has the same row of each 16.
    // By TMA where every position of it is in the sequence and on a page: a lane
    // a box of the item's rows on one page and 64 columns (at most 16).
    template <bool KEYS>
    __device__ __forceinline__ void item(const PgSegment &s, int j, int ids, int part, bool boxes) {
        if (!ok) return;
        const bool split = QT == 1 && !KEYS && z.v_keys == 64;
        const int width = KEYS ? a.d : a.dv, col0 = QT == 1 && KEYS ? 128 * part : 0, key0 = split ? 64 * part : 0;
        const int rows = split ? 64 : 128, runs = rows / 16;
        const int cols = min(split ? 256 : 128, (width + 15) / 16 * 16 - col0);   // to be filled
        const int p0 = (s.x.lo / KT + j) * KT + key0;
        const uint32_t dst = ring0 + put.slot * SLOT;
        const C *pool = (const C *)(KEYS ? a.k : a.v);
        uint64_t *full = &sh.full[put.slot];
        if constexpr (!E4) {
            if (boxes) {
                // all but the wait and the copies is done before the slot is free
                const int blocks = (cols + 63) / 64, lb = split ? 2 : 1, lrows = min(a.lpage, split ? 6 : 7);   // rows of a box
                const int b = lane & ((1 << lb) - 1), key = (lane >> lb) << lrows, x = col0 + 64 * b;
                const bool on = b < blocks && key < rows;
                const int page = __shfl_sync(0xffffffffu, ids, (key0 + key) / 16 & 7);
                const int y = ((page * a.G + s.g) << a.lpage) + (p0 + key & ((1 << a.lpage) - 1));
                const uint32_t at = dst + (b * rows + key) * 128;
                if ((items++ & (PR_WARPS - 1)) == wid) {
                    wait_for(&sh.empty[put.slot], put.phase ^ 1);
                    if (met) {
                        if (lane == 0) expect_tx(full, sh.sent[put.slot], put.phase, blocks * rows * 128);
                        __syncwarp();
                        if (on) tma_2d_at(at, KEYS ? mk : mv, x, y, full);
                        __syncwarp();
                    }
                }
                put.next(z.nslot);
                return;
            }
            if (master()) wait_for(&sh.empty[put.slot], put.phase ^ 1);
            agree();
            if (!ok) return;
            if (master() && lane == 0) sh.sent[put.slot] = 0;   // the boxes before were used
            constexpr int U = 4;   // runs in flight
#pragma unroll 1
            for (int i0 = 0; i0 < runs; i0 += U) {
                const C *src[U];
                bool in[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int page = __shfl_sync(0xffffffffu, ids, key0 / 16 + i0 + u), p = p0 + 16 * (i0 + u) + r4;
                    in[u] = page >= 0 && p >= s.x.lo && p <= s.x.hi;
                    src[u] = pg_at(pool, a, max(page, 0), s.g, p & ((1 << a.lpage) - 1), width) + col0 + 8 * l8;
                }
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const int c = 64 * b + 8 * l8;
                    if (64 * b >= cols) break;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const bool on = in[u] && col0 + c < width;
                        if (c < cols) copy16(dst + b * (rows * 128) + piece(16 * (i0 + u) + r4, l8), on ? src[u] + 64 * b : pool, on);
                    }
                }
            }
        }
        announce(full);
        put.next(z.nslot);
    }

    // e4m3. A warp of its own, the loader, brings codes and exponents by bulk
    // copies, 16 rows a lane and two items ahead; each of the four producer warps
    // converts a quarter of an item's rows. An item of codes is 128 rows of up to
    // 128 values, or 64 of up to 256: two of such keys fill two slots together.
    struct Item {
        bool keys;
        int j, part;
    };
    uint32_t raw0;   // shared address of the two buffers of codes
    __device__ __forceinline__ bool halves(const Item &x) const { return QT == 1 && (x.keys ? a.d : a.dv) > 128; }
    __device__ __forceinline__ int key0_of(const Item &x) const { return QT == 2 ? 0 : 64 * x.part; }
    // in the MMA issuer's order: QT = 1 runs a tile's scores ahead; false after the last
    __device__ __forceinline__ bool next(const PgSegment &s, Item &i) const {
        if (QT == 1 && ++i.part < (i.keys ? z.k_items : z.v_items)) return true;
        i.part = 0;
        if (QT == 2) {
            if (!i.keys) ++i.j;
            i.keys = !i.keys;
        } else if (i.keys) {
            if (i.j == s.t0 && i.j + 1 < s.t1) ++i.j;   // the second tile's keys
            else if (i.j == s.t0) i.keys = false;
            else i.keys = false, --i.j;
        } else {
            i.j += 2;
            i.keys = i.j < s.t1;
            if (!i.keys) --i.j;                           // no keys are left: the next values
        }
        return i.j < s.t1;
    }
    __device__ __forceinline__ void load_codes(const PgTable &tab, int units, PgShare share) {
        PgSegment s;
        uint32_t n = 0;   // items
        while (ok && pg_next<Plan<QT>>(a, tab, units, share, s)) {
            // pages of tiles t and on, t the last one whose values are to come
            int tile = s.t0, ids = page_of(entries(s, tile)), ids1 = page_of(entries(s, tile + 1)), next2 = entries(s, tile + 2);
            Item x = {true, s.t0, 0};
            do {
                while (tile + 1 < x.j || (tile < x.j && !x.keys)) {
                    ++tile;
                    ids = ids1;
                    ids1 = page_of(next2);
                    next2 = entries(s, tile + 2);
                }
                const int b = n & 1;
                ok = warp_wait(&sh.raw_empty[b], ((n >> 1) & 1) ^ 1, &sh.abort, a.wait_cycles);
                if (!ok) break;
                const int width = x.keys ? a.d : a.dv, key0 = key0_of(x), runs = halves(x) ? 4 : 8, mask = (1 << a.lpage) - 1;
                const int p0 = (s.x.lo / KT + x.j) * KT, page = x.j == tile ? ids : ids1;
                const uint32_t there = __ballot_sync(0xffffffffu, page >= 0) >> (key0 / 16) & ((1u << runs) - 1);
                if (lane == 0) {
                    sh.raw_there[b] = there;
                    expect_tx(&sh.raw_full[b], sh.sent_raw[b], (n >> 1) & 1, __popc(there) * 16 * (width + 1));
                }
                __syncwarp();
                const C *pool = (const C *)(x.keys ? a.k : a.v);
                const uint32_t dst = raw0 + b * RAW_ITEM;
                // lanes 0 to 7: 16 rows of codes each; 8 to 15: of exponents
                const int run = lane & 7, id = __shfl_sync(0xffffffffu, page, key0 / 16 + run & 7);
                const uint32_t row = (uint32_t)(((id * a.G + s.g) << a.lpage) + (p0 + key0 + 16 * run & mask));
                if (lane < 16 && there >> run & 1) {
                    if (lane < 8) bulk_load(dst + 16 * run * width, pool + (size_t)row * width, 16 * width, &sh.raw_full[b]);
                    else bulk_load(su32(sh.raw_exps[b]) + 16 * run, (x.keys ? a.ke : a.ve) + row, 16, &sh.raw_full[b]);
                }
                __syncwarp();
                ++n;
            } while (next(s, x));
        }
    }
    // Four threads cover the 64 columns of a block, and the 8 of a row write their
    // two pieces in opposite orders, so that no bank is hit twice.
    __device__ __forceinline__ void convert(const PgSegment &s, const Item &x, uint32_t n) {
        const int b = n & 1;
        const bool two = halves(x), pair = two && x.keys, open = !pair || x.part == 0, shut = !pair || x.part == 1;
        Ring second = put;   // of a pair of slots
        second.next(z.nslot);
        if (open) ok = ok && warp_wait(&sh.empty[put.slot], put.phase ^ 1, &sh.abort, a.wait_cycles);
        if (open && pair) ok = ok && warp_wait(&sh.empty[second.slot], second.phase ^ 1, &sh.abort, a.wait_cycles);
        ok = ok && warp_wait(&sh.raw_full[b], (n >> 1) & 1, &sh.abort, a.wait_cycles);
        if (!ok) return;
        const int width = x.keys ? a.d : a.dv, rows = two ? 64 : 128, key0 = key0_of(x), cols = (width + 15) / 16 * 16;
        const int odd = (l8 >> 2) & 1, p = 2 * (l8 & 3), row0 = (two ? 16 : 32) * wid + (lane >> 3);
        const int from = (s.x.lo / KT + x.j) * KT + key0;   // position of row 0
        const uint32_t src = raw0 + b * RAW_ITEM + row0 * width + 16 * l8, there = sh.raw_there[b];
        const uint32_t dst = ring0 + put.slot * SLOT, block = (pair ? 128 : rows) * 128;
        // columns of 128 and on: the same slot's next blocks, or a pair's second slot
        const uint32_t dst1 = pair ? ring0 + second.slot * SLOT : dst + 2 * block;
        const bool all = there == (two ? 15 : 255) && from >= s.x.lo && from + rows - 1 <= s.x.hi;
        // pieces in flight: more of them make the loop too long for the instruction
        // caches (the ragged batch took 89 us with 8, 80 with 4, 79 with 2, 81 with 1)
        constexpr int U = 2;
#pragma unroll 1
        for (int i0 = 0; i0 < 8; i0 += U) {
            uint4 w[U];
            uint32_t f[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u, row = row0 + 4 * (i >> two);
                f[u] = sh.raw_exps[b][row];
                w[u] = ld16(src + 4 * width * (i >> two) + (two ? 128 * (i & 1) : 0));
            }
            if (!all) {   // where no row attends it, memory may hold anything
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int row = row0 + 4 * ((i0 + u) >> two);
                    if (!(there >> (row >> 4) & 1) || from + row < s.x.lo || from + row > s.x.hi) w[u] = make_uint4(0u, 0u, 0u, 0u), f[u] = 0;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u, row = row0 + 4 * (i >> two), c = 16 * l8 + (two ? 128 * (i & 1) : 0);
                if (c < cols) {
                    const uint32_t f2 = f[u] * 0x00800080u;   // 2^(byte - 127) twice
                    const uint32_t at = (c >= 128 ? dst1 : dst) + (c >> 6 & 1) * block + (pair ? 64 * 128 * x.part : 0);
                    const __nv_bfloat162 fb = *(const __nv_bfloat162 *)&f2;
                    const uint4 lo = bf16_of_e4m3(make_uint2(w[u].x, w[u].y), fb), hi = bf16_of_e4m3(make_uint2(w[u].z, w[u].w), fb);
                    st16(at + piece(row, p + odd), odd ? hi : lo);
                    st16(at + piece(row, p + 1 - odd), odd ? lo : hi);
                }
            }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&sh.raw_empty[b]);
            if (shut) mbar_arrive(&sh.full[put.slot]);
            if (shut && pair) mbar_arrive(&sh.full[second.slot]);
        }
        if (!shut) return;
        put.next(z.nslot);
        if (pair) put.next(z.nslot);
    }
    __device__ __forceinline__ void run_codes(const PgTable &tab, int units, PgShare share) {
        PgSegment s;
        uint32_t n = 0;   // items
        while (ok && pg_next<Plan<QT>>(a, tab, units, share, s)) {
            Item x = {true, s.t0, 0};
            convert(s, x, n++);   // before the queries, whose place the segment before may still hold
            ok = ok && warp_wait(&sh.q_free, qp, &sh.abort, a.wait_cycles);
            if (!ok) break;
            qp ^= 1;
            queries(s);
            while (ok && next(s, x)) convert(s, x, n++);
        }
    }

    __device__ __forceinline__ void run(const PgTable &tab, int units, PgShare share) {
        if constexpr (E4) run_codes(tab, units, share);
        else run_rows(tab, units, share);
    }
    __device__ __forceinline__ void run_rows(const PgTable &tab, int units, PgShare share) {
        PgSegment s;
        while (ok && pg_next<Plan<QT>>(a, tab, units, share, s)) {
            // a tile of a 16-bit cache comes in boxes where some row of the
            // sequence attends every position of it (outside, memory may hold
            // anything); the warps decide together, whatever each read of the table.
            // Once a wait of any of them ran out no tile does, and the copies' vote
            // on their wait ends the loops of all: none walks the rest of the share,
            // past slots that another one skipped and whose phases are one behind.
            // (Such a slot, a ring later, could look free to a warp that had met no
            // wait between. Rings of 16-bit caches have four slots at least, so
            // that every warp has a wait of its own between.)
            auto boxes = [&](int j, int id) -> bool {
                if (E4 || j >= s.t1) return false;
                const int x0 = (s.x.lo / KT + j) * KT;
                return !any_of(!(met && x0 >= s.x.first && x0 + KT - 1 <= s.x.last && __all_sync(0xffffffffu, id >= 0)));
            };
            // in the MMA issuer's order: QT = 1 runs a tile's scores ahead
            auto keys = [&](int j, int id, bool bx) {
                for (int p = 0; ok && p < z.k_items; ++p) item<true>(s, j, id, p, bx);
            };
            auto values = [&](int j, int id, bool bx) {
                for (int p = 0; ok && p < z.v_items; ++p) item<false>(s, j, id, p, bx);
            };
            int ids = page_of(entries(s, s.t0)), ids1 = page_of(entries(s, s.t0 + 1));
            bool bx = boxes(s.t0, ids), bx1;
            keys(s.t0, ids, bx);   // before the queries, whose place the segment before may still hold
            if (master()) wait_for(&sh.q_free, qp);
            if (!ok) break;
            qp ^= 1;
            queries(s);
            for (int j = s.t0; ok && j < s.t1; ++j) {
                const int next2 = entries(s, j + 2);
                bx1 = boxes(j + 1, ids1);
                if (QT == 1 && j + 1 < s.t1) keys(j + 1, ids1, bx1);
                values(j, ids, bx);
                if (QT == 2 && j + 1 < s.t1) keys(j + 1, ids1, bx1);
                ids = ids1;
                ids1 = page_of(next2);
                bx = bx1;
            }
        }
    }
};

// ------------------------------------------------------------- MMA issuer

// The MMAs of n k16 steps of a score, and of 64 keys of P V. The whole warp takes
// the loops and the elected lane (`e`) the MMAs, with carried operands: warp-
// uniform control flow keeps them in uniform registers, and an MMA issues at
// its rate (from one lane's unrolled branch a step of 32 took 3700 cycles).
__device__ __forceinline__ void run_ss(bool e, uint32_t col, uint64_t qd, uint64_t kd, uint32_t id, int n, uint32_t acc) {
#pragma unroll 1
    for (; n > 0; n -= 4, qd += 1024, kd += 1024) {   // a 64-column block
        uint64_t q = qd, k = kd;
#pragma unroll 1
        for (int x = min(4, n); x > 0; --x) {
            if (e) mma_ss(col, q, k, id, acc);
            q += 2;
            k += 2;
            acc = 1;
        }
    }
}
// N terms 16 columns apart; STEP: columns from an odd step of 16 keys to the next.
template <int N, int STEP>
__device__ __forceinline__ void run_ts(bool e, uint32_t out, uint32_t p, uint64_t vd, uint32_t id, uint32_t acc) {
#pragma unroll 1
    for (int x = 0; x < 4; ++x) {
#pragma unroll
        for (int m = N - 1; m >= 0; --m) {
            if (e) mma_ts(out, p + 16 * m, vd, id, acc);
            acc = 1;
        }
        p += x & 1 ? STEP : 8;
        vd += 128;
    }
}

// QT = 2: a warp for either query tile, so that what stands between one's MMAs
// (waits, fences, commits) runs under the other's. A tile: S | PV S' | PV' S'' ...
// A ring slot is free once both have used it.
template <typename T, typename C>
__device__ __forceinline__ void issuer_of(int tile, const PgArgs &a, Shared &sh, const Shape &z, uint32_t q0, uint32_t ring0,
                                          uint32_t tmem, const PgTable &tab, int units, PgShare share) {
    using M = typename Types<T, C>::M;
    using Col = Cols<1>;
    const bool e = elect_one();
    const uint64_t dq = desc_sw128(q0) + (uint64_t)(tile * z.nqc * 1024), dk = desc_sw128(ring0), dv = desc_sw128_mn(ring0, KT * 128);
    const uint32_t id_s = idesc<M>(128, KT, 0), id_o = idesc<M>(128, z.nv, 1);
    const uint32_t sc = tmem + Col::score(tile), out = tmem + Col::out(tile);
    const long long wl = a.wait_cycles;
    bool ok = true;
    Ring get = {0, 0};
    uint32_t qp = 0, n = 0, nseg = 0;   // phase of q_full; tiles; segments of this query tile
    PgSegment s;
    auto commit = [&](uint64_t *bar) {
        if (e) mma_commit(bar);
    };
    auto item = [&]() -> bool {   // the next one is here
        ok = ok && warp_wait(&sh.full[get.slot], get.phase, &sh.abort, wl);
        tc_after();
        return ok;
    };
    auto scores = [&]() {
        if (!item()) return;
        run_ss(e, sc, dq, dk + (uint64_t)(get.slot * (SLOT / 16)), id_s, z.ksteps, 0);
        commit(&sh.s_full[tile]);
        commit(&sh.empty[get.slot]);
        get.next(z.nslot);
    };
    while (ok && pg_next<Plan<2>>(a, tab, units, share, s)) {
        ok = warp_wait(&sh.q_full, qp, &sh.abort, wl);
        if (!ok) break;
        qp ^= 1;
        const int nt = s.t1 - s.t0;
        if (s.x.nv <= 128 * tile) {   // no vector of this tile's
            for (int i = 0; i < 2 * nt && item(); ++i) {
                if (e) mbar_arrive(&sh.empty[get.slot]);
                if (e && i == 2 * nt - 1) mbar_arrive(&sh.q_free);
                get.next(z.nslot);
            }
            continue;
        }
        scores();
        for (int j = 0; ok && j < nt; ++j) {
            if (j == nt - 1) commit(&sh.q_free);   // the last scores are issued
            if (j == 0) ok = warp_wait(&sh.o_free[tile], (nseg & 1) ^ 1, &sh.abort, wl);
            // the later half of the keys first, as the softmax forms it
            ok = ok && warp_wait(&sh.p_full[2 * tile + 1], n & 1, &sh.abort, wl);
            if (!ok || !item()) break;
            const uint64_t vd = dv + (uint64_t)(get.slot * (SLOT / 16));
            run_ts<1, 8>(e, out, sc + 64, vd + 512, id_o, j > 0);
            commit(&sh.pv_half[tile]);
            ok = warp_wait(&sh.p_full[2 * tile], n & 1, &sh.abort, wl);
            if (!ok) break;
            tc_after();
            run_ts<1, 8>(e, out, sc, vd, id_o, 1);
            commit(&sh.pv_done[tile]);
            commit(&sh.empty[get.slot]);
            get.next(z.nslot);
            ++n;
            if (j + 1 < nt) scores();
        }
        ++nseg;
    }
    if (e) {
        mma_commit(&sh.fin);   // tracks every MMA issued, also after an abort
        mbar_drain(&sh.fin, 0);
    }
    __syncwarp();
}

template <typename T, typename C>
__device__ __forceinline__ void issuer(const PgArgs &a, Shared &sh, const Shape &z, uint32_t q0, uint32_t ring0, uint32_t tmem,
                                       const PgTable &tab, int units, PgShare share) {
    using M = typename Types<T, C>::M;
    constexpr int TERMS = Types<T, C>::TERMS;
    using Col = Cols<TERMS>;
    const bool e = elect_one();
    const uint64_t dq = desc_sw128(q0), dk = desc_sw128(ring0), dv = desc_sw128_mn(ring0, z.v_keys * 128);
    const uint32_t id_s = idesc<M>(128, KT, 0), id_o = idesc<M>(128, z.nv, 1);
    const long long wl = a.wait_cycles;
    bool ok = true;
    Ring get = {0, 0};
    uint32_t qp = 0;                 // phase of q_full
    uint32_t npv = 0, nseg = 0;      // P V issued, segments
    uint32_t nsc = 0;                // scores issued
    PgSegment s;
    auto commit = [&](uint64_t *bar) {
        if (e) mma_commit(bar);
    };
    auto filled = [&](const Ring &r) -> bool {
        ok = ok && warp_wait(&sh.full[r.slot], r.phase, &sh.abort, wl);
        return ok;
    };
    // scores from the key items at `r` on, released once used
    auto scores = [&](int buf, Ring r) {
        const uint32_t col = tmem + Col::score(buf);
        if constexpr (TERMS == 1) {
            for (int i = 0; i < z.k_items; ++i) {
                if (!filled(r)) return;
                tc_after();
                const uint64_t kd = dk + (uint64_t)(r.slot * (SLOT / 16)), qd = dq + (uint64_t)(2 * i * 1024);
                run_ss(e, col, qd, kd, id_s, min(8, z.ksteps - 8 * i), i > 0);
                commit(&sh.empty[r.slot]);
                r.next(z.nslot);
            }
        } else {
            // lower terms first: an accumulation rounds at the size of the sum so far
            Ring q = r;
            for (int i = 0; i < z.k_items; ++i, q.next(z.nslot))
                if (!filled(q)) return;
            tc_after();
            for (int m = TERMS - 1; m >= 0; --m) {
                q = r;
                for (int i = 0; i < z.k_items; ++i, q.next(z.nslot)) {
                    const uint64_t kd = dk + (uint64_t)(q.slot * (SLOT / 16));
                    const uint64_t qd = dq + (uint64_t)((m * z.nqc + 2 * i) * 1024);
                    run_ss(e, col, qd, kd, id_s, min(8, z.ksteps - 8 * i), m < TERMS - 1 || i > 0);
                }
            }
            q = r;
            for (int i = 0; i < z.k_items; ++i, q.next(z.nslot)) commit(&sh.empty[q.slot]);
        }
        commit(&sh.s_full[buf]);
    };
    // P V from the value items at `r` on
    auto values = [&](int buf, Ring r, bool acc) {
        const uint32_t out = tmem + Col::out(0), p = tmem + Col::score(buf);
        if constexpr (TERMS == 3) {   // one item; a sum of its own
            if (!filled(r)) return;
            tc_after();
            const uint64_t vd = dv + (uint64_t)(r.slot * (SLOT / 16));
            // lower terms first
            for (int h = 0; h < 2; ++h) run_ts<1, 8>(e, out, p + Col::p(4 * h, 2), vd + 512 * h, id_o, h > 0);
            for (int m = 1; m >= 0; --m)
                for (int h = 0; h < 2; ++h) run_ts<1, 24>(e, out, p + Col::p(4 * h, m), vd + 512 * h, id_o, 1);
            commit(&sh.empty[r.slot]);
        } else {
            for (int i = 0; i < z.v_items; ++i) {
                if (!filled(r)) return;
                tc_after();
                const uint64_t vd = dv + (uint64_t)(r.slot * (SLOT / 16));
                run_ts<TERMS, TERMS == 1 ? 8 : 24>(e, out, p + 64 * i, vd, id_o, acc || i > 0);
                if (z.v_items == 1) run_ts<TERMS, TERMS == 1 ? 8 : 24>(e, out, p + 64, vd + 512, id_o, 1);
                commit(&sh.empty[r.slot]);
                r.next(z.nslot);
            }
        }
        commit(&sh.pv_done[0]);
    };
    auto advance = [&](int n) {
        for (int i = 0; i < n; ++i) get.next(z.nslot);
    };
    while (ok && pg_next<Plan<1>>(a, tab, units, share, s)) {
        ok = warp_wait(&sh.q_full, qp, &sh.abort, wl);
        if (!ok) break;
        qp ^= 1;
        tc_after();
        const int nt = s.t1 - s.t0;
        scores(nsc & 1, get);
        ++nsc;
        advance(z.k_items);
        for (int j = 0; ok && j < nt; ++j) {
            if (j + 1 < nt) {
                scores(nsc & 1, get);
                if (!ok) break;
                ++nsc;
                advance(z.k_items);
            }
            if (j == nt - 1) commit(&sh.q_free);
            ok = warp_wait(&sh.p_full[npv & 1], (npv >> 1) & 1, &sh.abort, wl);
            // outputs given back: of the segment before, or (sums in registers) of the tile before
            if (ok && (TERMS == 3 || j == 0)) ok = warp_wait(&sh.o_free[0], ((TERMS == 3 ? npv : nseg) & 1) ^ 1, &sh.abort, wl);
            if (!ok) break;
            tc_after();
            values(npv & 1, get, j > 0);
            ++npv;
            advance(z.v_items);
        }
        ++nseg;
    }
    if (e) {
        mma_commit(&sh.fin);   // tracks every MMA issued, also after an abort
        mbar_drain(&sh.fin, 0);
    }
    __syncwarp();
}

// ---------------------------------------------------------------- softmax

// 8 floats to 8 values of T
__device__ __forceinline__ void st8(float *p, const float *x) {
    o1_st4(p, make_float4(x[0], x[1], x[2], x[3]));
    o1_st4(p + 4, make_float4(x[4], x[5], x[6], x[7]));
}
template <typename T>
__device__ __forceinline__ void st8(T *p, const float *x) {
    *(uint4 *)p = make_uint4(pack_m(p, x[0], x[1]), pack_m(p, x[2], x[3]), pack_m(p, x[4], x[5]), pack_m(p, x[6], x[7]));
}

// 32 bytes: 8 floats, or 16 values of T
__device__ __forceinline__ void st32_words(void *p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
__device__ __forceinline__ void st32(float *p, const float *x) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(x[i]);
    st32_words(p, w);
}
template <typename T>
__device__ __forceinline__ void st32(T *p, const float *x) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack_m(p, x[2 * i], x[2 * i + 1]);
    st32_words(p, w);
}

// ones from bit b on, of any b
__device__ __forceinline__ uint32_t ones_from(int b) { return b <= 0 ? ~0u : b > 31 ? 0u : ~0u << b; }

template <typename T, typename C, int QT>
__device__ __forceinline__ void softmax(const PgArgs &a, Shared &sh, const Shape &z, uint32_t tmem, const PgTable &tab, int units,
                                        PgShare share, int vecs) {
    using M = typename Types<T, C>::M;
    constexpr int TERMS = Types<T, C>::TERMS;
    constexpr bool REG = TERMS == 3;   // sums in registers
    constexpr PgReference REF(std::is_same<M, __half>::value);
    using Col = Cols<TERMS>;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = warp >> 2, row = tid & 127;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const float sc2 = a.scale * 1.4426950408889634f;   // scores in log2 units; scale > 0
    const long long wl = a.wait_cycles;
    if (tid == 0) {
        PgHead *head = &pg_parts(a.part, BLOCKS, vecs).head[blockIdx.x];
        head->last = -1;
        PgShare first = share;
        PgSegment f;
        if (pg_next<Plan<QT>>(a, tab, units, first, f)) pg_head<Plan<QT>>(head, share, f);
    }
    __syncwarp();
    bool ok = true;
    uint32_t n = 0, turns = 0;   // tiles so far, of this warpgroup's query tile, and in turn with the other's
    PgSegment s;
    while (pg_next<Plan<QT>>(a, tab, units, share, s)) {
        const int tile = QT == 2 ? wg : 0, v0 = 128 * tile;
        if (QT == 2 && s.x.nv <= v0) continue;
        const int pos = s.x.pos(a, min(v0 + row, s.x.nv - 1)), low = a.window ? pos - a.window + 1 : 0;
        // positions that every row of the tile attends
        const int plain_hi = s.x.pos(a, v0), last = s.x.pos(a, min(v0 + 127, s.x.nv - 1));
        const int plain_lo = a.window ? last - a.window + 1 : 0;
        const bool paired = s.x.nv > 128;   // both query tiles have vectors
        const bool idle = v0 + 32 * (warp & 3) >= s.x.nv;   // no row of this warp's
        float m = -INFINITY, l = 0.f;
        float o[REG ? 64 : 1];
        if (REG) {
#pragma unroll
            for (int i = 0; i < (REG ? 64 : 1); ++i) o[i] = 0.f;
        }
        // which runs of 16 positions have a page: four tiles a look, a lane a run
        auto look = [&](int j) {
            const int p = (s.x.lo / KT + j) * KT + 16 * lane;
            return j + (lane >> 3) >= s.t1 || p > s.x.hi || p + 15 < s.x.lo || pg_page(a, s.x.slot, p) >= 0;
        };
        bool next_runs = look(s.t0);
        uint32_t runs = 0;
        // P V of the tile before (number t), added to this warpgroup's columns
        auto add_values = [&](uint32_t t) {
            ok = ok && warp_wait(&sh.pv_done[0], t & 1, &sh.abort, wl);
            if (!ok) return;
            tc_after();
#pragma unroll
            for (int c = 0; c < 64; c += 32) {
                uint32_t r[32];
                TMEM_LD32(lanes + Col::out(0) + 64 * wg + c, r);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[REG ? c + i : 0] += __uint_as_float(r[i]);
            }
            tc_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.o_free[0]);
        };
        // (QT = 1: a warp whose wait ran out goes on to the next decision)
        for (int j = s.t0; j < s.t1 && (ok || (QT == 1 && j > s.t0)); ++j, ++n) {
            if (((j - s.t0) & 3) == 0) {
                runs = __ballot_sync(0xffffffffu, next_runs);
                next_runs = look(j + 4);
            }
            const uint32_t there = runs & 0xffu;
            runs >>= 8;
            const int x0 = (s.x.lo / KT + j) * KT, buf = QT == 2 ? tile : n & 1;
            const bool plain = x0 >= plain_lo && x0 + KT - 1 <= plain_hi && there == 0xffu;
            ok = ok && warp_wait(&sh.s_full[buf], QT == 2 ? n & 1 : (n >> 1) & 1, &sh.abort, wl);
            if (QT == 2 && !ok) break;
            tc_after();
            const uint32_t scol = lanes + Col::score(buf);
            if (QT == 2 && paired) {   // after the other tile's warp: one forms weights while the other's MMAs run
                ok = warp_wait(&sh.turn[wg][warp & 3], (turns & 1) ^ (wg == 0), &sh.abort, wl);
                if (!ok) break;
                ++turns;
            }
            bool added = !REG || j == s.t0;   // the tile before's values
            // 64 keys at a time (QT = 2: the later ones first; QT = 1: this
            // warpgroup's half), each a step of the running softmax. Weights are
            // taken from the reference as it stands, which the maximum, formed
            // beside them, only rarely passes by 2^8: then the reference moves and
            // they are formed again.
#pragma unroll 1
            for (int i = 0; i < QT; ++i) {
                const int h = QT == 2 ? 1 - i : wg;
                // (several terms: 32 keys at a time, for their maximum and again
                // for their weights)
                constexpr int NR = TERMS == 1 ? 64 : 32;
                uint32_t r[NR], w[TERMS == 1 ? 32 : 1];
                float sum = 0.f, early = -INFINITY;
                auto load = [&](int k0) {   // raw scores, those not attended -inf
#pragma unroll
                    for (int c = 0; c < NR; c += 32) TMEM_LD32(scol + 64 * h + k0 + c, (&r[c]));
                    tmem_ld_wait();
                    if (!plain) {
                        const int b0 = low - x0 - 64 * h - k0, b1 = pos - x0 - 64 * h - k0;
                        const uint32_t on = there >> (4 * h + k0 / 16);
#pragma unroll
                        for (int q = 0; q < NR; q += 32) {
                            const uint32_t at = (on >> (q / 16) & 1) * 0xffffu | (on >> (q / 16 + 1) & 1) * 0xffff0000u;
                            const uint32_t bits = at & ones_from(b0 - q) & ~ones_from(b1 - q + 1);
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!(bits >> c & 1)) r[q + c] = 0xff800000u;
                        }
                    }
                };
                if (ok && !idle) {
                    if constexpr (TERMS > 1) {
                        load(32);
#pragma unroll
                        for (int c = 0; c < NR; c += 2) early = max3(early, r[c], r[c + 1]);
                    }
                    load(0);
                }
#pragma unroll 1
                while (true) {
                    float top = -INFINITY;
                    const float ref = m > -INFINITY ? m : 0.f;
                    const F2 f2s = f2(sc2, sc2), f2r = f2(-ref, -ref);
                    if (ok && !idle) {
                        float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                        F2 part[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
                        for (int c = 0; c < NR / 2; ++c) {
                            t[c & 3] = max3(t[c & 3], r[2 * c], r[2 * c + 1]);
                            if constexpr (TERMS == 1) {
                                float x, y;
                                f2_get(f2_fma(f2(__uint_as_float(r[2 * c]), __uint_as_float(r[2 * c + 1])), f2s, f2r), x, y);
                                x = ex2(x);
                                y = ex2(y);
                                part[c & 1] = f2_add(part[c & 1], f2(x, y));
                                w[c] = pack_m((const M *)nullptr, x, y);
                            }
                        }
                        top = fmaxf(fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])), early) * sc2;
                        if constexpr (TERMS == 1) {
                            float a0, a1;
                            f2_get(f2_add(part[0], part[1]), a0, a1);
                            sum = a0 + a1;
                        }
                    }
                    // QT = 1: the two halves of a row decide together, also to give
                    // up (a barrier that one of them left would never be met)
                    bool move = top > m + REF.above;
                    if (QT == 2) move = __any_sync(0xffffffffu, move);
                    else move = sm_or(move || !ok);
                    if (!move) break;
                    if (QT == 1) {
                        sh.half[wg][row] = top;
                        ok = !sm_or(!ok);
                        if (!ok) break;
                        top = fmaxf(top, sh.half[wg ^ 1][row]);
                    }
                    const float mn = fmaxf(m, top - REF.below), f = m > -INFINITY ? ex2(m - mn) : 0.f;
                    m = mn;
                    l *= f;
                    if (REG) {
                        if (!added) add_values(n - 1);
                        added = true;
#pragma unroll
                        for (int c = 0; c < (REG ? 64 : 1); ++c) o[c] *= f;
                    } else if (j > s.t0 || i > 0) {
                        // all P V so far, of the tile before or of this one's first half
                        if (QT == 2 && i > 0) ok = warp_wait(&sh.pv_half[tile], n & 1, &sh.abort, wl);
                        else ok = warp_wait(&sh.pv_done[tile], (n - 1) & 1, &sh.abort, wl);
                        if (QT == 1) ok = !sm_or(!ok);
                        if (!ok) break;
                        tc_after();
                        // this warpgroup's columns: all of its tile's (QT = 2), or every other 32
#pragma unroll 1
                        for (int c = QT == 2 ? 0 : 32 * wg; c < z.nv; c += QT == 2 ? 32 : 64) {
                            uint32_t y[32];
                            TMEM_LD32(lanes + Col::out(tile) + c, y);
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 32; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * f);
                            TMEM_ST32(lanes + Col::out(tile) + c, y);
                        }
                    }
                    if (QT == 1) sm_sync();   // the maxima are read before they are written again
                }
                if (!ok) break;
                if (QT == 2 && paired && i == 0 && lane == 0) mbar_arrive(&sh.turn[wg ^ 1][warp & 3]);
                // P over the scores it comes from
                if (!idle) {
                    __syncwarp();   // the warp is together for the stores
                    if constexpr (TERMS == 1) {
                        l += sum;
                        TMEM_ST32(scol + 64 * h, w);
                    } else {
                        const float ref = m > -INFINITY ? m : 0.f;
#pragma unroll 1
                        for (int k0 = 0; k0 < 64; k0 += 32) {
                            if (k0) load(k0);
                            uint32_t w0[16], w1[16], w2[16];
#pragma unroll
                            for (int c = 0; c < 16; ++c) {
                                float x = ex2(fmaf(__uint_as_float(r[2 * c]), sc2, -ref));
                                float y = ex2(fmaf(__uint_as_float(r[2 * c + 1]), sc2, -ref));
                                l += x + y;
                                w0[c] = take_m<M>(x, y);
                                w1[c] = take_m<M>(x, y);
                                if constexpr (TERMS > 2) w2[c] = pack_m((const M *)nullptr, x, y);
                            }
                            __syncwarp();
                            TMEM_ST16(scol + 64 * h + k0, w0);
                            TMEM_ST16(scol + 64 * h + k0 + 16, w1);
                            if constexpr (TERMS > 2) TMEM_ST16(scol + 128 + 32 * h + k0 / 2, w2);
                        }
                    }
                }
                tmem_st_wait();
                tc_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_full[QT == 2 ? 2 * tile + h : buf]);
            }
            if (ok && !added) add_values(n - 1);
            if (QT == 2 && !ok) break;
        }
        // ---- the segment's end: its rows, or their partial results
        if (REG) {
            add_values(n - 1);
        } else {
            // a parity tells two phases apart: with scores a tile ahead (QT = 1) the
            // last scores do not say that the P V before the last is done
            if (QT == 1 && s.t1 - s.t0 > 1) ok = ok && warp_wait(&sh.pv_done[0], n & 1, &sh.abort, wl);
            ok = ok && warp_wait(&sh.pv_done[QT == 2 ? tile : 0], (n - 1) & 1, &sh.abort, wl);
            tc_after();
        }
        if (QT == 1) {
            sh.half[wg][row] = l;
            ok = !sm_or(!ok);   // both halves write, or none
            l += sh.half[wg ^ 1][row];
            sm_sync();
        }
        // the unit again, not held in registers meanwhile
        int u = s.u;
        asm volatile("" : "+r"(u));
        const PgUnit x = pg_unit<Plan<QT>::V>(a, tab, u);
        const PgParts parts = pg_parts(a.part, BLOCKS, vecs);
        const int v = v0 + row;
        const bool whole = s.whole(), in = v < x.nv;
        const float f = !ok ? NAN : !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
        const size_t ps = s.part();
        const bool wide = ((uintptr_t)a.out | a.os * sizeof(T) | a.dv * sizeof(T)) % 32 == 0;
        T *out = (T *)a.out + (in ? pg_vec_at(a, x.row0, x.vec0 + v, s.g, a.os, a.dv) : 0);
        if (in && !whole && (QT == 2 || wg == 0)) *(float2 *)(parts.stat + (ps * vecs + v) * 2) = ok ? make_float2(m, l) : make_float2(0.f, NAN);
        auto write = [&](int c, float *y) {   // 32 columns
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = ok ? y[i] * f : NAN;
            if (!in) return;
            if (!whole) {
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    if (c + i < a.dv) *pg_val(parts, ps, vecs, a.dv, v, c + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
                return;
            }
            // 32 bytes a store where the rows allow it: a lane writes a row of
            // its own, so that a store costs a line a lane whatever its width
            constexpr int W = 32 / sizeof(T);
            if (wide && c + 32 <= a.dv) {
#pragma unroll
                for (int i = 0; i < 32; i += W) st32(out + c + i, y + i);
            } else {
#pragma unroll
                for (int i = 0; i < 32; i += 8)
                    if (c + i < a.dv) st8(out + c + i, y + i);
            }
        };
        if constexpr (REG) {
            write(64 * wg, o);
            write(64 * wg + 32, o + 32);
        } else {
#pragma unroll 1
            for (int c = QT == 2 ? 0 : 32 * wg; c < a.dv; c += QT == 2 ? 32 : 64) {
                uint32_t y[32];
                float w[32];
                TMEM_LD32(lanes + Col::out(tile) + c, y);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) w[i] = __uint_as_float(y[i]);
                write(c, w);
                __syncwarp();
            }
            tc_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.o_free[QT == 2 ? tile : 0]);
        }
        __syncwarp();
    }
    if (!ok) tmem_st_wait();   // stores issued before a wait ran out are over before the TMEM is given back
}

template <typename T, typename C, int QT>
__global__ __launch_bounds__(THREADS, 1) void k_pg_tc(PgArgs a, const __grid_constant__ PgTable tab,
                                                      const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                                                      const __grid_constant__ CUtensorMap mv, int qrows, int units, int vecs) {
    constexpr int TERMS = Types<T, C>::TERMS;
    extern __shared__ unsigned char smraw[];
    __shared__ Shared sh;
    const Shape z = shape_of<QT, TERMS, sizeof(C) == 1>(a.d, a.dv);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t q0 = (su32(smraw) + 1023) & ~1023u, ring0 = q0 + z.raw + (sizeof(C) == 1 ? RAW_BYTES : 0);
    if (tid == 0) {
        for (int i = 0; i < MAX_SLOTS; ++i) {
            mbar_init(&sh.full[i], sizeof(C) == 1 ? PR_WARPS : 1);
            mbar_init(&sh.empty[i], QT);   // QT issuers
        }
        mbar_init(&sh.q_full, sizeof(C) == 1 && !qrows ? PR_WARPS : 1);
        for (int i = 0; i < 2; ++i) mbar_init(&sh.raw_full[i], 1), mbar_init(&sh.raw_empty[i], PR_WARPS);
        mbar_init(&sh.q_free, QT);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i], QT == 2 ? SM_WARPS / 2 : SM_WARPS);
            mbar_init(&sh.p_full[2 + i], SM_WARPS / 2);
            mbar_init(&sh.pv_done[i], 1);
            mbar_init(&sh.pv_half[i], 1);
            mbar_init(&sh.o_free[i], QT == 2 ? SM_WARPS / 2 : SM_WARPS);
        }
        mbar_init(&sh.fin, QT);
        for (int i = 0; i < 8; ++i) mbar_init(&sh.turn[i >> 2][i & 3], 1);
        for (int i = 0; i < MAX_SLOTS; ++i) sh.sent[i] = 0;
        sh.sent_q = sh.sent_raw[0] = sh.sent_raw[1] = 0;
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    if (warp == SM_WARPS + PR_WARPS) tmem_alloc512(&sh.tslot);
    tc_before();
    const PgShare share = pg_share<Plan<QT>, THREADS>(a, tab, units, sh.share);
    __syncthreads();
    tc_after();
    const uint32_t tmem = sh.tslot;
    using R = Regs;
    if (warp < SM_WARPS) {
        regs_more<R::SOFTMAX>();
        softmax<T, C, QT>(a, sh, z, tmem, tab, units, share, vecs);
    } else {
        const int w = warp - SM_WARPS;   // the producers', then the issuers'
        Producer<T, C, QT> p = {a, sh, z, q0, ring0, lane, 4 * w + (lane >> 3), lane & 7, qrows ? &mq : nullptr, &mk, &mv, qrows,
                                w, {0, 0}, true, true, 0, 1, q0 + z.raw};
        if (w < PR_WARPS) {
            regs_less<R::PRODUCER>();
            p.run(tab, units, share);
        } else {
            regs_less<R::ISSUER>();
            const int i = w - PR_WARPS;
            if (i < QT) {
                if constexpr (QT == 2) issuer_of<T, C>(i, a, sh, z, q0, ring0, tmem, tab, units, share);
                else issuer<T, C>(a, sh, z, q0, ring0, tmem, tab, units, share);
            } else if (sizeof(C) == 1 && i == 2) {
                p.load_codes(tab, units, share);
            }
        }
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (warp == SM_WARPS + PR_WARPS) tmem_free512(tmem);
    // Where no wait ran out, the issuers met all that was sent. Where one did, what
    // TMA still writes lands before the block ends, whichever role's wait it was:
    // the senders' own may all have been met.
    if (tid == 0 && sh.abort) {
        for (int i = 0; i < MAX_SLOTS; ++i) drain(&sh.full[i], sh.sent[i]);
        drain(&sh.q_full, sh.sent_q);
        for (int i = 0; i < 2; ++i) drain(&sh.raw_full[i], sh.sent_raw[i]);
        atomicOr(&pg_device_flags, (uint32_t)O1_FLAG_WAIT_EXPIRED);
    }
}

template <typename M>
bool encode(CUtensorMap *m, int rank, const void *base, const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box) {
    const auto enc = tensor_map_encoder();
    const cuuint32_t es[3] = {1, 1, 1};
    return enc && enc(m, std::is_same<M, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
                      (void *)base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// A pool as rows of `width` values, in boxes of 64 columns and `box` rows of a page.
template <typename M>
bool pool_map(CUtensorMap *m, const void *base, int width, uint64_t rows, uint32_t box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)width * 2};
    const cuuint32_t box[2] = {64, box_rows};
    return encode<M>(m, 2, base, dims, strides, box);
}

template <typename T, typename C, int QT>
cudaError_t launch_q(const PgArgs &a, int dtype, const PgTable &tab, int64_t vectors, cudaStream_t st) {
    static unsigned long long done = 0;
    unsigned long long bit = 0;
    auto *k = k_pg_tc<T, C, QT>;
    if (o1_attrs_needed(&done, &bit)) {
        cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM);
        if (e != cudaSuccess) return e;
        // a trade of more registers than the block starts with would wait for ever
        cudaFuncAttributes at;
        if ((e = cudaFuncGetAttributes(&at, k)) != cudaSuccess) return e;
        if (at.numRegs != REGS) return cudaErrorInvalidConfiguration;
        o1_attrs_done(&done, bit);
    }
    constexpr int V = Plan<QT>::V;
    const int vecs = (int)(vectors < V ? vectors : V);
    CUtensorMap mq = {}, mk = {}, mv = {};
    int qrows = 0;
    if constexpr (sizeof(C) == 2) {
        const uint64_t rows = ((uint64_t)a.n_pages * a.G) << a.lpage;
        const uint32_t page = 1u << a.lpage, most = a.dv > 128 ? 64 : 128;
        if (!pool_map<C>(&mk, a.k, a.d, rows, page < 128 ? page : 128) || !pool_map<C>(&mv, a.v, a.dv, rows, page < most ? page : most))
            return cudaErrorInvalidValue;
    }
    if constexpr (sizeof(T) == 2 && Types<T, C>::TERMS == 1)
        if (128 % a.hpg == 0) {
            qrows = 128 / a.hpg;
            const cuuint64_t dims[3] = {(cuuint64_t)a.d, (cuuint64_t)a.G * a.hpg, (cuuint64_t)vectors / a.hpg};
            const cuuint64_t strides[2] = {(cuuint64_t)a.d * 2, (cuuint64_t)a.qs * 2};
            const cuuint32_t box[3] = {64, (cuuint32_t)a.hpg, (cuuint32_t)qrows};
            if (!encode<T>(&mq, 3, a.q, dims, strides, box)) return cudaErrorInvalidValue;
        }
    k<<<BLOCKS, THREADS, SMEM, st>>>(a, tab, mq, mk, mv, qrows, tab.total, vecs);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? pg_launch_join(a, dtype, BLOCKS, BLOCKS, vecs, vecs, st) : e;
}
// Two query tiles a block where both fit beside a ring of five slots: one term
// and rows of up to 128 values.
template <typename T, typename C>
cudaError_t launch_t(const PgArgs &a, int dtype, const PgTable &tab, int64_t vectors, cudaStream_t st) {
    if constexpr (Types<T, C>::TERMS == 1)
        if (a.d <= 128 && a.dv <= 128) return launch_q<T, C, 2>(a, dtype, tab, vectors, st);
    return launch_q<T, C, 1>(a, dtype, tab, vectors, st);
}

}  // namespace

int pg_tc_vectors(const o1_pg_geom &g) {
    const bool wide = g.d > 128 || g.dv > 128;
    if (g.dtype == O1_F32) return wide ? 0 : 128;   // three terms of Q, and P's third
    if (g.dtype == O1_F16 && g.cache_dtype == O1_E4M3) return 128;
    return wide ? 128 : 256;
}

size_t pg_tc_scratch(const o1_pg_geom &g, int64_t vectors) {
    const int v = pg_tc_vectors(g);
    return v ? pg_parts_bytes(BLOCKS, (int)(vectors < v ? vectors : v), g.dv) : 0;
}

cudaError_t pg_launch_tc(const PgArgs &a, const o1_pg_geom &g, const PgTable &tab, int64_t vectors, cudaStream_t st) {
    if (g.dtype == O1_F32)
        return g.cache_dtype == O1_E4M3 ? launch_t<float, uint8_t>(a, g.dtype, tab, vectors, st)
                                        : launch_t<float, __nv_bfloat16>(a, g.dtype, tab, vectors, st);
    if (g.dtype == O1_BF16)
        return g.cache_dtype == O1_E4M3 ? launch_t<__nv_bfloat16, uint8_t>(a, g.dtype, tab, vectors, st)
                                        : launch_t<__nv_bfloat16, __nv_bfloat16>(a, g.dtype, tab, vectors, st);
    return g.cache_dtype == O1_E4M3 ? launch_t<__half, uint8_t>(a, g.dtype, tab, vectors, st)
                                    : launch_t<__half, __half>(a, g.dtype, tab, vectors, st);
}

// As lin_flags: reset only where it was read as raised.
int pg_flags(uint32_t *flags, int clear, cudaStream_t st) {
    if (cudaMemcpyFromSymbolAsync(flags, pg_device_flags, sizeof(uint32_t), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return O1_ERR_CUDA;
    if (!clear || !*flags) return O1_OK;
    static const uint32_t zero = 0;
    if (cudaMemcpyToSymbolAsync(pg_device_flags, &zero, sizeof(uint32_t), 0, cudaMemcpyHostToDevice, st) != cudaSuccess)
        return O1_ERR_CUDA;
    return cudaStreamSynchronize(st) == cudaSuccess ? O1_OK : O1_ERR_CUDA;
}
