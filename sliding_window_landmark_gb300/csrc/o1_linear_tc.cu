// Linear attention with a decay per head over prompts, on the tensor cores.
//
// The recurrence S = l S + k v^T, o = q S over the n rows of a segment (128 or
// 256) with entering state S_in (l = e^{log_decay}):
//   o_i   = l^{i+1} q_i S_in + sum_{j <= i} l^{i-j} (q_i . k_j) v_j
//   S_out = l^n S_in + dS,   dS = sum_j (l^{n-1-j} k_j) v_j^T
// so that only the segments' states are sequential:
//   k_lin_split  fp16 and fp32 rows: q, k, v as bf16 terms, once
//   k_lin_inc    dS of every (segment, head): one product of depth n
//   k_lin_scan   per state element, over the segments of a sequence: dS is
//                replaced by the state entering the segment (as bf16 terms),
//                and the last state goes to its slot
//   k_lin_out    every (128-row tile, head)'s outputs: q S_in, scores against
//                the segment's tiles so far, weighted and masked into P, P V
// No step carries a weight above 1 (every power of l has an exponent >= 0), so
// nothing overflows whatever the decay.
//
// Precision. The MMAs take bf16 operands with fp32 accumulation. An fp32
// value is split into three bf16 terms (each the bf16 of what the earlier ones
// leave, the subtractions exact; what is left is below 2^-24 of it), an fp16
// value into two (exactly), a bf16 value is one; of a product's term pairs
// those down to 2^-16 (two terms) or 2^-24 (three) are taken. bf16 terms have
// fp32's exponent range, so no scaling is needed. States are fp32 sums: the
// weighted keys l^{n-1-j} k_j are always three terms. The entering state and P
// only reach the outputs: two terms where those are 16-bit, three for fp32.
// An accumulation rounds at the size of the sum so far, so smaller products
// come first, or have accumulators of their own: summed as they come, 600 fp32
// rows were 1.5e-6 off in the 2-norm instead of 2.4e-7 (plain fp32: 3e-7).
//
// Layout. All panels are rows of 64-column blocks of bf16, 128-byte swizzled,
// and serve as K-major or MN-major operands as they lie: keys are K-major
// for the scores and (weighted) MN-major for dS, values and S_in are MN-major.
// Both kernels of MMAs are persistent and split by warp: TMA (or, for weighted
// keys, staging warps), an MMA issuer, P warps, and warps that store.
//
// Bound, measured at 32768 bf16 rows of 8 heads of 256 (341 us, 4 passes; a
// pass's kernels alone, under the profiler, take 45, 29 and 14 us, 351 in all:
// in the call a kernel's set-up runs under the one before): the outputs by the
// L2-to-shared-memory ingest, 46 bytes a clock and SM at best, 31 on average;
// the increments by the keys' weighting and splitting beside MMAs that read 96
// of the 128 bytes a clock shared memory gives; the scan by its bytes, 9 TB/s
// in the L2. fp32 (4096 rows: 128 us) reads three terms: its 128 x 128 MMAs
// alone take the whole shared-memory bandwidth.
#include <math.h>

#include "o1_linear.cuh"
#include "o1_tc.cuh"

static __device__ uint32_t lin_device_flags;

namespace {

constexpr int TN = 128;   // columns of a tile of dv (and of d, for dS)
constexpr int KV = 64;    // rows or columns of a staged panel's short side
constexpr int PROD_WARPS = 16, PROD = 32 * PROD_WARPS;
constexpr int LIST = 64;  // units of a CTA, decoded once at its start

// bf16 terms of the inputs (q, k, v) and of what is formed on the way (the
// entering state, P).
template <typename T>
struct Terms {
    static constexpr int in = 1;    // bf16 terms of q, k, v
    static constexpr int mid = 2;   // of the entering state and P
};
template <>
struct Terms<__half> {
    static constexpr int in = 2, mid = 2;
};
template <>
struct Terms<float> {
    static constexpr int in = 3, mid = 3;
};
__host__ __device__ constexpr int max_sum(int a, int b) { return a > b ? a - 1 : b - 1; }
__host__ __device__ inline int ceil16(int x) { return (x + 15) & ~15; }

// ---------------------------------------------------------------- staging

// 8 consecutive values of T as loaded: one 16-byte word, two for fp32.
template <typename T>
constexpr int WORDS = sizeof(T) == 4 ? 2 : 1;

__device__ __forceinline__ void words_floats(const uint4 *r, float (&x)[8], const float *) {
    const uint32_t u[8] = {r[0].x, r[0].y, r[0].z, r[0].w, r[1].x, r[1].y, r[1].z, r[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(u[i]);
}
__device__ __forceinline__ void words_floats(const uint4 *r, float (&x)[8], const __nv_bfloat16 *) {
    const uint32_t u[4] = {r[0].x, r[0].y, r[0].z, r[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void words_floats(const uint4 *r, float (&x)[8], const __half *) {
    const uint32_t u[4] = {r[0].x, r[0].y, r[0].z, r[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*(const __half2 *)&u[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// x[2i], x[2i + 1] as bf16 pairs (the lower index in the low half), x left
// with what the rounding dropped (exact)
__device__ __forceinline__ uint32_t take_pair(float &x0, float &x1) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
    const uint32_t w = *(const uint32_t *)&h;
    x0 -= __uint_as_float(w << 16);
    x1 -= __uint_as_float(w & 0xffff0000u);
    return w;
}
// x[8] as NT bf16 terms, term t's 16 bytes at dst + t * panel
template <int NT>
__device__ __forceinline__ void store_terms(unsigned char *dst, uint32_t panel, float (&x)[8]) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = take_pair(x[2 * i], x[2 * i + 1]);
        *(uint4 *)(dst + t * panel) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// A panel of bf16 in shared memory: `rows` rows in blocks of 64 columns
// (rows * 128 bytes each), 128-byte swizzled. Byte offset of the 8-column
// group cg of row r:
__device__ __forceinline__ uint32_t panel_off(int rows, int r, int cg) {
    return (uint32_t)((cg >> 3) * rows * 128 + r * 128 + (((cg & 7) ^ (r & 7)) << 4));
}

// What a producer stages into a slot of the ring: a panel of ROWS x COLS
// values of a row tensor (rows past nr and columns past width read as zero),
// as NT bf16 terms. Thread pt takes one 8-column group of every STEP-th row, so
// that its addresses on both sides are one base and constant steps: producers
// are few warps a scheduler, and every dependent instruction shows.
template <typename T, int ROWS, int COLS>
struct Panel {
    static constexpr int GPR = COLS / 8, STEP = PROD / GPR, IT = ROWS / STEP, W = WORDS<T>;
    static_assert(ROWS % STEP == 0 && STEP % 8 == 0, "rows a thread");
    static __device__ __forceinline__ uint32_t row(uint32_t pt) { return pt / GPR; }
    static __device__ __forceinline__ uint32_t off(uint32_t pt) { return panel_off(ROWS, pt / GPR, pt % GPR); }
    static __device__ __forceinline__ void load(uint4 *raw, const T *src, size_t stride, int nr, int width, uint32_t pt) {
        const uint32_t r = pt / GPR, cg = pt % GPR;
        const char *p = (const char *)(src + (size_t)r * stride + 8 * cg);
        const size_t step = STEP * stride * sizeof(T);
        nr = 8 * (int)cg < width ? nr - (int)r : 0;   // of this thread's rows
#pragma unroll
        for (int i = 0; i < IT; ++i, p += step)
#pragma unroll
            for (int j = 0; j < W; ++j) raw[i * W + j] = STEP * i < nr ? ((const uint4 *)p)[j] : make_uint4(0, 0, 0, 0);
    }
    // NT terms of w[i] * x, w the weights of this thread's rows; dst: the panel + off(pt)
    template <int NT>
    static __device__ __forceinline__ void split(const uint4 *raw, unsigned char *dst, const float (&w)[IT]) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            float x[8];
            words_floats(raw + i * W, x, (const T *)nullptr);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= w[i];
            store_terms<NT>(dst + i * STEP * 128, ROWS * COLS * 2, x);
        }
    }
};

// MMAs over `steps` steps of 16 of the contraction for the term pairs
// (ta, tb), ta + tb <= MAXS, into `d` for the pair (0, 0) and `dc` for the
// others (dc may be d). An accumulation rounds at the size of the sum so far;
// the corrections are 2^-8 of the whole, so that in an accumulator of their own
// (where the result is fp32) they round at that much smaller a size. a, b:
// descriptors (a: TMEM address where TS) of step 0 of term 0; AT, AS, BT, BS:
// what a term and a step add. The whole warp takes the loop and the elected
// lane (`e`) the MMA: warp-uniform control flow keeps the operands in uniform
// registers, and a 128 x 128 x 16 MMA issues every 64 cycles, its rate; from
// one lane's branch it took 86 (and with descriptors built in place 198).
template <int TA, int TB, int MAXS, bool TS, int AT, int AS, int BT, int BS, typename A>
__device__ __forceinline__ void issue(bool e, uint32_t d, uint32_t dc, uint32_t id, int steps, bool acc, A a, uint64_t b) {
    bool accc = acc;
#pragma unroll
    for (int sum = MAXS; sum >= 0; --sum)
#pragma unroll
        for (int ta = 0; ta < TA; ++ta) {
            const int tb = sum - ta;
            if (tb < 0 || tb >= TB) continue;
            const bool main = sum == 0 && dc != d;
            const uint32_t dst = main ? d : dc;
            A pa = a + (A)(ta * AT);
            uint64_t pb = b + (uint64_t)(tb * BT);
            uint32_t ac = main ? acc : accc;
#pragma unroll 1
            for (int k = 0; k < steps; ++k) {
                if (e) {
                    if constexpr (TS) mma_ts(dst, pa, pb, id, ac);
                    else mma_ss(dst, pa, pb, id, ac);
                }
                pa += AS;
                pb += BS;
                ac = 1;
            }
            if (!main) accc = true;
        }
}

// A piece's rows: the table entry that owns index c of its numbering.
template <typename F>
__device__ __forceinline__ const LinWork &find_piece(const LinWorkTable &t, int c, F first) {
    int lo = 0, hi = t.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first(t.w[mid]) <= c) lo = mid;
        else hi = mid - 1;
    }
    return t.w[lo];
}

// A warp's 32 rows (a lane a row) of W 4-byte words to memory rows: through
// shared memory (W + 4 words a row), so that stores cover whole lines of a row.
constexpr int STAGE_WORDS = 32 * 36;
template <int W>
__device__ __forceinline__ void store_rows(uint32_t *stage, const uint32_t *x, void *dst, size_t stride, int nr, int width,
                                           int lane) {
    constexpr int LANES = W / 4, ROWS = 32 / LANES;   // 16-byte lanes of a row, rows of a store
    __syncwarp();
#pragma unroll
    for (int i = 0; i < LANES; ++i)
        *(uint4 *)(stage + lane * (W + 4) + 4 * i) = make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    __syncwarp();
    const int c = lane % LANES;
    if (16 * c < width) {
#pragma unroll
        for (int i = 0; i < 32 / ROWS; ++i) {
            const int r = ROWS * i + lane / LANES;
            if (r < nr) *(uint4 *)((char *)dst + r * stride + 16 * c) = *(const uint4 *)(stage + r * (W + 4) + 4 * c);
        }
    }
}

// Word i of a row of outputs y.
__device__ __forceinline__ uint32_t out_word(const float *, const float *y, int i) { return __float_as_uint(y[i]); }
__device__ __forceinline__ uint32_t out_word(const __nv_bfloat16 *, const float *y, int i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
    return *(const uint32_t *)&h;
}
__device__ __forceinline__ uint32_t out_word(const __half *, const float *y, int i) {
    const __half2 h = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
    return *(const uint32_t *)&h;
}

// Panels by TMA (one warp, all lanes): rows row .. row + ROWS - 1 and `boxes`
// blocks of 64 columns of each of NT terms of a row panel, term t to dst + t *
// PANEL, published on `full`. The MMAs take value rows up to the next multiple
// of 16 past nr under zero weights. A split panel holds zeros there; a bf16
// tensor is read in place, and its rows from nr on are another sequence's or
// padding, which under a zero weight would still spread a NaN: where nr cuts
// a step of 16 the rows are zeroed after the copy has landed, and the slot is
// published then.
template <int NT, int ROWS, int PANEL>
__device__ __forceinline__ void tma_panel(unsigned char *dst, const CUtensorMap *map, int col, int head, int row, int boxes,
                                          uint64_t *bar, int lane) {
    if (lane == 0)
        for (int t = 0; t < NT; ++t)
            for (int i = 0; i < boxes; ++i)
                tma_4d(dst + t * PANEL + i * ROWS * 128, map, col + 64 * i, head, row, t, bar);
}
template <int NT, int ROWS, int PANEL>
__device__ __forceinline__ bool tma_values(unsigned char *dst, const CUtensorMap *map, int col, int head, int row, int boxes,
                                           int nr, uint64_t *full, uint64_t *tail, uint32_t &tail_phase,
                                           volatile int *abort, int lane) {
    const bool cut = NT == 1 && nr < ROWS && nr % 16;
    uint64_t *bar = cut ? tail : full;
    if (lane == 0) mbar_expect_tx(bar, NT * boxes * ROWS * 128);
    tma_panel<NT, ROWS, PANEL>(dst, map, col, head, row, boxes, bar, lane);
    if (!cut) return true;
    __syncwarp();
    // in flight: waited for with the full limit
    const bool ok = warp_wait(tail, tail_phase, abort, O1_WAIT_CYCLES_FULL);
    if (!ok) mbar_drain(tail, tail_phase);
    tail_phase ^= 1;
    const int z = ceil16(nr) - nr;   // rows of zeros
    for (int i = lane; i < z * 8 * boxes; i += 32) {
        const int r = nr + (i >> 3) % z, b = (i >> 3) / z;
        *(uint4 *)(dst + b * ROWS * 128 + r * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(full);
    return ok;
}

// ------------------------------------------------------------------ split

// Rows of q, k and v as the bf16 terms the MMAs take (types of more than one
// term): panels [NT][prows][heads][width], a piece's rows from prow0 on, padded
// with zeros to a multiple of 16. A block a row. Done once, where each
// key would otherwise be split again by every tile, head and column block that
// reads it (12 times for 4 heads a group of 256 columns).
struct SplitArgs {
    uint16_t *q, *k, *v;
    int prows;
};
template <typename T>
__global__ __launch_bounds__(256) void k_lin_split(LinArgs a, const __grid_constant__ LinWorkTable t, SplitArgs s) {
    constexpr int NT = Terms<T>::in;
    o1_chain_wait();
    const int pr = blockIdx.x;
    const LinWork &w = find_piece(t, pr, [](const LinWork &p) { return p.prow0; });
    const int r = pr - w.prow0;
    const bool in = r < w.rows;
    const size_t row = (size_t)w.row0 + r;
    const int nq = a.nh * a.d / 8, nk = a.G * a.d / 8, nv = a.G * a.dv / 8;
    for (int i = threadIdx.x; i < nq + nk + nv; i += 256) {
        const T *src;
        uint16_t *dst;
        int n, c = i;
        if (c < nq) {
            src = (const T *)a.q + row * a.qs, dst = s.q, n = nq;
        } else if ((c -= nq) < nk) {
            src = (const T *)a.k + row * a.ks, dst = s.k, n = nk;
        } else {
            c -= nk;
            src = (const T *)a.v + row * a.vs, dst = s.v, n = nv;
        }
        uint4 raw[WORDS<T>];
#pragma unroll
        for (int j = 0; j < WORDS<T>; ++j) raw[j] = in ? ((const uint4 *)(src + 8 * c))[j] : make_uint4(0, 0, 0, 0);
        float x[8];
        words_floats(raw, x, (const T *)nullptr);
#pragma unroll
        for (int m = 0; m < NT; ++m) {
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = take_pair(x[2 * e], x[2 * e + 1]);
            *(uint4 *)(dst + ((size_t)m * s.prows + pr) * n * 8 + 8 * c) = make_uint4(y[0], y[1], y[2], y[3]);
        }
    }
    o1_chain_release();   // here, not at the top: the next kernel's CTAs, one an SM, would take this one's room
}

// ------------------------------------------------------------- increments

// One unit: dS[d0 .. +128][v0 .. +N] of (segment, head).
struct IncUnit {
    int row0, prow, nr, seg, h, g, d0, v0;   // prow: first row in the panels
};

// N columns of dv a unit: 256 for bf16 values (the weighted keys are then
// staged once for all of dv), 128 where values take more terms.
template <typename T, int N>
struct IncCfg {
    static constexpr int NT = Terms<T>::in;
    // accumulators: two, so that one is stored (7500 cycles for 256 columns)
    // while the other is summed: 36 -> 28 us a pass of 8192 bf16 rows of 8 heads
    // of 256. With 128 columns main and corrections apart (the state's
    // relative error over 600 rows 1.2e-7; in one, 256 columns, 1.6e-7)
    static constexpr int NB = 2, CORR = N == 128 ? 128 : 0, COLS = N + CORR;
    static constexpr int KSLOT = 3 * KV * TN * 2, NK = 2;
    static constexpr int VSLOT = NT * KV * N * 2, NV = NT == 3 ? 2 : 3;
    static constexpr int THREADS = 32 * (4 + 2 + PROD_WARPS);
    static constexpr size_t SMEM = 1024 + (size_t)NK * KSLOT + (size_t)NV * VSLOT + 4 * STAGE_WORDS * 4;
};

// dS of every (segment, head): A = weighted keys (M = d), B = values (N = dv),
// both MN-major, contraction over the rows, 64 of them a step. Persistent: a
// CTA takes units in turn. Warps: 0-3 store a finished unit, 4 issues the
// MMAs, 5 the values' TMA, 6-21 stage the weighted keys, running ahead over
// the rings.
template <typename T, int N>
__global__ __launch_bounds__((IncCfg<T, N>::THREADS), 1) void k_lin_inc(LinArgs a, const __grid_constant__ LinWorkTable t,
                                                                      const __grid_constant__ CUtensorMap mv, int units,
                                                                      float *inc) {
    using C = IncCfg<T, N>;
    constexpr int NT = C::NT, NK = C::NK, NV = C::NV;
    extern __shared__ unsigned char smraw[];
    __shared__ uint64_t kfull[NK], kempty[NK], vfull[NV], vempty[NV], done[2], freed[2], tail, fin;
    __shared__ uint32_t tslot;
    __shared__ int abort_s;
    __shared__ IncUnit list[LIST];
    volatile int *abort = &abort_s;
    unsigned char *sK = (unsigned char *)(((uintptr_t)smraw + 1023) & ~(uintptr_t)1023), *sV = sK + NK * C::KSLOT;
    uint32_t *stage = (uint32_t *)(sV + NV * C::VSLOT);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int count = (units - 1 - (int)blockIdx.x) / (int)gridDim.x + 1;   // <= LIST
    if (tid == 0) {
        for (int i = 0; i < NK; ++i) {
            mbar_init(&kfull[i], PROD_WARPS);
            mbar_init(&kempty[i], 1);
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(&vfull[i], 1);
            mbar_init(&vempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&done[i], 1);
            mbar_init(&freed[i], 4);
        }
        mbar_init(&tail, 1);
        mbar_init(&fin, 1);
        abort_s = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tmem_alloc512(&tslot);
    if (tid >= 64 && tid < 64 + count) {
        const int vt = (a.dv + N - 1) / N, dt = (a.d + TN - 1) / TN;
        int u = blockIdx.x + gridDim.x * (tid - 64);
        IncUnit x;
        x.v0 = (u % vt) * N;
        u /= vt;
        x.d0 = (u % dt) * TN;
        u /= dt;
        x.h = u % a.nh;
        x.g = x.h / a.hpg;
        x.seg = u / a.nh;
        const LinWork &w = find_piece(t, x.seg, [](const LinWork &p) { return p.seg0; });
        const int off = (x.seg - w.seg0) * a.seg;
        x.row0 = w.row0 + off;
        x.prow = (NT == 1 ? w.row0 : w.prow0) + off;
        x.nr = min(a.seg, w.rows - off);
        list[tid - 64] = x;
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = tslot;
    o1_chain_wait();   // the set-up above overlaps the kernel before
    const long long wl = a.wait_cycles;

    if (warp >= 6) {
        // ------------------------------------------------------- producers
        // the next panel's loads are in flight while one is stored
        using P = Panel<T, KV, TN>;
        const uint32_t pt = tid - 192, off = P::off(pt), prow = P::row(pt);
        uint4 ra[P::IT * WORDS<T>], rb[P::IT * WORDS<T>];
        int ik = 0;
        bool ok = true;
        auto load_k = [&](uint4 *r, const IncUnit &x, int s) {
            P::load(r, (const T *)a.k + (size_t)(x.row0 + KV * s) * a.ks + (size_t)x.g * a.d + x.d0, a.ks, x.nr - KV * s,
                    a.d - x.d0, pt);
        };
        float g = 0.f, gstep = 0.f;
        // weights e^{g (nr - 1 - row)} of the thread's rows, from the last
        // back; rows past the end are zeros under any finite weight
        auto store_k = [&](const uint4 *r, const IncUnit &x, int s) {
            const int b = ik % NK;
            ok = warp_wait(&kempty[b], ((ik / NK) & 1) ^ 1, abort, wl);
            if (!ok) return;
            const int last = x.nr - 1 - KV * s - (int)prow;
            float w[P::IT];
            w[P::IT - 1] = lin_pow(g, max(last - P::STEP * (P::IT - 1), 0));
#pragma unroll
            for (int i = P::IT - 2; i >= 0; --i)
                w[i] = last >= P::STEP * (i + 1) ? w[i + 1] * gstep : lin_pow(g, max(last - P::STEP * i, 0));
            P::template split<3>(r, sK + b * C::KSLOT + off, w);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&kfull[b]);
            ++ik;
        };
        IncUnit x = list[0], y;
        load_k(ra, x, 0);
        for (int n = 0; n < count && ok; ++n, x = y) {
            const int ns = (x.nr + KV - 1) / KV;
            g = a.decay[x.h];
            gstep = lin_pow(g, P::STEP);
            y = list[n + 1 < count ? n + 1 : n];
            // two buffers in turn, a unit's first panel in ra
            for (int s = 0; s < ns; s += 2) {
                if (s + 1 < ns) load_k(rb, x, s + 1);
                store_k(ra, x, s);
                if (!ok) break;
                if (s + 2 < ns) load_k(ra, x, s + 2);
                else if (n + 1 < count) load_k(ra, y, 0);
                if (s + 1 < ns) store_k(rb, x, s + 1);
                if (!ok) break;
            }
        }
    } else if (warp == 5) {
        // ------------------------------------------------- TMA of the values
        int iv = 0;
        uint32_t tp = 0;
        bool ok = true;
        for (int n = 0; n < count && ok; ++n) {
            const IncUnit x = list[n];
            const int boxes = (min(N, a.dv - x.v0) + 63) / 64;
            for (int s = 0; KV * s < x.nr && ok; ++s, ++iv) {
                const int b = iv % NV;
                ok = warp_wait(&vempty[b], ((iv / NV) & 1) ^ 1, abort, wl);
                if (!ok) break;
                ok = tma_values<NT, KV, KV * N * 2>(sV + b * C::VSLOT, &mv, x.v0, x.g, x.prow + KV * s, boxes, x.nr - KV * s,
                                                    &vfull[b], &tail, tp, abort, lane);
            }
        }
        // copies published on their slots are over before the block ends
        if (lane == 0)
            for (int i = max(0, iv - NV); i < iv; ++i) mbar_drain(&vfull[i % NV], (i / NV) & 1);
    } else if (warp == 4) {
        // ------------------------------------------------------ MMA issuer
        const bool e = elect_one();
        int it = 0;
        bool ok = true;
        const uint32_t k0 = su32(sK), v0 = su32(sV);
        constexpr int KTERM = KV * TN * 2 / 16, VTERM = KV * N * 2 / 16;
        for (int n = 0; n < count && ok; ++n) {
            const int nr = list[n].nr;
            const uint32_t id = idesc_bf16(128, min(N, ceil16(a.dv - list[n].v0)), 1, 1);
            const uint32_t d = tmem + (n % C::NB) * C::COLS;
            ok = warp_wait(&freed[n % C::NB], ((n / C::NB) & 1) ^ 1, abort, wl);
            for (int s = 0; KV * s < nr && ok; ++s, ++it) {
                const int bk = it % NK, bv = it % NV;
                ok = warp_wait(&kfull[bk], (it / NK) & 1, abort, wl) && warp_wait(&vfull[bv], (it / NV) & 1, abort, wl);
                if (!ok) break;
                tc_after();
                issue<3, NT, 2, false, KTERM, 128, VTERM, 128>(e, d, d + C::CORR, id, min(KV, ceil16(nr - KV * s)) / 16, s > 0,
                                                               desc_sw128_mn(k0 + bk * C::KSLOT, KV * 128),
                                                               desc_sw128_mn(v0 + bv * C::VSLOT, KV * 128));
                if (e) {
                    mma_commit(&kempty[bk]);
                    mma_commit(&vempty[bv]);
                }
            }
            if (ok && e) mma_commit(&done[n % C::NB]);
        }
        if (e) {
            mma_commit(&fin);   // tracks every MMA issued, also after an abort
            mbar_drain(&fin, 0);
        }
        __syncwarp();
    } else {
        // -------------------------------------------------------- epilogue
        bool ok = true;
        for (int n = 0; n < count; ++n) {
            const IncUnit x = list[n];
            const uint32_t lanes = tmem + (n % C::NB) * C::COLS + ((uint32_t)(32 * warp) << 16);
            if (ok) ok = warp_wait(&done[n % C::NB], (n / C::NB) & 1, abort, wl);
            tc_after();
            float *o = inc + ((size_t)x.seg * a.nh + x.h) * a.d * a.dv + (size_t)(x.d0 + 32 * warp) * a.dv + x.v0;
            const int nr = a.d - x.d0 - 32 * warp, wv = min(N, a.dv - x.v0);
#pragma unroll 1
            for (int c = 0; c < wv; c += 32) {
                uint32_t r0[32], r1[32];
                TMEM_LD32(lanes + c, r0);
                if (C::CORR) TMEM_LD32(lanes + C::CORR + c, r1);
                tmem_ld_wait();
                if (C::CORR) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) r0[i] = __float_as_uint(__uint_as_float(r0[i]) + __uint_as_float(r1[i]));
                }
                if (!ok) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) r0[i] = __float_as_uint(NAN);
                }
                store_rows<32>(stage + warp * STAGE_WORDS, r0, o + c, a.dv * 4, nr, 4 * (wv - c), lane);
            }
            tc_before();
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(&freed[n % C::NB]);
        }
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (warp == 0) tmem_free512(tmem);
    if (tid == 0 && abort_s) atomicOr(&lin_device_flags, (uint32_t)O1_FLAG_WAIT_EXPIRED);
}

// ------------------------------------------------------------------- scan

// Per state element, over a piece's segments: the increment is replaced by
// the state entering the segment, S <- l^n S + dS, the last S goes to its
// slot. The entering state is stored as the bf16 terms that the outputs
// multiply: two in the increment's own bytes, each row of dv values as dv
// first terms, then dv second ones (a row is one warp's, a lane the columns 4
// lane and, J = 2, 128 + 4 lane, so that it is read before it is overwritten),
// a third in `third` [states][d][dv]. Bound: the scratch's bytes, read and
// written once, as long as enough loads are out: a warp takes R rows and U
// segments at a time, and the next U are on their way while these are stored
// (one row and four segments a warp, loaded when the last four were stored: 17
// us instead of 14 for 32 segments of 2 MB, 189 instead of 40 for 64 sequences
// of one segment of 1 MB).
template <int MT, int R, int J>
__global__ __launch_bounds__(256, 2) void k_lin_scan(LinArgs a, const __grid_constant__ LinWorkTable t, float *inc,
                                                     uint16_t *third) {
    constexpr int U = 8 / (R * J);
    const LinWork w = t.w[blockIdx.z];
    const int h = blockIdx.y, row = (blockIdx.x * 8 + (threadIdx.x >> 5)) * R, lane = threadIdx.x & 31;
    if (row >= a.d) return;   // d is a multiple of R
    const size_t n = (size_t)a.d * a.dv, step = (size_t)a.nh * n;
    const int nc = (w.rows + a.seg - 1) / a.seg;
    const float gd = a.decay[h], full = lin_pow(gd, a.seg), last = lin_pow(gd, w.rows - (nc - 1) * a.seg);
    float *sp = a.state + ((size_t)w.slot * a.nh + h) * n + (size_t)row * a.dv;
    const size_t first = ((size_t)w.seg0 * a.nh + h) * n + (size_t)row * a.dv;
    float *p = inc + first;
    float4 s[R][J], x[U][R][J], y[U][R][J];
    bool in[J];
    auto load = [&](float4 (&z)[U][R][J], int c) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (c + u < nc && in[j]) z[u][r][j] = *(const float4 *)(p + (size_t)(c + u) * step + r * a.dv + 4 * lane + 128 * j);
    };
#pragma unroll
    for (int j = 0; j < J; ++j) in[j] = 4 * lane + 128 * j < a.dv;
    load(x, 0);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (in[j]) s[r][j] = *(const float4 *)(sp + r * a.dv + 4 * lane + 128 * j);
    for (int c = 0; c < nc; c += U) {
        load(y, c + U);
        __syncwarp();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (c + u >= nc) break;
            const float l = c + u == nc - 1 ? last : full;
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    if (!in[j]) continue;
                    const int col = 4 * lane + 128 * j;
                    float4 &e = s[r][j];
                    const float4 d = x[u][r][j];
                    float4 m = e;
                    const uint2 t0 = make_uint2(take_pair(m.x, m.y), take_pair(m.z, m.w));
                    const uint2 t1 = make_uint2(take_pair(m.x, m.y), take_pair(m.z, m.w));
                    const size_t at = (size_t)(c + u) * step + r * a.dv;
                    *(uint2 *)((uint16_t *)(p + at) + col) = t0;
                    *(uint2 *)((uint16_t *)(p + at) + a.dv + col) = t1;
                    if (MT == 3) *(uint2 *)(third + first + at + col) = make_uint2(take_pair(m.x, m.y), take_pair(m.z, m.w));
                    e = make_float4(fmaf(e.x, l, d.x), fmaf(e.y, l, d.y), fmaf(e.z, l, d.z), fmaf(e.w, l, d.w));
                }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int j = 0; j < J; ++j) x[u][r][j] = y[u][r][j];
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (in[j]) *(float4 *)(sp + r * a.dv + 4 * lane + 128 * j) = s[r][j];
    o1_chain_release();   // as in the split
}

template <int MT, int R, int J>
void scan_launch_r(const LinArgs &a, const LinWorkTable &t, float *inc, uint16_t *third, cudaStream_t st) {
    k_lin_scan<MT, R, J><<<dim3((a.d + 8 * R - 1) / (8 * R), a.nh, t.n), 256, 0, st>>>(a, t, inc, third);
}
// Rows of a warp: several where pieces have few segments to load ahead and the
// rows are many.
template <int MT, int J>
void scan_launch(const LinArgs &a, const LinWorkTable &t, int segs, float *inc, uint16_t *third, cudaStream_t st) {
    int R = segs <= 2 * t.n ? 4 / J : segs <= 4 * t.n ? 2 : 1;
    while (R > 1 && (int64_t)a.d * a.nh * t.n < (int64_t)R * LIN_SMS * 16) R /= 2;
    if (R == 1) scan_launch_r<MT, 1, J>(a, t, inc, third, st);
    else if (R == 2) scan_launch_r<MT, 2, J>(a, t, inc, third, st);
    else if constexpr (J == 1) scan_launch_r<MT, 4, J>(a, t, inc, third, st);
}

// ---------------------------------------------------------------- outputs

// Warps: 0-7 P (a thread a row and half of its columns), 8-11 epilogue, 12 MMA
// issuer, 13 TMA. One CTA an SM: two with half the ring and TMEM each took 57
// us a pass instead of 48.
constexpr int P_WARPS = 8, OUT_THREADS = 32 * (P_WARPS + 6);
template <typename T>
struct OutCfg {
    static constexpr int NT = Terms<T>::in, MT = Terms<T>::mid;
    static constexpr bool PAIR = NT == 1;      // Q and K of a step share a slot
    static constexpr int DK = 64;              // values of d a step: a block of the panels
    static constexpr int SLOT = NT == 3 ? 49152 : 32768, NSLOT = NT == 3 ? 4 : 6;
    static constexpr int VR = NT == 1 ? 128 : 64;   // value rows of a slot
    static constexpr bool SPLIT = NT == 3;     // corrections in accumulators of their own
    // TMEM: outputs ACC (two buffers; SPLIT: one, main and corrections), then
    // scores X (two buffers; SPLIT: one, main and corrections). P overlays X.
    static constexpr int XB = SPLIT ? 1 : 2, AB = SPLIT ? 1 : 2;
    static constexpr size_t SMEM = 1024 + (size_t)NSLOT * SLOT + 4 * STAGE_WORDS * 4;
    static __device__ __forceinline__ uint32_t acc(int n) { return SPLIT ? 0u : 128u * (n & 1); }
    static __device__ __forceinline__ uint32_t x(int u) { return 256u + (SPLIT ? 0u : 128u * (u & 1)); }
    static constexpr uint32_t CORR = SPLIT ? 128u : 0u;
};

// One P warp's powers of a head's decay l.
struct alignas(16) Powers {
    float col[32];                    // l^{31 - i}
    float pow[32 + LIN_CHUNK + 1];    // l^i from 32 on; zeros before, read by lanes left of the diagonal
    __device__ __forceinline__ float at(int i) const { return pow[32 + i]; }
    __device__ __forceinline__ void fill(float g, int lane) {
        __syncwarp();
        col[lane] = lin_pow(g, 31 - lane);
        pow[lane] = 0.f;
        for (int i = lane; i <= LIN_CHUNK; i += 32) pow[32 + i] = lin_pow(g, i);
        __syncwarp();
    }
};

// One tile: 128 query rows x 128 value columns of a head; its units are the
// key tiles kt = 0 .. nkt - 1 of the segment up to its own rows (the last).
struct OutTile {
    int row0, nr;        // query rows
    int prow, kprow;     // in the panels: the tile's and its segment's first row
    int i0, seg;         // row in the segment; the segment's state
    int h, g, v0, nkt;   // nkt: 1 or 2 (LIN_SEG rows a segment at most)
    int nv;              // value columns, rounded to 16
};
struct Cursor {
    int n, u, kt;        // tile of the list, units so far, key tile
    OutTile x;
    __device__ __forceinline__ void start(const OutTile *list) {
        n = u = kt = 0;
        x = list[0];
    }
    // the next unit: false after the last
    __device__ __forceinline__ bool next(const OutTile *list, int count) {
        ++u;
        if (++kt < x.nkt) return true;
        kt = 0;
        if (++n >= count) return false;
        x = list[n];
        return true;
    }
    __device__ __forceinline__ bool diag() const { return kt == x.nkt - 1; }
    __device__ __forceinline__ int keys() const { return diag() ? x.nr : LIN_CHUNK; }
    __device__ __forceinline__ int key0() const { return x.kprow + LIN_CHUNK * kt; }
};

// Outputs. Weights: with i0 the tile's first row and s0 its segment's,
//   o_i = l^{i-s0+1} q_i S_in + sum_{j<i0} l^{i-i0+1} l^{i0-1-j} s_ij v_j
//         + sum_{i0<=j<=i} l^{i-j} s_ij v_j
// so the accumulator is weighted once, by row, after q S_in, the earlier key
// tiles' scores by row and column. The MMA thread issues the next unit's scores (and a
// next tile's q S_in) ahead of this unit's P V where TMEM holds two score
// buffers, so that P is formed under them.
template <typename T>
__global__ __launch_bounds__(OUT_THREADS, 1) void k_lin_out(LinArgs a, const __grid_constant__ LinWorkTable t,
                                                            const __grid_constant__ CUtensorMap mq,
                                                            const __grid_constant__ CUtensorMap mk,
                                                            const __grid_constant__ CUtensorMap mv,
                                                            const __grid_constant__ CUtensorMap ms,
                                                            const __grid_constant__ CUtensorMap ms3, int tiles) {
    using C = OutCfg<T>;
    constexpr int NT = C::NT, MT = C::MT;
    extern __shared__ unsigned char smraw[];
    __shared__ uint64_t full[C::NSLOT], empty[C::NSLOT], sc_full[2], p_full[2], acc_ready[2], o_done[2], acc_free[2], tail,
        fin;
    __shared__ uint32_t tslot;
    __shared__ int abort_s;
    __shared__ Powers powers[P_WARPS];
    __shared__ OutTile list[LIST];
    volatile int *abort = &abort_s;
    unsigned char *sm = (unsigned char *)(((uintptr_t)smraw + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int count = (tiles - 1 - (int)blockIdx.x) / (int)gridDim.x + 1;   // <= LIST
    if (tid == 0) {
        for (int i = 0; i < C::NSLOT; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sc_full[i], 1);
            mbar_init(&p_full[i], P_WARPS);
            mbar_init(&acc_ready[i], 1);
            mbar_init(&o_done[i], 1);
            mbar_init(&acc_free[i], 4);
        }
        mbar_init(&tail, 1);
        mbar_init(&fin, 1);
        abort_s = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tmem_alloc512(&tslot);
    if (tid >= 64 && tid < 64 + count) {
        const int vt = (a.dv + TN - 1) / TN;
        int c = blockIdx.x + gridDim.x * (tid - 64);
        OutTile x;
        x.v0 = (c % vt) * TN;
        c /= vt;
        x.h = c % a.nh;
        x.g = x.h / a.hpg;
        c /= a.nh;
        const LinWork &w = find_piece(t, c, [](const LinWork &p) { return p.tile0; });
        const int off = (c - w.tile0) * LIN_CHUNK, sl = off / a.seg;
        x.row0 = w.row0 + off;
        x.nr = min(LIN_CHUNK, w.rows - off);
        x.seg = w.seg0 + sl;
        x.i0 = off - sl * a.seg;
        x.prow = (NT == 1 ? w.row0 : w.prow0) + off;
        x.kprow = x.prow - x.i0;
        x.nkt = x.i0 / LIN_CHUNK + 1;
        x.nv = min(TN, ceil16(a.dv - x.v0));
        list[tid - 64] = x;
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = tslot;
    o1_chain_wait();   // the set-up above overlaps the scan
    const long long wl = a.wait_cycles;
    const int nb = (a.d + C::DK - 1) / C::DK;   // steps of d

    if (warp == P_WARPS + 4) {
        // ------------------------------------------------------ MMA issuer
        // Ring items in order: per unit, for each step of d the Q and K
        // panels and (first unit of a tile) the entering state's; the unit's
        // values (a unit later where scores run ahead). The tensor pipe holds
        // an MMA or two, so what this warp does between them shows: positions
        // are carried, not computed.
        const bool e = elect_one();
        bool ok = true, vq = true, vv = true;
        Cursor cq, cv;
        cq.start(list);
        cv.start(list);
        const uint32_t base = su32(sm);
        const uint64_t dk = desc_sw128(base), ds = desc_sw128_mn(base, C::DK * 128), dv = desc_sw128_mn(base, C::VR * 128);
        const uint32_t id_x = idesc_bf16(128, 128, 0, 0);
        int slot = 0;              // of the next ring item
        uint32_t phase = 0;
        auto take = [&]() -> int {   // the next item's slot, once filled
            const int s = slot;
            ok = ok && warp_wait(&full[s], phase, abort, wl);
            if (++slot == C::NSLOT) slot = 0, phase ^= 1;
            return s;
        };
        auto commit = [&](uint64_t *bar) {
            if (e) mma_commit(bar);
        };
        // scores of a unit, and with a tile's first unit its q S_in; 64
        // columns of Q and K (a block of their panels) at a time
        auto scores = [&]() {
            const int n = cq.n % C::AB;
            const uint32_t x = tmem + C::x(cq.u), acc = tmem + C::acc(cq.n), id_a = idesc_bf16(128, cq.x.nv, 0, 1);
            const bool state = cq.kt == 0;
#pragma unroll 1
            for (int b = 0; b < nb; ++b) {
                const int steps = (min(C::DK, a.d - C::DK * b) + 15) / 16, sq = take(), sk = C::PAIR ? sq : take();
                if (!ok) return;
                tc_after();
                const uint64_t qd = dk + (uint64_t)(sq * (C::SLOT / 16));
                const uint64_t kd = C::PAIR ? qd + C::DK * 16 : dk + (uint64_t)(sk * (C::SLOT / 16));
                issue<NT, NT, NT - 1, false, 1024, 2, 1024, 2>(e, x, x + C::CORR, id_x, steps, b > 0, qd, kd);
                if (!C::PAIR) commit(&empty[sk]);
                if (b == nb - 1) commit(&sc_full[cq.u % C::XB]);
                if (state) {
                    if (b == 0) ok = warp_wait(&acc_free[n], ((cq.n / C::AB) & 1) ^ 1, abort, wl);
                    const int ss = take();
                    if (!ok) return;
                    tc_after();
                    const uint64_t sd = ds + (uint64_t)(ss * (C::SLOT / 16));
                    issue<NT, MT, max_sum(NT, MT), false, 1024, 2, C::DK * TN * 2 / 16, 128>(e, acc, acc + C::CORR, id_a, steps,
                                                                                             b > 0, qd, sd);
                    commit(&empty[ss]);
                }
                commit(&empty[sq]);
            }
            if (state) commit(&acc_ready[n]);
            vq = cq.next(list, count);
        };
        auto values = [&]() {
            const uint32_t x = tmem + C::x(cv.u), acc = tmem + C::acc(cv.n), id_a = idesc_bf16(128, cv.x.nv, 0, 1);
            const int keys = (cv.keys() + 15) / 16;   // steps
            ok = warp_wait(&p_full[cv.u % C::XB], (cv.u / C::XB) & 1, abort, wl);
#pragma unroll 1
            for (int i = 0; i < LIN_CHUNK / C::VR; ++i) {
                const int sv = take();
                if (!ok) return;
                tc_after();
                const int steps = min(C::VR / 16, keys - C::VR / 16 * i);
                const uint64_t vd = dv + (uint64_t)(sv * (C::SLOT / 16));
                constexpr int TERM = C::VR * TN * 2 / 16;
                if (steps > 0) {
                    // P's terms 0 and 1 of 16 keys are 16 columns; the third's 8 lie apart
                    if constexpr (MT == 3)
                        issue<1, 1, 0, true, 0, 8, 0, 128>(e, acc + C::CORR, acc + C::CORR, id_a, steps, true,
                                                           x + 128 + C::VR * i, vd);
                    issue<2, NT, max_sum(MT, NT), true, 8, 16, TERM, 128>(e, acc, acc + C::CORR, id_a, steps, true,
                                                                         x + C::VR * i, vd);
                }
                commit(&empty[sv]);
            }
            if (cv.diag()) commit(&o_done[cv.n % C::AB]);
            vv = cv.next(list, count);
        };
        for (int ahead = 0; vv && ok;) {   // units scored, their P V not issued
            if (vq && ahead < C::XB) {
                scores();
                ++ahead;
            } else {
                values();
                --ahead;
            }
        }
        if (e) {
            mma_commit(&fin);   // tracks every MMA issued, also after an abort
            mbar_drain(&fin, 0);
        }
        __syncwarp();
    } else if (warp > P_WARPS + 4) {
        // ------------------------------------------------------------- TMA
        int it = 0;
        bool ok = true, vq = true, vv = true;
        uint32_t tp = 0;
        Cursor cq, cv;
        cq.start(list);
        cv.start(list);
        uint64_t *f = full;
        auto slot = [&]() -> unsigned char * {   // the next item's, once free
            const int s = it % C::NSLOT;
            ok = ok && warp_wait(&empty[s], ((it / C::NSLOT) & 1) ^ 1, abort, wl);
            f = &full[s];
            if (ok) ++it;
            return sm + (size_t)s * C::SLOT;
        };
        auto expect = [&](int bytes) {
            if (lane == 0) mbar_expect_tx(f, bytes);
        };
        auto scores = [&]() {
            const int vb = (cq.x.nv + 63) / 64, state = cq.x.seg * a.nh + cq.x.h;
            for (int b = 0; b < nb; ++b) {
                unsigned char *d = slot();
                if (!ok) return;
                expect(16384 * (C::PAIR ? 2 : NT));
                tma_panel<NT, 128, 16384>(d, &mq, C::DK * b, cq.x.h, cq.x.prow, 1, f, lane);
                if (C::PAIR) {
                    d += C::DK * 256;
                } else {
                    d = slot();
                    if (!ok) return;
                    expect(16384 * NT);
                }
                tma_panel<NT, 128, 16384>(d, &mk, C::DK * b, cq.x.g, cq.key0(), 1, f, lane);
                if (cq.kt == 0) {
                    d = slot();
                    if (!ok) return;
                    expect(MT * vb * C::DK * 128);
                    if (lane == 0)
                        for (int m = 0; m < MT; ++m)
                            for (int i = 0; i < vb; ++i)
                                tma_4d(d + C::DK * (256 * m + 128 * i), m < 2 ? &ms : &ms3, cq.x.v0 + 64 * i, m < 2 ? m : 0,
                                       C::DK * b, state, f);
                }
            }
            vq = cq.next(list, count);
        };
        auto values = [&]() {
            for (int i = 0; i < LIN_CHUNK / C::VR; ++i) {
                unsigned char *d = slot();
                if (!ok) return;
                ok = tma_values<NT, C::VR, C::VR * TN * 2>(d, &mv, cv.x.v0, cv.x.g, cv.key0() + C::VR * i,
                                                           (cv.x.nv + 63) / 64, cv.keys() - C::VR * i, f, &tail,
                                                           tp, abort, lane);
                if (!ok) return;
            }
            vv = cv.next(list, count);
        };
        for (int ahead = 0; vv && ok;) {   // in the MMA issuer's order
            if (vq && ahead < C::XB) {
                scores();
                ++ahead;
            } else {
                values();
                --ahead;
            }
        }
        // copies are over before the block ends
        if (lane == 0)
            for (int i = max(0, it - C::NSLOT); i < it; ++i) mbar_drain(&full[i % C::NSLOT], (i / C::NSLOT) & 1);
    } else if (warp < P_WARPS) {
        // --------------------------------------------------------------- P
        Cursor c;
        c.start(list);
        bool have = true, ok = true;
        const int r0 = 32 * (warp & 3), row = r0 + lane, c0 = 64 * (warp >> 2);   // this warp's rows and columns
        const uint32_t lanes = tmem + ((uint32_t)r0 << 16);
        int table = -1;   // head of the power table
        Powers &pw = powers[warp];
        float g = 0.f;
        uint32_t rp[2] = {0, 0};   // phases of acc_ready, one a tile
        // the accumulator times f, once what it holds so far is complete
        auto weight = [&](float f) -> bool {
            const int i = c.n % C::AB;
            if (!warp_wait(&acc_ready[i], i ? rp[1] : rp[0], abort, wl)) return false;
            if (i) rp[1] ^= 1;
            else rp[0] ^= 1;
            tc_after();
            const int wv = min(c0 + 64, c.x.nv);
            for (int half = 0; half <= (C::SPLIT ? 1 : 0); ++half)
#pragma unroll 1
                for (int cb = c0; cb < wv; cb += 32) {
                    const uint32_t ad = lanes + C::acc(c.n) + 128 * half + cb;
                    uint32_t r[32];
                    TMEM_LD32(ad, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
                    TMEM_ST32(ad, r);
                }
            return true;
        };
        while (have && ok) {
            if (table != c.x.h) {
                table = c.x.h;
                g = a.decay[table];
                pw.fill(g, lane);
            }
            ok = warp_wait(&sc_full[c.u % C::XB], (c.u / C::XB) & 1, abort, wl);
            if (!ok) break;
            tc_after();
            const bool diag = c.diag();
            // weights: l^{row - j} up to the diagonal; for the tile before
            // l^{127 - j} for all its keys, and l^{row + 1}
            const int base = diag ? row : LIN_CHUNK - 1;
            const float tf = diag ? 1.f : pw.at(row + 1);
            const uint32_t x = lanes + C::x(c.u);
            // P over the scores of the same keys; a third term of 32 keys
            // takes 16 columns of the corrections, of keys this warp has read.
            // Left of the diagonal a block's weights are a power of the column
            // (one for all lanes, four a load) times one of the row.
#pragma unroll 1
            for (int cb = c0; cb < c0 + 64; cb += 32) {
                uint32_t r[32], third[16];
                float s[32];
                TMEM_LD32(x + cb, r);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) s[i] = __uint_as_float(r[i]);
                if (C::SPLIT) {
                    TMEM_LD32(x + C::CORR + cb, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i) s[i] += __uint_as_float(r[i]);
                }
                if (!diag || cb < r0) {
                    const float f = pw.at(base - cb - 31) * tf;
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 w = *(const float4 *)(pw.col + i);
                        s[i] *= w.x * f;
                        s[i + 1] *= w.y * f;
                        s[i + 2] *= w.z * f;
                        s[i + 3] *= w.w * f;
                    }
                } else if (cb == r0) {
                    const float *w = pw.pow + 32 + lane;
#pragma unroll
                    for (int i = 0; i < 32; ++i) s[i] = i <= lane ? s[i] * w[-i] : 0.f;
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) s[i] = 0.f;
                }
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float &x0 = s[16 * q + 2 * e], &x1 = s[16 * q + 2 * e + 1];
                        r[16 * q + e] = take_pair(x0, x1);
                        r[16 * q + 8 + e] = take_pair(x0, x1);
                        if (C::SPLIT) third[8 * q + e] = take_pair(x0, x1);
                    }
                __syncwarp();   // the warp is together for the stores
                TMEM_ST32(x + cb, r);
                if (C::SPLIT) TMEM_ST16(x + 128 + c0 + (cb - c0) / 2, third);
            }
            if (c.kt == 0) ok = weight(lin_pow(g, c.x.i0) * pw.at(row + 1));
            if (!ok) break;
            tmem_st_wait();
            tc_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[c.u % C::XB]);
            have = c.next(list, count);
        }
        if (!ok) tmem_st_wait();   // stores issued before a wait ran out are over before the TMEM is given back
    } else {
        // -------------------------------------------------------- epilogue
        // The accumulator is read into registers, as output words, and given
        // back before the stores (fp32: half of it at a time).
        constexpr int W = 8 * sizeof(T), B = sizeof(T) == 2 ? 4 : 2;   // words of 32 columns; such blocks held
        uint32_t *stage = (uint32_t *)(sm + (size_t)C::NSLOT * C::SLOT) + (warp & 3) * STAGE_WORDS;
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        bool ok = true;
        for (int n = 0; n < count; ++n) {
            const OutTile x = list[n];
            if (ok) ok = warp_wait(&o_done[n % C::AB], (n / C::AB) & 1, abort, wl);
            tc_after();
            T *o = (T *)a.out + (size_t)(x.row0 + 32 * (warp & 3)) * a.os + (size_t)x.h * a.dv + x.v0;
            const int nr = x.nr - 32 * (warp & 3), wv = min(TN, a.dv - x.v0);
#pragma unroll 1
            for (int c0 = 0; c0 < TN; c0 += 32 * B) {
                uint32_t w[B * W];
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    const uint32_t ad = lanes + C::acc(n) + c0 + 32 * b;
                    uint32_t r[32];
                    float y[32];
                    TMEM_LD32(ad, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i) y[i] = __uint_as_float(r[i]);
                    if (C::SPLIT) {
                        TMEM_LD32(ad + C::CORR, r);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) y[i] += __uint_as_float(r[i]);
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) y[i] = ok ? y[i] * a.scale : NAN;
#pragma unroll
                    for (int i = 0; i < W; ++i) w[b * W + i] = out_word((const T *)nullptr, y, i);
                }
                if (c0 + 32 * B == TN) {
                    tc_before();
                    __syncwarp();
                    if (ok && lane == 0) mbar_arrive(&acc_free[n % C::AB]);
                }
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    const int c = c0 + 32 * b;
                    if (c < wv)
                        store_rows<W>(stage, w + b * W, o + c, a.os * sizeof(T), nr, (wv - c) * (int)sizeof(T), lane);
                }
            }
        }
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (warp == 0) tmem_free512(tmem);
    if (tid == 0 && abort_s) atomicOr(&lin_device_flags, (uint32_t)O1_FLAG_WAIT_EXPIRED);
}

// ----------------------------------------------------------------- launch

bool encode(CUtensorMap *m, const void *base, const cuuint64_t *dims, const cuuint64_t *strides, int rows_dim, int rows) {
    const auto enc = tensor_map_encoder();
    cuuint32_t boxes[4] = {64, 1, 1, 1}, es[4] = {1, 1, 1, 1};
    boxes[rows_dim] = (cuuint32_t)rows;
    return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, (void *)base, dims, strides, boxes, es,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// A row panel [terms][rows][heads][width] in boxes of 64 columns of `box` rows.
bool rows_map(CUtensorMap *m, const void *base, int width, int heads, int rows, size_t stride, int terms, int box) {
    const cuuint64_t dims[4] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)rows, (cuuint64_t)terms};
    const cuuint64_t strides[3] = {(cuuint64_t)width * 2, (cuuint64_t)stride * 2, (cuuint64_t)rows * stride * 2};
    return encode(m, base, dims, strides, 2, box);
}
// Entering states as the scan leaves them: [states][d][terms][dv].
bool states_map(CUtensorMap *m, const void *base, const LinArgs &a, int states, int terms, int box) {
    const cuuint64_t dims[4] = {(cuuint64_t)a.dv, (cuuint64_t)terms, (cuuint64_t)a.d, (cuuint64_t)states};
    const cuuint64_t row = (cuuint64_t)a.dv * 2 * terms;
    const cuuint64_t strides[3] = {(cuuint64_t)a.dv * 2, row, a.d * row};
    return encode(m, base, dims, strides, 2, box);
}

// CTAs of a persistent grid: one an SM, more where a CTA's list would overflow.
int grid_of(int units) {
    const int ctas = units < LIN_SMS ? units : LIN_SMS, need = (units + LIST - 1) / LIST;
    return ctas > need ? ctas : need;
}

template <typename T, int N>
bool pass_t(const LinArgs &a, const LinWorkTable &t, int dtype, int segs, int tiles, int prows, void *scratch, bool first,
            cudaStream_t st) {
    using CI = IncCfg<T, N>;
    using CO = OutCfg<T>;
    static unsigned long long done = 0;
    unsigned long long bit = 0;
    if (o1_attrs_needed(&done, &bit)) {
        cudaFuncSetAttribute(k_lin_inc<T, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)CI::SMEM);
        cudaFuncSetAttribute(k_lin_out<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)CO::SMEM);
        o1_attrs_done(&done, bit);
    }
    // the pass's scratch: increments and entering states, third terms, panels
    char *at = (char *)scratch;
    float *inc = (float *)at;
    at += lin_pass_states(a.nh, a.d, a.dv, dtype, segs).inc;
    uint16_t *third = (uint16_t *)at;
    at += lin_pass_states(a.nh, a.d, a.dv, dtype, segs).third;
    SplitArgs sp = {};
    const void *q = a.q, *k = a.k, *v = a.v;
    size_t qs = a.qs, ks = a.ks, vs = a.vs;
    int rows = a.rows;
    if (CO::NT > 1) {
        rows = prows;
        qs = (size_t)a.nh * a.d;
        ks = (size_t)a.G * a.d;
        vs = (size_t)a.G * a.dv;
        const size_t n = (size_t)prows * CO::NT;
        q = sp.q = (uint16_t *)at;
        k = sp.k = sp.q + n * qs;
        v = sp.v = sp.k + n * ks;
        sp.prows = prows;
    }
    CUtensorMap mq, mk, mv, mvi, ms, ms3;
    if (!rows_map(&mq, q, a.d, a.nh, rows, qs, CO::NT, LIN_CHUNK) || !rows_map(&mk, k, a.d, a.G, rows, ks, CO::NT, LIN_CHUNK) ||
        !rows_map(&mv, v, a.dv, a.G, rows, vs, CO::NT, CO::VR) || !rows_map(&mvi, v, a.dv, a.G, rows, vs, CO::NT, KV) ||
        !states_map(&ms, inc, a, segs * a.nh, 2, CO::DK))
        return false;
    ms3 = ms;
    if (CO::MT == 3 && !states_map(&ms3, third, a, segs * a.nh, 1, CO::DK)) return false;
    const int dt = (a.d + TN - 1) / TN, units = segs * a.nh * dt * ((a.dv + N - 1) / N);
    const int ot = tiles * a.nh * ((a.dv + TN - 1) / TN);
    // Chained launches: a kernel's set-up runs under the end of the one before
    // (1024 fp32 rows 45.5 -> 43 us). Not the first of a call (64 fp32 rows in a
    // loop 23.3 -> 27.2 us, in a graph 21.3 -> 21.6), since what ran before it is
    // unknown: a chained kernel waits for the one kernel before it, which may
    // itself have been chained and not have waited; and one that lets its
    // successor start and takes tensor memory only then would wait for ever on
    // an SM whose tensor memory k_lin_inc already holds. Not the scan: its
    // blocks, small and many, would pile up on the SMs that finish first (1024
    // bf16 rows of 256 columns 24.6 -> 27 us).
    if constexpr (CO::NT > 1) o1_launch_chained(!first, k_lin_split<T>, dim3(prows), dim3(256), 0, st, a, t, sp);
    o1_launch_chained(CO::NT > 1 || !first, k_lin_inc<T, N>, dim3(grid_of(units)), dim3(CI::THREADS), CI::SMEM, st, a, t, mvi, units, inc);
    if (a.dv > 128) scan_launch<CO::MT, 2>(a, t, segs, inc, third, st);
    else scan_launch<CO::MT, 1>(a, t, segs, inc, third, st);
    o1_launch_chained(true, k_lin_out<T>, dim3(grid_of(ot)), dim3(OUT_THREADS), CO::SMEM, st, a, t, mq, mk, mv, ms, ms3, ot);
    return true;
}

}  // namespace

bool lin_launch_pass(const LinArgs &a, int dtype, const LinWorkTable &t, int segs, int tiles, int prows, void *scratch,
                     bool first, cudaStream_t st) {
    if (dtype == O1_F32) return pass_t<float, 128>(a, t, dtype, segs, tiles, prows, scratch, first, st);
    if (dtype == O1_F16) return pass_t<__half, 128>(a, t, dtype, segs, tiles, prows, scratch, first, st);
    return a.dv > 128 ? pass_t<__nv_bfloat16, 256>(a, t, dtype, segs, tiles, prows, scratch, first, st)
                      : pass_t<__nv_bfloat16, 128>(a, t, dtype, segs, tiles, prows, scratch, first, st);
}

// The word is reset only where it was read as raised, after the read is over: a
// flag that a kernel on another stream raises in between is then the one that
// is reported, and none is dropped unread.
int lin_flags(uint32_t *flags, int clear, cudaStream_t st) {
    if (cudaMemcpyFromSymbolAsync(flags, lin_device_flags, sizeof(uint32_t), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return O1_ERR_CUDA;
    if (!clear || !*flags) return O1_OK;
    static const uint32_t zero = 0;
    if (cudaMemcpyToSymbolAsync(lin_device_flags, &zero, sizeof(uint32_t), 0, cudaMemcpyHostToDevice, st) != cudaSuccess)
        return O1_ERR_CUDA;
    return cudaStreamSynchronize(st) == cudaSuccess ? O1_OK : O1_ERR_CUDA;
}
