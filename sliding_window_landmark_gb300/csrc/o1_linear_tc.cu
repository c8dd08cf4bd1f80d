// Linear attention with a decay per head over prompts, on the tensor cores.
//
// The recurrence S = l S + k v^T, o = q S over a chunk of C = 128 rows with
// entering state S_in (l = e^{log_decay}):
//   o_i   = l^{i+1} q_i S_in + sum_{j <= i} l^{i-j} (q_i . k_j) v_j
//   S_out = l^n S_in + dS,   dS = sum_j (l^{n-1-j} k_j) v_j^T   (n rows)
// so that only the chunk states are sequential:
//   k_lin_inc   dS of every (chunk, head): one product of depth n
//   k_lin_scan  per state element, over the chunks of a sequence: dS is
//               replaced by the state entering the chunk, and the last state
//               goes to its slot
//   k_lin_out   every (chunk, head)'s outputs: scores Q K^T, weighted and
//               masked into P; acc = Q S_in, then P V; o joins the two with
//               the row's decay in fp32
// No step carries a weight above 1 (every power of l has an exponent >= 0), so
// nothing overflows whatever the decay.
//
// Precision. The MMAs take bf16 operands with fp32 accumulation. An fp32
// value is split into three bf16 terms (x = x0 + x1 + x2 exactly but for
// 2^-24, each the bf16 of what the earlier leave; the subtractions are exact), an fp16
// value into two (exactly), a bf16 value is one; of a product's term pairs
// those down to 2^-16 (two terms) or 2^-24 (three) are taken. bf16 terms have
// fp32's exponent range, so no scaling is needed. States are fp32 sums: the
// weighted keys l^{n-1-j} k_j are always three terms. The entering state and P
// only reach the outputs: two terms where those are 16-bit, three for fp32.
//
// Layout. All panels are [rows][128 columns] of bf16 in two blocks of 64
// columns, 128-byte swizzled, and serve as K-major or MN-major operands as
// they lie: the keys are K-major for the scores and (weighted) MN-major for
// dS, values and S_in are MN-major. Threads stage them, since every operand but a bf16 one
// is split or weighted on the way. A chunk's rows past its sequence's end are
// staged as zeros: what lies there is never multiplied.
#include <math.h>

#include "o1_linear.cuh"
#include "o1_tc.cuh"

static __device__ uint32_t lin_device_flags;

namespace {

constexpr int COLS = 128;   // columns of a panel: d or dv of one tile

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

struct Chunk {
    int row0, nr;   // rows row0 .. row0 + nr - 1
};
__device__ __forceinline__ Chunk find_chunk(const LinWorkTable &t, int c) {
    int lo = 0, hi = t.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.w[mid].chunk0 <= c) lo = mid;
        else hi = mid - 1;
    }
    const int off = (c - t.w[lo].chunk0) * LIN_CHUNK;
    return {t.w[lo].row0 + off, min(LIN_CHUNK, t.w[lo].rows - off)};
}

// 8 consecutive values as loaded
struct Raw32 {
    float4 a, b;
};
template <typename T>
struct RawOf {
    using type = uint4;
};
template <>
struct RawOf<float> {
    using type = Raw32;
};
__device__ __forceinline__ void raw_zero(uint4 &r) { r = make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void raw_zero(Raw32 &r) { r.a = r.b = make_float4(0.f, 0.f, 0.f, 0.f); }
__device__ __forceinline__ void raw_load(uint4 &r, const void *p) { r = *(const uint4 *)p; }
__device__ __forceinline__ void raw_load(Raw32 &r, const void *p) {
    r.a = ((const float4 *)p)[0];
    r.b = ((const float4 *)p)[1];
}
__device__ __forceinline__ void raw_floats(const Raw32 &r, float (&x)[8], const float *) {
    x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w;
    x[4] = r.b.x; x[5] = r.b.y; x[6] = r.b.z; x[7] = r.b.w;
}
__device__ __forceinline__ void raw_floats(const uint4 &r, float (&x)[8], const __nv_bfloat16 *) {
    const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void raw_floats(const uint4 &r, float (&x)[8], const __half *) {
    const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*(const __half2 *)&u[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// x[8] as NT bf16 terms, term t's 16 bytes at dst + t * panel
template <int NT>
__device__ __forceinline__ void store_terms(unsigned char *dst, size_t panel, float (&x)[8]) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *(const uint32_t *)&h;
            if (t + 1 < NT) {
                x[2 * i] -= __uint_as_float(w[i] << 16);
                x[2 * i + 1] -= __uint_as_float(w[i] & 0xffff0000u);
            }
        }
        *(uint4 *)(dst + t * panel) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Byte offset of the 8-column group cg of row r in a panel of `rows` rows.
__device__ __forceinline__ uint32_t panel_off(int rows, int r, int cg) {
    return (uint32_t)((cg >> 3) * rows * 128 + r * 128 + (((cg & 7) ^ (r & 7)) << 4));
}

// A tile of ROWS rows in flight from global memory to a panel: 8-column
// groups in order along a row, NTHR threads. cgs: groups per row as a power of
// two (8 or 16), so that narrow tiles keep all threads busy.
template <typename T, int ROWS, int NTHR>
struct Tile {
    static constexpr int IT = ROWS * (COLS / 8) / NTHR;
    typename RawOf<T>::type raw[IT];

    // rows [0, nr) and columns [0, width) of src (row stride in values); the rest reads as zero
    __device__ __forceinline__ void load(const T *src, size_t stride, int nr, int width, int cgs) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int item = threadIdx.x + NTHR * i, r = cgs == 8 ? item >> 3 : item >> 4, cg = item & (cgs - 1);
            raw_zero(raw[i]);
            if (r < min(nr, ROWS) && 8 * cg < width) raw_load(raw[i], src + (size_t)r * stride + 8 * cg);
        }
    }
    // NT terms, each a panel of ROWS rows; w: weight of each row, or null
    template <int NT>
    __device__ __forceinline__ void store(unsigned char *dst, int cgs, const float *w) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int item = threadIdx.x + NTHR * i, r = cgs == 8 ? item >> 3 : item >> 4, cg = item & (cgs - 1);
            if (r >= ROWS) break;
            unsigned char *p = dst + panel_off(ROWS, r, cg);
            put<NT>(p, raw[i], w ? w[r] : 1.f, w != nullptr);
        }
    }
    template <int NT, typename R>
    __device__ __forceinline__ void put(unsigned char *p, const R &r, float w, bool weighted) {
        float x[8];
        raw_floats(r, x, (const T *)nullptr);
        if (weighted) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= w;
        }
        store_terms<NT>(p, (size_t)ROWS * COLS * 2, x);
    }
};

// Waits of a block that moves in step: every thread polls; a wait that runs
// out anywhere ends the block's work (uniformly) with the flag raised.
struct Waits {
    uint64_t *bar;
    volatile int *abort;
    long long limit;
    uint32_t phase;   // completed phases of the one barrier, modulo 2
    __device__ __forceinline__ bool wait() {
        const bool ok = mbar_wait(bar, phase, abort, limit);
        phase ^= 1;
        return !__syncthreads_or(!ok);
    }
};

// MMAs D[128][N] (+)= A B over `steps` steps of 16 of the contraction, for the
// term pairs (ta, tb) with ta + tb <= MAXS, the smallest products first: an
// accumulation is rounded at the size of the sum so far, so only the last
// pair's steps round at the result's own size. A step moves `a_block` /
// `b_block` or 32 bytes in a K-major panel, 16 rows in an MN-major one.
template <int TA, int TB, int MAXS>
__device__ __forceinline__ void issue(uint32_t d, uint32_t a, uint32_t a_panel, bool a_mn, uint32_t a_block, uint32_t b,
                                      uint32_t b_panel, bool b_mn, uint32_t b_block, uint32_t id, int steps, bool acc) {
#pragma unroll
    for (int sum = MAXS; sum >= 0; --sum)
#pragma unroll
        for (int ta = 0; ta < TA; ++ta) {
            const int tb = sum - ta;
            if (tb < 0 || tb >= TB) continue;
            for (int s = 0; s < steps; ++s) {
                const uint32_t pa = a + ta * a_panel + (a_mn ? 2048u * s : (s >> 2) * a_block + 32u * (s & 3));
                const uint32_t pb = b + tb * b_panel + (b_mn ? 2048u * s : (s >> 2) * b_block + 32u * (s & 3));
                mma_ss(d, a_mn ? desc_sw128_mn(pa, a_block) : desc_sw128(pa),
                       b_mn ? desc_sw128_mn(pb, b_block) : desc_sw128(pb), id, acc);
                acc = true;
            }
        }
}

__device__ __forceinline__ void tmem_alloc(uint32_t *slot, int cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(slot)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, int cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}

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

// ------------------------------------------------------------- increments

constexpr int INC_ROWS = 64;   // keys staged at a time
constexpr int INC_THREADS = 256;
constexpr uint32_t INC_PANEL = INC_ROWS * COLS * 2, INC_BLOCK = INC_ROWS * 128;

template <typename T>
constexpr size_t inc_smem() { return 1024 + (3 + Terms<T>::in) * (size_t)INC_PANEL; }

// dS[d][dv] of one (chunk, head), a tile of 128 x 128 of it a CTA:
// A = weighted keys (M = d), B = values (N = dv), both MN-major, contraction
// over the keys, 64 staged at a time while the previous 64 multiply.
template <typename T>
__global__ __launch_bounds__(INC_THREADS, Terms<T>::in == 1 ? 3 : 2) void k_lin_inc(LinArgs a,
                                                                                    const __grid_constant__ LinWorkTable t,
                                                                                    float *inc) {
    extern __shared__ unsigned char smraw[];
    __shared__ uint64_t bar;
    __shared__ uint32_t tslot;
    __shared__ int abort;
    __shared__ float pw[LIN_CHUNK];   // weight of each key
    unsigned char *sm = (unsigned char *)(((uintptr_t)smraw + 1023) & ~(uintptr_t)1023);
    unsigned char *sK = sm, *sV = sm + 3 * INC_PANEL;
    constexpr int NT = Terms<T>::in;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c = blockIdx.x, h = blockIdx.y, g = h / a.hpg;
    const int vt = (a.dv + COLS - 1) / COLS, d0 = (blockIdx.z / vt) * COLS, v0 = (blockIdx.z % vt) * COLS;
    const int wd = min(COLS, a.d - d0), wv = min(COLS, a.dv - v0);
    const int cgd = wd > 64 ? 16 : 8, cgv = wv > 64 ? 16 : 8;
    const Chunk ch = find_chunk(t, c);
    if (tid == 0) {
        mbar_init(&bar, 1);
        abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tmem_alloc(&tslot, 128);
    if (tid < LIN_CHUNK) pw[tid] = tid < ch.nr ? lin_pow(a.decay[h], ch.nr - 1 - tid) : 0.f;
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = tslot;
    Waits w{&bar, &abort, a.wait_cycles, 0};
    const T *k = (const T *)a.k + (size_t)ch.row0 * a.ks + (size_t)g * a.d + d0;
    const T *v = (const T *)a.v + (size_t)ch.row0 * a.vs + (size_t)g * a.dv + v0;
    Tile<T, INC_ROWS, INC_THREADS> tk, tv;
    tk.load(k, a.ks, ch.nr, wd, cgd);
    tv.load(v, a.vs, ch.nr, wv, cgv);
    bool ok = true;
    for (int s = 0; s * INC_ROWS < ch.nr; ++s) {
        if (s > 0) {
            ok = w.wait();   // the panels are free
            if (!ok) break;
        }
        tk.template store<3>(sK, cgd, pw + s * INC_ROWS);
        tv.template store<NT>(sV, cgv, nullptr);
        fence_async_smem();
        __syncthreads();
        if (tid == 0) {
            tc_after();
            const int left = ch.nr - s * INC_ROWS;
            issue<3, NT, 2>(tmem, su32(sK), INC_PANEL, true, INC_BLOCK, su32(sV), INC_PANEL, true, INC_BLOCK,
                            idesc_bf16(128, ceil16(wv), 1, 1), min(INC_ROWS, ceil16(left)) / 16, s > 0);
            mma_commit(&bar);
        }
        const int nx = (s + 1) * INC_ROWS;
        if (nx < ch.nr) {
            tk.load(k + (size_t)nx * a.ks, a.ks, ch.nr - nx, wd, cgd);
            tv.load(v + (size_t)nx * a.vs, a.vs, ch.nr - nx, wv, cgv);
        }
    }
    if (ok) ok = w.wait();
    tc_after();
    // lane = state row: warps 0-3 columns 0-63, warps 4-7 columns 64-127
    float *o = inc + ((size_t)c * a.nh + h) * a.d * a.dv;
    const int row = 32 * (warp & 3) + lane, cb = 64 * (warp >> 2);
    if (ok) {
        for (int q = 0; q < 2; ++q) {
            const int col = cb + 32 * q;
            if (col >= wv) break;
            uint32_t r[32];
            TMEM_LD32(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + col, r);
            tmem_ld_wait();
            if (row < wd) {
                float *p = o + (size_t)(d0 + row) * a.dv + v0 + col;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (col + 4 * i < wv)
                        *(float4 *)(p + 4 * i) = make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]),
                                                             __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3]));
            }
        }
    } else if (row < wd) {
        for (int col = cb; col < min(wv, cb + 64); ++col) o[(size_t)(d0 + row) * a.dv + v0 + col] = NAN;
    }
    if (!ok && tid == 0) {
        mbar_drain(&bar, w.phase ^ 1);   // the commit whose wait ran out: the only one in flight
        atomicOr(&lin_device_flags, (uint32_t)O1_FLAG_WAIT_EXPIRED);
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (warp == 0) tmem_free(tmem, 128);
}

// ------------------------------------------------------------------- scan

// Per state element, over a piece's chunks: inc <- the state entering the
// chunk, S <- l^n S + dS, the last S to its slot. Bound: the scratch's
// bytes (read and written once, L2-resident for a pass); 4 chunks' loads
// go out ahead of their use.
__global__ __launch_bounds__(256) void k_lin_scan(LinArgs a, const __grid_constant__ LinWorkTable t, float *inc) {
    const LinWork w = t.w[blockIdx.z];
    const int h = blockIdx.y;
    const size_t n = (size_t)a.d * a.dv;
    const size_t e = 4 * ((size_t)blockIdx.x * 256 + threadIdx.x);
    if (e >= n) return;
    float4 *sp = (float4 *)(a.state + ((size_t)w.slot * a.nh + h) * n + e);
    const size_t step = (size_t)a.nh * n / 4;
    float4 *p = (float4 *)(inc + ((size_t)w.chunk0 * a.nh + h) * n + e);
    const int nc = (w.rows + LIN_CHUNK - 1) / LIN_CHUNK;
    const float gd = a.decay[h], full = lin_pow(gd, LIN_CHUNK), last = lin_pow(gd, w.rows - (nc - 1) * LIN_CHUNK);
    float4 s = *sp;
    for (int c = 0; c < nc; c += 4) {
        float4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < nc) x[i] = p[(size_t)(c + i) * step];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (c + i >= nc) break;
            p[(size_t)(c + i) * step] = s;
            const float l = c + i == nc - 1 ? last : full;
            s.x = fmaf(s.x, l, x[i].x);
            s.y = fmaf(s.y, l, x[i].y);
            s.z = fmaf(s.z, l, x[i].z);
            s.w = fmaf(s.w, l, x[i].w);
        }
    }
    *sp = s;
}

// ---------------------------------------------------------------- outputs

constexpr uint32_t OUT_PANEL = LIN_CHUNK * COLS * 2, OUT_BLOCK = LIN_CHUNK * 128;
constexpr int OUT_ACC = 0, OUT_SC = 128;   // TMEM columns: Q S_in; scores, later P V

template <typename T>
constexpr int out_threads() { return Terms<T>::in == 1 ? 256 : 512; }
template <typename T>
constexpr size_t out_smem() {
    const int b = Terms<T>::in > Terms<T>::mid ? Terms<T>::in : Terms<T>::mid;
    return 1024 + (size_t)(Terms<T>::in + b) * OUT_PANEL;
}

// The outputs of one (chunk, head), a tile of 128 value columns a CTA. Two
// shared-memory regions: A holds Q, then V; B holds K, then S_in, then P. d
// above 128 runs Q, K and S_in in two rounds. Two CTAs an SM (bf16) hide each
// other's staging.
template <typename T>
__global__ __launch_bounds__(out_threads<T>(), Terms<T>::in == 1 ? 2 : 1) void k_lin_out(
    LinArgs a, const __grid_constant__ LinWorkTable t, const float *inc) {
    extern __shared__ unsigned char smraw[];
    __shared__ uint64_t bar;
    __shared__ uint32_t tslot;
    __shared__ int abort;
    __shared__ float pw[LIN_CHUNK + 1];   // powers of the decay
    constexpr int NT = Terms<T>::in, MT = Terms<T>::mid, NTHR = out_threads<T>(), NW = NTHR / 32;
    constexpr int WC = COLS / (NW / 4);   // columns a warp takes of its 32 TMEM lanes
    unsigned char *sm = (unsigned char *)(((uintptr_t)smraw + 1023) & ~(uintptr_t)1023);
    unsigned char *sA = sm, *sB = sm + NT * OUT_PANEL;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c = blockIdx.x, h = blockIdx.y, g = h / a.hpg, v0 = blockIdx.z * COLS;
    const int wv = min(COLS, a.dv - v0), cgv = wv > 64 ? 16 : 8;
    const Chunk ch = find_chunk(t, c);
    if (tid == 0) {
        mbar_init(&bar, 1);
        abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tmem_alloc(&tslot, 256);
    if (tid <= LIN_CHUNK) pw[tid] = lin_pow(a.decay[h], tid);
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = tslot;
    Waits w{&bar, &abort, a.wait_cycles, 0};
    const T *q = (const T *)a.q + (size_t)ch.row0 * a.qs + (size_t)h * a.d;
    const T *k = (const T *)a.k + (size_t)ch.row0 * a.ks + (size_t)g * a.d;
    const T *v = (const T *)a.v + (size_t)ch.row0 * a.vs + (size_t)g * a.dv + v0;
    const float *S = inc + ((size_t)c * a.nh + h) * a.d * a.dv + v0;
    const uint32_t A = su32(sA), B = su32(sB);
    bool ok = true;
    Tile<T, LIN_CHUNK, NTHR> tv;
    for (int d0 = 0; d0 < a.d && ok; d0 += COLS) {
        const int wd = min(COLS, a.d - d0), cgd = wd > 64 ? 16 : 8, ks = ceil16(wd) / 16;
        {
            Tile<T, LIN_CHUNK, NTHR> tq, tk;
            tq.load(q + d0, a.qs, ch.nr, wd, cgd);
            tk.load(k + d0, a.ks, ch.nr, wd, cgd);
            tq.template store<NT>(sA, cgd, nullptr);
            tk.template store<NT>(sB, cgd, nullptr);
        }
        fence_async_smem();
        __syncthreads();
        if (tid == 0) {
            tc_after();
            issue<NT, NT, NT - 1>(tmem + OUT_SC, A, OUT_PANEL, false, OUT_BLOCK, B, OUT_PANEL, false, OUT_BLOCK,
                                  idesc_bf16(128, 128, 0, 0), ks, d0 > 0);
            mma_commit(&bar);
        }
        Tile<float, LIN_CHUNK, NTHR> ts;   // S_in rows d0 ..: panel rows are d
        ts.load(S + (size_t)d0 * a.dv, a.dv, wd, wv, cgv);
        ok = w.wait();
        if (!ok) break;
        ts.template store<MT>(sB, cgv, nullptr);
        fence_async_smem();
        __syncthreads();
        if (tid == 0) {
            tc_after();
            issue<NT, MT, max_sum(NT, MT)>(tmem + OUT_ACC, A, OUT_PANEL, false, OUT_BLOCK, B, OUT_PANEL, true, OUT_BLOCK,
                                           idesc_bf16(128, ceil16(wv), 0, 1), ks, d0 > 0);
            mma_commit(&bar);
        }
        if (d0 + COLS >= a.d) tv.load(v, a.vs, ch.nr, wv, cgv);
        ok = w.wait();
    }
    const int row = 32 * (warp & 3) + lane, cw = WC * (warp >> 2);
    const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    if (ok) {
        // P_ij = l^{i-j} s_ij for j <= i, else 0 (also for keys past the end)
        tv.template store<NT>(sA, cgv, nullptr);
        tc_after();
        for (int cb = cw; cb < cw + WC; cb += 32) {
            uint32_t r[32];
            TMEM_LD32(lane_base + OUT_SC + cb, r);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int j = cb + 8 * i + e;
                    x[e] = j <= row ? __uint_as_float(r[8 * i + e]) * pw[row - j] : 0.f;
                }
                store_terms<MT>(sB + panel_off(LIN_CHUNK, row, (cb >> 3) + i), OUT_PANEL, x);
            }
        }
        tc_before();
        fence_async_smem();
        __syncthreads();
        if (tid == 0) {
            tc_after();
            issue<MT, NT, max_sum(MT, NT)>(tmem + OUT_SC, B, OUT_PANEL, false, OUT_BLOCK, A, OUT_PANEL, true, OUT_BLOCK,
                                           idesc_bf16(128, ceil16(wv), 0, 1), ceil16(ch.nr) / 16, false);
            mma_commit(&bar);
        }
        ok = w.wait();
    }
    tc_after();
    const float lr = pw[row + 1];
    for (int cb = cw; cb < cw + WC; cb += 32) {
        if (cb >= wv) break;
        uint32_t r0[32], r1[32];
        TMEM_LD32(lane_base + OUT_ACC + cb, r0);
        TMEM_LD32(lane_base + OUT_SC + cb, r1);
        tmem_ld_wait();
        if (row < ch.nr) {
            T *o = (T *)a.out + (size_t)(ch.row0 + row) * a.os + (size_t)h * a.dv + v0 + cb;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (cb + 4 * i >= wv) continue;
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    y[e] = ok ? a.scale * fmaf(lr, __uint_as_float(r0[4 * i + e]), __uint_as_float(r1[4 * i + e])) : NAN;
                o1_st4(o + 4 * i, make_float4(y[0], y[1], y[2], y[3]));
            }
        }
    }
    if (!ok && tid == 0) {
        mbar_drain(&bar, w.phase ^ 1);   // the commit whose wait ran out: the only one in flight
        atomicOr(&lin_device_flags, (uint32_t)O1_FLAG_WAIT_EXPIRED);
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (warp == 0) tmem_free(tmem, 256);
}

template <typename T>
void pass_t(const LinArgs &a, const LinWorkTable &t, int chunks, float *inc, cudaStream_t st) {
    static unsigned long long done = 0;
    unsigned long long bit = 0;
    if (o1_attrs_needed(&done, &bit)) {
        cudaFuncSetAttribute(k_lin_inc<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)inc_smem<T>());
        cudaFuncSetAttribute(k_lin_out<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)out_smem<T>());
        o1_attrs_done(&done, bit);
    }
    const int dt = (a.d + COLS - 1) / COLS, vt = (a.dv + COLS - 1) / COLS;
    k_lin_inc<T><<<dim3(chunks, a.nh, dt * vt), INC_THREADS, inc_smem<T>(), st>>>(a, t, inc);
    k_lin_scan<<<dim3((a.d * a.dv / 4 + 255) / 256, a.nh, t.n), 256, 0, st>>>(a, t, inc);
    k_lin_out<T><<<dim3(chunks, a.nh, vt), out_threads<T>(), out_smem<T>(), st>>>(a, t, inc);
}

}  // namespace

void lin_launch_pass(const LinArgs &a, int dtype, const LinWorkTable &t, int chunks, float *inc, cudaStream_t st) {
    if (dtype == O1_F32) pass_t<float>(a, t, chunks, inc, st);
    else if (dtype == O1_BF16) pass_t<__nv_bfloat16>(a, t, chunks, inc, st);
    else pass_t<__half>(a, t, chunks, inc, st);
}

int lin_flags(uint32_t *flags, int clear, cudaStream_t st) {
    if (cudaMemcpyFromSymbolAsync(flags, lin_device_flags, sizeof(uint32_t), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess)
        return O1_ERR_CUDA;
    static const uint32_t zero = 0;
    if (clear &&
        cudaMemcpyToSymbolAsync(lin_device_flags, &zero, sizeof(uint32_t), 0, cudaMemcpyHostToDevice, st) != cudaSuccess)
        return O1_ERR_CUDA;
    return cudaStreamSynchronize(st) == cudaSuccess ? O1_OK : O1_ERR_CUDA;
}
