/*
 * o1.h — C ABI of the sealed O(1) layer attention library (libo1.so, CUDA,
 * sm_103a).
 *
 * A sealed layer's attention: every query row attends to
 *   (1) a few sink keys,
 *   (2) a ring-buffer window of recent keys (the causal rows of the call
 *       included), and
 *   (3) a constant-size far field that summarises every key evicted from the
 *       ring: per (group, head, landmark query b) a running max M_b, mass Z_b
 *       and value sum T_b of exp(scale * qt_b . k_evicted - M_b), read back
 *       through the landmark keys kt and the coefficients mu.
 * The method is the one of "cortiq-engine 0.8.51 src/gpu_wgpu/o1_batch.rs"
 * (module doc; kernels o1b_far_e, o1b_attend, o1b_far_commit,
 * o1b_ring_commit, o1b_meta); the one-row variant is the one of
 * "cortiq-engine 0.8.82 src/gpu_metal/o1c.rs" (encode_tok) and of
 * "cortiq-engine 0.8.77 src/gpu_wgpu/dory.rs" (dory_os ... dory_ogate), whose
 * rotation (dory_prep) and output gate (dory_gate1) it also applies.
 *
 * Conventions, for every entry point:
 *  - Ownership: the caller allocates and frees every buffer. The library
 *    allocates no device or host memory for a call; a state buffer carries
 *    its own header. What it keeps itself: the second CUDA stream and two
 *    events of the chunk path (one set per host thread and device, made by
 *    the first chunk call and released when that thread exits; see
 *    O1_NUM_STAGES) and the static scratch array of o1_token_attend_noalloc.
 *  - Pointers: "device" pointers are CUDA global memory of the current
 *    device, "host" pointers are ordinary process memory. Device buffers must
 *    be 16-byte aligned (a torch or cudaMalloc allocation always is); the
 *    state and scratch buffers 256-byte aligned.
 *  - Layouts are row-major fp32 unless stated; shapes are written [a][b][c]
 *    with the last index fastest.
 *  - Streams: `stream` is a cudaStream_t passed as void* (NULL = the legacy
 *    default stream). Calls are asynchronous on it except where stated. A
 *    state must be used from one stream at a time.
 *  - Errors: every call validates its arguments before launching anything
 *    and returns O1_OK or a negative status; nothing falls back to another
 *    implementation. O1_ERR_CUDA reports a failed launch or copy
 *    (cudaGetLastError after the launches, which also clears a launch
 *    error so that it is reported once; or the copy's status).
 *  - State and geometry: the state's header (magic, geometry) lives on the
 *    device. The calls that synchronise anyway (o1_state_read, _write,
 *    _flags) check it against `geom` and return O1_ERR_STATE on a mismatch.
 *    The attend, commit and rewind calls do not read it back: that would
 *    cost a device round trip per call and make them uncapturable. They
 *    must be given the geometry the state was initialised with.
 */
#ifndef O1_H
#define O1_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define O1_API __attribute__((visibility("default")))
#else
#define O1_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
enum {
    O1_OK = 0,
    O1_ERR_ARG = -1,          /* null or misaligned pointer, bad size        */
    O1_ERR_UNSUPPORTED = -2,  /* geometry outside the library's limits       */
    O1_ERR_CUDA = -3,         /* a CUDA launch or copy failed                */
    O1_ERR_STATE = -4         /* state header does not match the geometry    */
};

/* Geometry of one sealed layer ("cortiq-engine 0.8.51 src/gpu_wgpu/o1_batch.rs",
 * struct Geom). Limits: groups >= 1, heads_per_group in [1, 16],
 * d in [8, 256] with d % 8 == 0, dv in [4, 256] with dv % 4 == 0,
 * sinks in [0, 64], window in [1, 1 << 20], landmarks in [1, 64]. */
typedef struct o1_geom {
    int32_t groups;           /* G: KV groups                                  */
    int32_t heads_per_group;  /* hpg: query heads per KV group (nh = G * hpg)  */
    int32_t d;                /* key / query width                             */
    int32_t dv;               /* value width                                   */
    int32_t sinks;            /* ns: sink keys per group                       */
    int32_t window;           /* w: ring stride = the widest group window      */
    int32_t landmarks;        /* m: landmark queries per head                  */
    int32_t rect_far_mass;    /* 1: u_b = max(u_b, 0) (the pages' rect_fm)     */
    float scale;              /* score scale, normally 1/sqrt(d)               */
    float rope_base;          /* rotary base (e.g. 1e6); 0 = no rotation       */
} o1_geom;

/* Host-side view of a state, for o1_state_read / o1_state_write. Every
 * pointer is host memory and may be NULL (that part is skipped). */
typedef struct o1_state_host {
    uint32_t *meta;    /* [G][4]: len, head, farl, group window                */
    int64_t *pos;      /* [1]: absolute position of the next row               */
    float *ring_k;     /* [G][window][d]: rotated keys by ring slot            */
    float *ring_v;     /* [G][window][dv]                                      */
    float *far_max;    /* M [G*hpg][m]; -inf while the far field is empty      */
    float *far_mass;   /* Z [G*hpg][m], rounded to f32 (the state keeps a low
                          part beside it; a write sets that part to zero)    */
    float *far_val;    /* T [G*hpg][m][dv]                                     */
} o1_state_host;

/* Bytes of device memory a state of this geometry needs (0 if the geometry is
 * outside the limits). Host-only; no CUDA call.
 * The state holds the buffers of one sealed layer that "cortiq-engine 0.8.51
 * src/gpu_wgpu/o1_batch.rs" lists in struct State (meta, ring_k, ring_v,
 * sink_k, sink_v, k_tilde, qt, mu, the far max and mass mz, the far value
 * sum that), sized from struct Geom, plus a header of this library's
 * (magic, geometry, position, rotary frequencies, flags). */
O1_API size_t o1_state_bytes(const o1_geom *geom);

/* Bytes of device scratch that lets one o1_chunk_attend launch process up to
 * `max_rows` rows in one pass (longer calls run in passes of that many rows).
 * 0 if the geometry is unsupported or max_rows < 1. Host-only.
 * The pages size a per-call scratch from the geometry ("cortiq-engine 0.8.51
 * src/gpu_wgpu/o1_batch.rs", Geom::scratch_len: the far-field exponents and
 * prefixes of one 64-row sub-chunk plus a max and a rescale per head and
 * landmark). This library runs every 64-row block of a pass at once, so its
 * scratch holds those planes for all of them, plus the rotated rows, the
 * window and side partials and, on the tensor-core path, fp16 panels. */
O1_API size_t o1_scratch_bytes(const o1_geom *geom, int32_t max_rows);

/* Start a sealed layer from an empty ring and far field ("cortiq-engine
 * 0.8.51 src/gpu_wgpu/o1_batch.rs", struct State and the meta layout of
 * o1b_meta; an empty far field has M = -inf, Z = 0 as o1b_far_e's comment
 * states).
 *   state          device, o1_state_bytes(geom) bytes, 256-byte aligned; overwritten
 *   group_windows  host [G] or NULL: each group's window (meta slot 3),
 *                  0 = geom->window; every value <= geom->window
 *   sink_k, sink_v device [G][ns][d], [G][ns][dv] (may be NULL if ns == 0)
 *   k_tilde        device [G][m][d]      landmark keys, one set per group
 *   q_tilde        device [G][hpg][m][d] landmark queries, per head
 *   mu             device [G*hpg][m][m]  mu[a][b], a = landmark key, b = query
 *   pos0           absolute position of the first row (rotation angle)
 * Sinks and landmarks are used as given (already rotated). Asynchronous. */
O1_API int o1_state_init(void *state, const o1_geom *geom, const int32_t *group_windows,
                  const float *sink_k, const float *sink_v, const float *k_tilde,
                  const float *q_tilde, const float *mu, int64_t pos0, void *stream);

/* Attention of `rows` consecutive rows, and the state advanced past them
 * ("cortiq-engine 0.8.51 src/gpu_wgpu/o1_batch.rs": encode and the kernels
 * o1b_far_e, o1b_attend, o1b_far_commit, o1b_ring_commit, o1b_meta; gate as
 * dory_gate1 of "cortiq-engine 0.8.77 src/gpu_wgpu/dory.rs").
 *   q     device [rows][G*hpg][d]  queries, NOT rotated (rotated here at pos)
 *   k     device [rows][G][d]      keys, not rotated
 *   v     device [rows][G][dv]
 *   gate  device [rows][G*hpg][dv] gate logits, or NULL for no gate
 *   out   device [rows][G*hpg][dv] o / (1 + exp(-gate)); must not alias q/k/v/gate
 *   scratch, scratch_bytes  device scratch, at least o1_scratch_bytes(geom, 1)
 * The output equals the rows processed one at a time (rope, far insert, ring
 * push, attend, gate), up to rounding. Asynchronous.
 * Window path: when d % 64 == 0, d <= 256, dv % 32 == 0, dv <= 256 and
 * window >= 512, the window part of a pass with two or more rows runs on the
 * tensor cores, each fp32 operand split into two fp16 halves (hi + lo, three
 * products). It needs every rotated query, rotated key and value to lie
 * inside the fp16 range (|x| < 65504); one outside it raises
 * O1_FLAG_FP16_RANGE in the state's flags and that pass's output is not
 * valid. Other geometries, and one-row calls (which take the one-row path),
 * run in fp32 throughout. */
O1_API int o1_chunk_attend(void *state, const o1_geom *geom, void *scratch, size_t scratch_bytes,
                    const float *q, const float *k, const float *v, const float *gate,
                    int32_t rows, float *out, void *stream);

/* Speculative verification ("cortiq-engine 0.8.82 src/gpu_metal/o1c.rs":
 * encode with commit = false, then spec_commit over the accepted rows).
 *
 * o1_chunk_attend_spec: the attention of `rows` draft rows, exactly as
 * o1_chunk_attend would compute it (same arguments, layouts, checks and
 * output), but the state is left as it was: no far insert, ring push, meta
 * or position change. The draft must fit in one pass of the scratch
 * (rows <= the max_rows the scratch was sized for), else O1_ERR_ARG. A
 * one-row draft runs as a one-row pass of the chunk path, not the decode
 * path. Asynchronous.
 *
 * o1_spec_commit: moves the state over the first `rows` accepted rows, given
 * their keys and values again (k [rows][G][d] unrotated, v [rows][G][dv],
 * device, 16-byte aligned; the same values the verify call was given): the
 * rotation of the keys at the state's position, the far insert of every key
 * they evict, the ring push, meta and position. The state afterwards equals
 * the one o1_chunk_attend over those rows leaves, up to rounding; nothing is
 * attended and no output is written. rows = 0 does nothing. Rows above the
 * scratch's capacity run as several passes. Same scratch rules as
 * o1_chunk_attend. Asynchronous. */
O1_API int o1_chunk_attend_spec(void *state, const o1_geom *geom, void *scratch, size_t scratch_bytes,
                                const float *q, const float *k, const float *v, const float *gate,
                                int32_t rows, float *out, void *stream);
O1_API int o1_spec_commit(void *state, const o1_geom *geom, void *scratch, size_t scratch_bytes,
                          const float *k, const float *v, int32_t rows, void *stream);

/* Exact sliding-window attention, the comparator of the sealed layer (the
 * pages time the same model chunk with exact attention against the sealed
 * layer's per-row loop; "cortiq-engine 0.8.77 src/gpu_wgpu/dory.rs",
 * dory_score / dory_soft / dory_sum / dory_gate). Each row attends to the
 * sinks and to the last min(group window, len + r + 1) keys of [ring, oldest
 * first] ++ [this call's rows] ending at its own; keys that leave the window
 * are dropped, and there is no far field. Same arguments, layouts, checks,
 * rotation and gate as o1_chunk_attend, and the same window kernels. The
 * state is only read (no push, no position change), so the rows must fit in
 * one pass of the scratch, else O1_ERR_ARG. From a fresh state with a window
 * of at least `rows`, the output is exact causal softmax attention over the
 * sinks and every key. Asynchronous. */
O1_API int o1_window_attend(void *state, const o1_geom *geom, void *scratch, size_t scratch_bytes,
                            const float *q, const float *k, const float *v, const float *gate,
                            int32_t rows, float *out, void *stream);

/* One row (a decode step): the same as o1_chunk_attend with rows = 1, by a
 * path built for it ("cortiq-engine 0.8.82 src/gpu_metal/o1c.rs" encode_tok:
 * near partials split across blocks, the far part, a merge, the commit).
 *   q [G*hpg][d], k [G][d], v [G][dv], gate [G*hpg][dv] or NULL, out [G*hpg][dv]
 *   scratch  device, at least o1_scratch_bytes(geom, 1) bytes
 * Where that path's shared memory would exceed a block's (windows of a few
 * hundred thousand keys and more), the row runs as a one-row chunk pass,
 * with the same result. Asynchronous. */
O1_API int o1_token_attend(void *state, const o1_geom *geom, void *scratch, size_t scratch_bytes,
                    const float *q, const float *k, const float *v, const float *gate,
                    float *out, void *stream);

/* Stages of one chunk pass, in launch order: rope, far_block, far_tscan,
 * side_readout, gather_tc, near, merge, commit. The far-field stages
 * (far_block .. side_readout) run on a second, high-priority stream of the
 * library's, concurrently with gather_tc and near; it is forked from and
 * joined back into the caller's stream by events, so a stream capture of a
 * call captures both branches. The stream and its two events are created by
 * the first call on each host thread and device (make that call before a
 * stream capture) and live until that thread exits. A stage that does not apply to the geometry
 * (the fp16 panel gather outside the tensor-core window path) launches
 * nothing and times as empty. A pass of at most 16 rows runs its far field
 * and sinks as one short kernel (timed as side_readout; far_block and
 * far_tscan stay empty) and, from 2 rows, its window as key-slice kernels
 * (timed as near). */
#define O1_NUM_STAGES 8

/* o1_chunk_attend that also records caller-created CUDA events (cudaEvent_t
 * handles, passed as void*): events[2i] just before and events[2i + 1] just
 * after stage i of a pass, on the stream that stage runs on, so that
 * cudaEventElapsedTime(events[2i], events[2i + 1]) is stage i's time (with
 * the other branch running concurrently). With several passes (rows above
 * the scratch's capacity) the events end up holding the last pass. n_events
 * must be at least 2 * O1_NUM_STAGES. Same arguments, checks and result as
 * o1_chunk_attend otherwise. */
O1_API int o1_chunk_attend_timed(void *state, const o1_geom *geom, void *scratch, size_t scratch_bytes,
                                 const float *q, const float *k, const float *v, const float *gate,
                                 int32_t rows, float *out, void *const *events, int32_t n_events,
                                 void *stream);

/* Name of stage i of a chunk pass (NULL outside [0, O1_NUM_STAGES)). The
 * pages time a forward stage by stage by keeping only some dispatch kinds
 * ("cortiq-engine 0.8.77 src/gpu_wgpu/dory.rs", the keep-one stage table);
 * here each stage records events around itself instead, and every stage
 * still runs. */
O1_API const char *o1_stage_name(int32_t stage);

/* Size of the library's own device scratch used by o1_token_attend_noalloc:
 * 4 MiB, held by every GPU that loads the library until the process exits. */
#define O1_NOALLOC_SCRATCH_BYTES (4u << 20)

/* o1_token_attend for callers that cannot allocate device memory: no
 * scratch argument, no cudaMalloc, cudaFree or allocating library call.
 * For a plugin whose interface hands over no workspace, or a decode loop
 * that must not call cudaMalloc (it can synchronise the device and stall
 * other streams) nor keep a buffer of its own. The paper has no
 * counterpart; this is a convenience of this library.
 *   q, k, v, gate, out, state, stream: as o1_token_attend.
 * The scratch is one static device array of O1_NOALLOC_SCRATCH_BYTES in
 * this library, shared by every call on a device: calls that overlap on
 * the GPU (other streams, other threads) race on it, so serialise them.
 * Nothing in it needs to start at zero: a call writes every scratch value
 * before reading it. The first call on each device looks the array's
 * device address up (cudaGetSymbolAddress, that device current) and keeps
 * it for the life of the process; make that first call before any stream
 * capture. The kept address does not survive cudaDeviceReset of that device
 * (a new context holds the array elsewhere): do not reset a device and go on
 * calling this entry point on it in the same process. Returns O1_ERR_UNSUPPORTED when the
 * geometry's one-row scratch exceeds O1_NOALLOC_SCRATCH_BYTES, else as
 * o1_token_attend. */
O1_API int o1_token_attend_noalloc(void *state, const o1_geom *geom, const float *q, const float *k,
                                   const float *v, const float *gate, float *out, void *stream);

/* Copy the state's mutable parts to host memory (NULL fields skipped).
 * Synchronises `stream`. Returns O1_ERR_STATE if the state's header does not
 * hold this geometry.
 * What is read is the state a chunk leaves behind for the next chunk or the
 * one-row path to carry on from ("cortiq-engine 0.8.51
 * src/gpu_wgpu/o1_batch.rs", module doc on o1b_far_commit, o1b_ring_commit
 * and o1b_meta; the buffers of struct State): meta, ring keys and values by
 * slot, and the far field M, Z, T. */
O1_API int o1_state_read(const void *state, const o1_geom *geom, o1_state_host *dst, void *stream);

/* Overwrite the state's mutable parts from host memory (NULL fields kept):
 * snapshots and test set-up. Synchronises `stream`. The caller keeps the
 * state consistent (len <= group window, head < group window, M = -inf
 * exactly where farl == 0, ...).
 * The same parts as o1_state_read: the state a chunk hands on to the next
 * chunk or to the one-row path ("cortiq-engine 0.8.51
 * src/gpu_wgpu/o1_batch.rs", module doc and struct State). The pages upload
 * a sealed layer's state from the host the same way ("cortiq-engine 0.8.77
 * src/gpu_wgpu/dory.rs", seal: the far states built on the CPU are
 * uploaded). */
O1_API int o1_state_write(void *state, const o1_geom *geom, const o1_state_host *src, void *stream);

/* Sticky conditions a kernel records in the state header (bits of the value
 * o1_state_flags returns). */
#define O1_FLAG_WAIT_EXPIRED 1u  /* a bounded in-kernel wait ran out (about 2 s);
                                    that pass's output is incomplete      */
#define O1_FLAG_FP16_RANGE 2u    /* an operand of the tensor-core window path
                                    was outside the fp16 range             */
#define O1_FLAG_BACK_REFUSED 4u  /* an o1_state_back was larger than some
                                    group could rewind; nothing was changed */

/* Rewind the last `rows` ring pushes of every KV group, for looped-layer KV
 * modes that push the same positions again ("cortiq-engine 0.8.77
 * src/gpu_wgpu/dory.rs", dory_o1_back, applied once per row): a full ring
 * (len == group window) steps its head back by one and forgets one eviction
 * (farl - 1) per row; a ring not yet full drops its newest entry (len - 1).
 * The position moves back by `rows`. Ring contents and the far field (M, Z,
 * T) are not undone, as on the page: keys already folded into the far field
 * stay there. A rewind some group cannot take in full (len < rows while not
 * full, farl < rows while full) or one longer than the position is refused on
 * the device, with nothing changed, and raises O1_FLAG_BACK_REFUSED (the
 * state's meta lives on the device, so this call cannot see it). rows = 0
 * does nothing. One single-thread launch; asynchronous. */
O1_API int o1_state_back(void *state, const o1_geom *geom, int32_t rows, void *stream);

/* Limit, in SM clock cycles, of the kernels' waits (on their own copies and
 * tensor-core work) for calls made from now on, in this process; a call
 * captured in a CUDA graph keeps the limit it was captured with.
 * cycles < 1, or above the default of 4e9 (about 2 s at the maximum SM
 * clock), restores the default. A wait that runs out raises
 * O1_FLAG_WAIT_EXPIRED and that call's output is not valid; the kernel still
 * waits, with the default limit, for the work it had already issued before
 * it exits. A tiny limit makes the first waits run out on purpose, which is
 * how that path is tested; in use the default is meant to stay. Host-only,
 * no CUDA call; always O1_OK. (The pages' kernels wait on no barrier of
 * this kind, so there is no counterpart to cite.) */
O1_API int o1_set_wait_limit(int64_t cycles);

/* Read the state's flags into *flags (host) and, if `clear` is non-zero,
 * reset them to 0. Synchronises `stream`.
 * The pages report a failed dispatch or readback through the encoder's
 * boolean result ("cortiq-engine 0.8.82 src/gpu_metal/o1c.rs", encode and
 * spec_commit return false; the command buffer's error status is checked).
 * A kernel here cannot return a value, so it records such conditions as
 * these sticky bits. */
O1_API int o1_state_flags(void *state, const o1_geom *geom, uint32_t *flags, int32_t clear, void *stream);

/* ------------------------------------------------------------------ heads
 * What stands around a sealed layer in a hybrid model: the normalisation of
 * query and key heads before attention, and the other attention with a state
 * of constant size, linear attention with a decay per head. These entry
 * points take rows of several element types and with a stride:
 *  - a row tensor [rows][heads][width] has its heads and widths contiguous
 *    and `*_stride` elements from one row to the next (a slice of a fused
 *    projection's rows, say), heads * width <= stride, the base address and
 *    the stride in bytes multiples of 16;
 *  - weights, frequencies and decays are fp32;
 *  - outputs may not overlap inputs except where stated (row tensors of the
 *    same row stride whose columns are apart, as slices of one buffer, do not
 *    overlap).
 * Rows that an entry point is not told to compute are left as they were. */

/* Element types of row tensors. */
enum { O1_F32 = 0, O1_BF16 = 1, O1_F16 = 2 };

/* Norms of o1_head_prep. */
enum {
    O1_NORM_NONE = 0,
    O1_NORM_RMS = 1,   /* y = x / sqrt(mean(x^2) + eps) */
    O1_NORM_UNIT = 2   /* y = x / sqrt(sum(x^2) + eps)  */
};

/* Limits: q_heads and k_heads in [0, 4096], at least one head; d in [8, 256]
 * with d % 8 == 0; rot in [0, d] with rot % 8 == 0; eps finite, >= 0;
 * out_dtype O1_F32 or equal to in_dtype. */
typedef struct o1_prep_geom {
    int32_t q_heads, k_heads;  /* heads of the two row tensors; 0 = absent     */
    int32_t d;                 /* head width                                   */
    int32_t rot;               /* leading values of a head that rotate         */
    int32_t norm;              /* O1_NORM_*                                    */
    int32_t in_dtype, out_dtype;
    float eps;
} o1_prep_geom;

/* Norm of every query and key head and their rotation in one pass
 * ("cortiq-engine 0.8.77 src/gpu_wgpu/dory.rs", dory_prep: rotate, unit-
 * normalise each head, scale; here the norm comes first, as query / key norms
 * of models in use do, and a per-value weight carries the scale). Per row r
 * and head, x its d values:
 *   y = norm(x) * weight            (weight NULL: 1; a zero head under
 *                                    eps = 0 stays zero)
 *   z_j          = y_j cos a - y_{j + rot/2} sin a,   a = p inv_freq[j],
 *   z_{j + rot/2} = y_{j + rot/2} cos a + y_j sin a,  j < rot/2,
 * and z = y past rot. p = pos[r], or pos0 + r when pos is NULL.
 *   q, k           device row tensors [rows][q_heads][d], [rows][k_heads][d]
 *   q_weight, k_weight  device [d] or NULL, 16-byte aligned
 *   inv_freq       device [rot/2], 0 <= inv_freq < 2^24 (NULL if rot == 0)
 *   pos            device int64 [rows] or NULL
 *   q_out, k_out   device row tensors; either may be its own input exactly
 *                  (same address, stride and type)
 * Sums and the rotation are fp32; the angle is reduced exactly in fixed point
 * (a turn is 2^64), so far positions keep fp32 accuracy. The sum of squares
 * of a head must be finite in fp32; it may be as small as it likes, and a NaN
 * in a head makes the head NaN under a norm. The result feeds o1_chunk_attend
 * and its kin with rope_base = 0, or the linear layer. rows = 0 does nothing.
 * Asynchronous; one launch. */
O1_API int o1_head_prep(const o1_prep_geom *geom, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                        const float *q_weight, const float *k_weight, const float *inv_freq, const int64_t *pos,
                        int64_t pos0, int32_t rows, void *q_out, int64_t q_out_stride, void *k_out,
                        int64_t k_out_stride, void *stream);

/* Geometry of a linear layer: limits groups in [1, 4096], heads_per_group in
 * [1, 16], at most 65535 heads, d and dv in [8, 256] with both % 8 == 0, scale finite. Heads of a
 * group share its keys and values; each head has a decay and a state of its
 * own. */
typedef struct o1_lin_geom {
    int32_t groups;           /* G: KV groups                                  */
    int32_t heads_per_group;  /* query heads per group (nh = G * hpg)          */
    int32_t d, dv;            /* key / query and value width                   */
    int32_t dtype;            /* O1_F32, O1_BF16, O1_F16: q, k, v and out      */
    float scale;              /* output scale, normally 1/sqrt(d)              */
} o1_lin_geom;

/* One sequence of a packed batch (host memory): rows row0 .. row0 + rows - 1
 * of the row tensors, on state slot `slot`. */
typedef struct o1_lin_seq {
    int32_t row0, rows, slot;
} o1_lin_seq;

/* Bytes of `slots` states, fp32 [slots][nh][d][dv], 16-byte aligned, which
 * the caller sets to zero (an empty sequence) or to any finite state before
 * first use, copies and keeps as it likes: there is no header. 0 if the
 * geometry is unsupported, slots < 1, or the size does not fit 64 bits.
 * Host-only. */
O1_API size_t o1_lin_state_bytes(const o1_lin_geom *geom, int32_t slots);

/* Bytes of device scratch that o1_lin_chunk_attend has a use for in a call of
 * `rows` rows of at most `seqs` sequences. A call runs in one pass over what
 * the scratch holds, or in several: large calls in passes of about 64 MB of
 * states (256 MB with the rows of fp16 and fp32) and 128 sequences, whatever
 * the scratch, and the size returned is no larger than such a pass. Any size
 * from o1_lin_scratch_bytes(geom, 1, 1) on works, in passes as small as it is.
 * Host-only; 0 if unsupported or a count is below 1. */
O1_API size_t o1_lin_scratch_bytes(const o1_lin_geom *geom, int32_t rows, int32_t seqs);

/* Linear attention with a decay per head over packed sequences: the state of
 * each advanced past its rows. Per sequence, head h and row t,
 *   S = e^{log_decay[h]} S + k_t v_t^T;   out_t = scale q_t S,
 * up to rounding (the rows of a long sequence run in chunks: products inside
 * a chunk, and one state a chunk). It is the chunk / one-row pair of a sealed
 * layer ("cortiq-engine 0.8.51 src/gpu_wgpu/o1_batch.rs", module doc: a state
 * of constant size, a chunk at once, the next chunk continuing from it) for
 * the attention whose state is a plain sum; the pages have no such layer.
 *   state      device fp32 [n_slots][nh][d][dv]
 *   scratch    device, 256-byte aligned, see o1_lin_scratch_bytes
 *   q, k, v    device row tensors [total_rows][nh][d], [..][G][d], [..][G][dv]
 *   log_decay  device [nh], each in [-inf, 0] (0: no decay)
 *   seqs       host [n_seq], n_seq <= 4096, read during the call; rows of a
 *              sequence may be 0; row ranges may not overlap, row0 + rows <=
 *              total_rows, and slots are distinct and in [0, n_slots) (else
 *              O1_ERR_ARG)
 *   out        device row tensor [total_rows][nh][dv]; rows of no sequence
 *              are left as they were
 * q, k, v and the state are finite, in fp32 at most 3.38e38 (the largest bf16
 * value), and so are the sums q_i . k_j of a row and the rows up to 255 before
 * it in its sequence, which longer sequences form. A non-finite one spoils
 * rows and the state of its own sequence only: from its row on, and up to 127
 * rows before it. Rows of no sequence may hold anything. States and sums are fp32. Longer sequences run on the tensor cores:
 * operands are split into bf16 terms that hold fp32 and fp16 values and the
 * decayed keys to fp32 accuracy; for 16-bit outputs the entering state and
 * the scores are taken to 2^-16. Calls that may overlap on the GPU (other
 * streams, captured graphs) need a scratch each. Asynchronous. */
O1_API int o1_lin_chunk_attend(float *state, int32_t n_slots, const o1_lin_geom *geom, void *scratch,
                               size_t scratch_bytes, const void *q, int64_t q_stride, const void *k,
                               int64_t k_stride, const void *v, int64_t v_stride, const float *log_decay,
                               const o1_lin_seq *seqs, int32_t n_seq, void *out, int64_t out_stride,
                               int32_t total_rows, void *stream);

/* One row of each of `rows` sequences (a decode step of a batch): row r
 * advances slot slots[r] (NULL: slot r) by the same recurrence. slots is a
 * device array, so that a captured step can be replayed on other slots. A row
 * whose slot is outside [0, n_slots) is padding: its output is left as it
 * was. Of rows that name the same slot the first counts and the others are
 * padding (with slots, every row looks at those of the rows before it: a time
 * that grows with the square of the rows and shows from some thousands on).
 * At most 65536 rows. No scratch; one launch; asynchronous. */
O1_API int o1_lin_token_attend(float *state, int32_t n_slots, const o1_lin_geom *geom, const void *q,
                               int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                               const float *log_decay, const int32_t *slots, void *out, int64_t out_stride,
                               int32_t rows, void *stream);

/* Read the sticky flags that the chunk kernels of linear layers raised on the
 * current device into *flags (host) and, if `clear` is non-zero, reset them:
 * O1_FLAG_WAIT_EXPIRED (a bounded wait ran out, see o1_set_wait_limit; the
 * outputs and states that the block was to write are NaN). The states have no
 * header to hold them. Synchronises `stream`. */
O1_API int o1_lin_flags(uint32_t *flags, int32_t clear, void *stream);

/* ------------------------------------------------------------ paged cache
 * The layers of a hybrid model that are not sealed attend to every key kept
 * ("cortiq-engine 0.8.77 src/gpu_wgpu/dory.rs", dory_score, dory_soft and
 * dory_sum: exact attention over the cached rows of a layer). Their cache
 * grows with the sequences, so it is held in pages that a table assigns, in 16
 * bits or in 8: written as rows come (o1_pg_write, o1_pg_token_write), attended
 * by chunks of new rows or by one row of each sequence (o1_pg_chunk_attend,
 * o1_pg_token_attend), and read back as rows (o1_pg_read), say for o1_spec_commit
 * to move a sealed layer over them. Row tensors are those of the section
 * above. The caller owns pages and table; the library keeps nothing. */

/* Element type of a cache of 8 bits: e4m3 values under a power of two a head's
 * row. A row x of d values is held as x / 2^e, rounded to nearest (ties to
 * even), with 2^e the smallest power of two for which max |x| <= 448 * 2^e
 * (e >= -126), and the byte e + 127. The division is exact, so what is held
 * has one rounding (2^-4 of a value, or 2^-10 * 2^e if that is more). Infinities and NaN are held as NaN and do not count in the max.
 * Only a cache_dtype. */
enum { O1_E4M3 = 3 };

/* Geometry of a paged cache and the attention over it. Limits: groups in
 * [1, 4096], heads_per_group in [1, 16], at most 65535 heads, d and dv in
 * [8, 256], both % 8 == 0 (O1_E4M3: % 16 == 0), page in {16, 32, 64, 128, 256},
 * window >= 0, scale finite and above 0; cache_dtype O1_E4M3, or O1_F16 for dtype O1_F16 and
 * O1_BF16 for the others. */
typedef struct o1_pg_geom {
    int32_t groups;           /* G: KV groups                                  */
    int32_t heads_per_group;  /* query heads per group (nh = G * hpg)          */
    int32_t d, dv;            /* key / query and value width                   */
    int32_t page;             /* positions of a page                           */
    int32_t window;           /* positions a row attends, its own included; 0: all */
    int32_t dtype;            /* O1_F32, O1_BF16, O1_F16: q, k, v and out      */
    int32_t cache_dtype;      /* O1_BF16, O1_F16, O1_E4M3                      */
    float scale;              /* score scale, normally 1/sqrt(d)               */
} o1_pg_geom;

/* A cache (device pointers, 16-byte aligned; this struct is host memory).
 * Position p of the sequence in slot s is row p % page of page
 * table[s][p / page]. Limits: n_pages, n_slots, width >= 1, n_pages * G * page
 * and width * page < 2^31. A table entry outside [0, n_pages) is an absent
 * page: nothing is written to it or read from it, and its positions are left
 * out of the attention. Sequences may share pages that no call writes. */
typedef struct o1_pg_cache {
    void *k, *v;              /* [n_pages][G][page][d] and [..][dv], cache_dtype */
    uint8_t *k_exp, *v_exp;   /* [n_pages][G][page], e + 127 (1 to 254); NULL unless O1_E4M3 */
    const int32_t *table;     /* [n_slots][width]                              */
    int32_t n_pages, n_slots, width;
} o1_pg_cache;

/* One sequence of a packed batch (host memory): rows row0 .. row0 + rows - 1 of
 * the row tensors are positions pos0 .. pos0 + rows - 1 of slot `slot`. */
typedef struct o1_pg_seq {
    int32_t row0, rows, slot, pos0;
} o1_pg_seq;

/* Write rows of keys and values into the cache, rounded to nearest or quantised
 * on the way. Sequences: host [n_seq], n_seq <= 4096, read during the call; row
 * ranges in [0, total_rows) and apart, positions in [0, width * page), slots in
 * [0, n_slots), no position of a slot twice (else O1_ERR_ARG). Rows of no
 * sequence are not read. Two positions that the table puts in one place (a page
 * named twice) leave a mixture there.
 *   k, v  device row tensors [total_rows][G][d], [total_rows][G][dv]
 * Asynchronous; a launch every 128 sequences. */
O1_API int o1_pg_write(const o1_pg_geom *geom, const o1_pg_cache *cache, const void *k, int64_t k_stride,
                       const void *v, int64_t v_stride, const o1_pg_seq *seqs, int32_t n_seq, int32_t total_rows,
                       void *stream);

/* The same for one row of each of `rows` sequences (a decode step): row r is
 * position pos[r] (device int64, also o1_head_prep's) of slot slots[r] (device
 * int32; NULL: slot r). A row whose slot or position is out of range is padding
 * and written nowhere. Of rows that name the same position of a slot the first
 * counts (with the slots' look of o1_lin_token_attend: each row is compared with all
 * before it, work that grows with the square of the rows). At most 65536 rows.
 * One launch; asynchronous. */
O1_API int o1_pg_token_write(const o1_pg_geom *geom, const o1_pg_cache *cache, const void *k, int64_t k_stride,
                             const void *v, int64_t v_stride, const int32_t *slots, const int64_t *pos, int32_t rows,
                             void *stream);

/* Read cached rows back: row row0 + i of a sequence is what position pos0 + i of
 * its slot holds, rounded to the row tensors' type (exact for all but e4m3 values
 * beyond fp16's range). Sequences as for o1_pg_write, except that positions may
 * be read more than once. Rows of no sequence, and those of absent pages, are
 * left as they were.
 *   k, v  device row tensors [total_rows][G][d], [total_rows][G][dv], written
 * Asynchronous; a launch every 128 sequences. */
O1_API int o1_pg_read(const o1_pg_geom *geom, const o1_pg_cache *cache, const o1_pg_seq *seqs, int32_t n_seq, void *k,
                      int64_t k_stride, void *v, int64_t v_stride, int32_t total_rows, void *stream);

/* Bytes of device scratch of the two attend calls for up to `rows` rows (the
 * partial results of heads whose keys are split over several blocks); it does
 * not grow with the cache. Host-only; 0 if the geometry is unsupported or rows <
 * 1. */
O1_API size_t o1_pg_scratch_bytes(const o1_pg_geom *geom, int32_t rows);

/* Attention of the rows of packed sequences over the cache: the row at position
 * p of a slot attends its positions max(0, p - window + 1) .. p (window 0: from
 * 0) on present pages,
 *   out = sum_j w_j v_j / sum_j w_j,  w_j = e^{scale q . k_j},
 * per query head, with the keys and values of its group. The rows' own keys and
 * values are in the cache before (o1_pg_write). A row with no position left is 0.
 *   scratch  device, 256-byte aligned, o1_pg_scratch_bytes(geom, total_rows) at least
 *   q        device row tensor [total_rows][nh][d]
 *   seqs     as for o1_pg_read; rows * heads_per_group < 2^31 - 512 of each
 *   out      device row tensor [total_rows][nh][dv]; rows of no sequence are
 *            left as they were
 * q and what is attended are finite, and scores below 2^127 in fp32. A
 * non-finite key or value spoils rows of its own sequence only: from its
 * position on, and less than 384 before it. Positions that no row of the
 * sequence attends (past its end, before its window) may hold anything.
 * Scores, the softmax's maxima and sums and the outputs' sums are fp32. The
 * products run on the tensor cores with the cached values as they are; of the
 * other operand, q is exact (16-bit rows over e4m3: to 2^-25 of its largest
 * value), and the softmax's weights are rounded to 2^-8 (bf16 rows), 2^-11 (fp16
 * rows) or 2^-24 (fp32 rows) of their value. Some are held in fp16: those of fp16
 * rows over fp16, and of 16-bit rows over e4m3 in token batches and in calls whose
 * sequences all have rows * heads_per_group <= 16 (2^-11, of bf16 rows too). These
 * are off by up to 2^-32 of the row's largest weight where that is more; over e4m3,
 * where a weight is held times its value's power of two, of the largest such
 * product.
 * One kernel takes all sequences of a call (where some have rows * heads_per_group
 * > 16, in tiles of 128 or 256 query vectors), so that single rows of long sequences
 * beside a prompt's chunk are better attended by a call of their own.
 * Calls that may overlap on the GPU (other streams, captured graphs) need a
 * scratch each. Asynchronous. */
O1_API int o1_pg_chunk_attend(const o1_pg_geom *geom, const o1_pg_cache *cache, void *scratch, size_t scratch_bytes,
                              const void *q, int64_t q_stride, const o1_pg_seq *seqs, int32_t n_seq, void *out,
                              int64_t out_stride, int32_t total_rows, void *stream);

/* The same for one row of each of `rows` sequences (a decode step of a batch):
 * row r is position pos[r] (device int64) of slot slots[r] (device int32; NULL:
 * slot r), whatever lengths the arrays hold when it runs, so that a captured
 * step can be replayed as the sequences grow. A row whose slot or position is
 * out of range is padding: its output is left as it was. A slot may be named by
 * several rows (draft rows at successive positions). At most 65536 rows. The
 * keys of all rows are split evenly over the GPU. Two launches at most;
 * asynchronous. */
O1_API int o1_pg_token_attend(const o1_pg_geom *geom, const o1_pg_cache *cache, void *scratch, size_t scratch_bytes,
                              const void *q, int64_t q_stride, const int32_t *slots, const int64_t *pos, void *out,
                              int64_t out_stride, int32_t rows, void *stream);

/* Read the sticky flags that o1_pg_chunk_attend's kernels raised on the current
 * device into *flags (host) and, if `clear` is non-zero, reset them:
 * O1_FLAG_WAIT_EXPIRED (a bounded wait ran out, see o1_set_wait_limit; the
 * outputs that the block was to write are NaN). Synchronises `stream`. */
O1_API int o1_pg_flags(uint32_t *flags, int32_t clear, void *stream);

/* A static, human-readable name for a status code. (The pages' geometry
 * gates refuse a shape instead of running it: "cortiq-engine 0.8.82
 * src/gpu_metal/o1c.rs", admits and tok_ok; this library returns
 * O1_ERR_UNSUPPORTED there.) */
O1_API const char *o1_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* O1_H */
