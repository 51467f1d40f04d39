/*
 * nvfp4.h -- C ABI of the MI355X (gfx950) NVFP4 activation producer and
 * block-scaled GEMM.
 *
 * What is computed (page title, section):
 *  - "NVFP4 Modulation Producer Fusion", Dataflow / Exactness Contract: the
 *    producer reads the normalized BF16 activation twice, reproduces the
 *    per-segment AdaLN modulation y = (x * (scale + 1)) + shift with BF16
 *    rounding after each operation, reduces |y| to its absolute maximum in the
 *    first pass, and writes packed QDATA and E4M3 block scales into
 *    caller-owned buffers in the second; y never reaches memory.
 *  - "NVFP4 Streaming Design", Numerical Constraint: the tensor's exact BF16
 *    maximum magnitude gives a single FP32 tensor scale; each 16 values get
 *    an E4M3 scale; E2M1 codes come from both scales; no tile can
 *    be packed before the global reduction completes (two passes).
 *  - "FC2 NVFP4 Library Scheduling", Exact Operation: packed activation rows
 *    [M,K] against packed weight rows [N,K], giving BF16 [M,N]; FP32 compute;
 *    alpha = activation tensor scale * weight tensor scale, read from device
 *    memory; no bias; 37,810 logical rows padded to 37,824; the FC2 producer
 *    fuses an exact BF16 SwiGLU.
 *
 * The quantizer the pages leave open is fixed here as:
 *   s_g = amax / 2688 (= 6 * 448), or 1 when amax == 0
 *   sf  = E4M3(RN(RN(a16 / 6) / s_g)), nearest-even, saturating at 448
 *   q   = E2M1(RN(y / RN(float(sf) * s_g))), nearest with ties to the even
 *         code, saturating at +-6, sign kept; all 16 codes 0 when sf is 0
 *         (or the NaN code)
 * with every operation a correctly rounded binary32 operation (no FMA
 * contraction, no flush-to-zero, no approximate reciprocal).
 *
 * Layouts (all row-major, bf16 given as uint16_t bit patterns):
 *   x       [M, D]   bf16, row stride ldx elements
 *   qdata   [M_pad, D/2]  uint8: byte j of a row holds element 2j in bits 3..0
 *                         and element 2j+1 in bits 7..4
 *   sfa     [M_pad, D/16] uint8 E4M3FN, one per 16 consecutive elements
 *   rows M..M_pad-1 of qdata and sfa are written as zero.
 *
 * Conventions:
 *  - Every pointer is device memory except nvfp4_segments.row_start (host).
 *  - Buffers are caller-owned; the library allocates nothing and never
 *    synchronizes the host.  Work is enqueued on `stream` (a hipStream_t
 *    passed as void*; NULL = the null stream) in stream order, so
 *    absmax -> pack -> gemm on one stream need no synchronization.
 *  - Argument errors are reported synchronously, before anything is enqueued.
 *    A launch failure returns NVFP4_ERR_HIP; nvfp4_last_hip_error() gives the
 *    HIP error code of the calling thread's last failure.
 *  - Data-dependent conditions are not reported: a non-finite input yields a
 *    non-finite tensor scale, which the caller can test.
 *  - Calls that share a workspace or outputs must not overlap in time (for
 *    example on two streams without ordering between them).
 *  - The SwiGLU entry points first enqueue a small kernel that fills a
 *    65,536-entry bf16 silu table held in the library's own module-scope
 *    device memory (128 KB per device, part of the code object, not an
 *    allocation); calls overlapping on other streams write identical values.
 */
#ifndef NVFP4_H
#define NVFP4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    NVFP4_OK = 0,
    NVFP4_ERR_INVALID_ARGUMENT = 1, /* null pointer, non-positive size, ld too small */
    NVFP4_ERR_SHAPE = 2,            /* width not a multiple of 16 (64 for the GEMM's K), M_pad < pad64(M) */
    NVFP4_ERR_ALIGNMENT = 3,        /* base pointer or stride breaks the 16-byte rule */
    NVFP4_ERR_SEGMENTS = 4,         /* bad segment table */
    NVFP4_ERR_HIP = 5               /* kernel launch failed */
} nvfp4_status;

/* Per-segment modulation parameters ("NVFP4 Modulation Producer Fusion",
 * Exactness Contract: each segment selects its own shift and scale).  Segment s
 * covers rows [row_start[s], row_start[s+1]); row_start has count+1 HOST
 * entries with row_start[0] = 0, strictly increasing, row_start[count] = M,
 * 1 <= count <= NVFP4_MAX_SEGMENTS.  shift and scale are DEVICE bf16 arrays
 * [count, D] with row stride ld (>= D, multiple of 8, 16-byte aligned base). */
#define NVFP4_MAX_SEGMENTS 16
typedef struct {
    int32_t count;
    const int64_t* row_start;
    const uint16_t* shift;
    const uint16_t* scale;
    int64_t ld;
} nvfp4_segments;

/* ceil(m / 64) * 64: the padded row count of QDATA/SFA (37,810 -> 37,824,
 * "FC2 NVFP4 Library Scheduling", Exact Operation). */
int64_t nvfp4_padded_rows(int64_t m);

/* Bytes of device workspace the absmax passes and the single launches need
 * (16,640: the global maximum and a counter of the two-pass kernels, and the
 * single launch's result word and one arrival word and one claim word per
 * workgroup).  The workspace must be zero-filled before its first use; after
 * that any sequence of calls may reuse it without clearing (the two-pass
 * kernels return their words to zero, the single launch tags its words with
 * a tag no earlier launch in the process used).  It must not be shared by
 * calls that may overlap. */
size_t nvfp4_absmax_workspace_bytes(void);

/* Byte offset, within that workspace, of a uint32 count of the single
 * launches on it whose grid-barrier wait passed its bound (each such launch
 * adds one, from the device).  The library never resets it; zeroing the
 * workspace does.  A caller checks for timed-out launches without a host
 * synchronization by copying these 4 bytes asynchronously, or by reading them
 * in a later kernel on the same stream.  nvfp4_modulate_quantize_noalloc keeps
 * no such count (it clears its words on every call). */
#define NVFP4_WORKSPACE_TIMEOUT_COUNT_OFFSET 192

/* Sets the bound on the single launches' grid-barrier wait, in microseconds
 * (default 1,000,000), for launches enqueued from then on; returns the
 * previous bound.  A launch whose wait passes the bound completes with a NaN
 * tensor scale and amax, scale code 0x7F and zero codes in every block; 0
 * makes every single launch do so at once (a way to test that path). */
uint64_t nvfp4_set_barrier_timeout_us(uint64_t microseconds);

/* Sets how long a workgroup of a single launch waits at the grid barrier
 * before it computes the pass 1 of workgroups that have not arrived, in
 * microseconds (default 100), for launches enqueued from then on; returns the
 * previous value.  Results do not depend on it; 0 makes every workgroup help
 * from its arrival on (a way to test the helping path). */
uint64_t nvfp4_set_barrier_help_us(uint64_t microseconds);

/* Pass 1 of the modulation producer ("NVFP4 Modulation Producer Fusion",
 * Dataflow, prototype step 1; "NVFP4 Streaming Design", Numerical Constraint,
 * steps 1-2).  Computes y for every element of x [M, D] (row stride ldx, in
 * elements), reduces max |y| over all M rows, and writes
 *   *tensor_scale = amax == 0 ? 1 : RN(amax / 2688)   (device float)
 *   *amax_out     = amax                              (device float, may be NULL)
 * Requirements: M >= 1, D >= 16, D % 16 == 0, ldx >= D, ldx % 8 == 0, x
 * 16-byte aligned; seg valid for M rows and width D. */
nvfp4_status nvfp4_modulate_absmax(const uint16_t* x, int64_t M, int64_t D, int64_t ldx,
                                   const nvfp4_segments* seg, void* workspace,
                                   float* tensor_scale, float* amax_out, void* stream);

/* Pass 2 of the modulation producer ("NVFP4 Modulation Producer Fusion",
 * Dataflow, prototype step 2; "NVFP4 Streaming Design", Numerical Constraint,
 * steps 3-4).  Recomputes y and writes qdata [M_pad, D/2] and sfa
 * [M_pad, D/16] using the device scalar *tensor_scale (normally written by
 * nvfp4_modulate_absmax on the same stream).  Rows M..M_pad-1 are zero.
 * Requirements as for absmax, plus M_pad >= nvfp4_padded_rows(M) and qdata
 * 4-byte aligned. */
nvfp4_status nvfp4_modulate_pack(const uint16_t* x, int64_t M, int64_t D, int64_t ldx,
                                 const nvfp4_segments* seg, const float* tensor_scale,
                                 uint8_t* qdata, uint8_t* sfa, int64_t M_pad, void* stream);

/* Both passes of the modulation producer in one launch (same results as
 * nvfp4_modulate_absmax followed by nvfp4_modulate_pack, byte for byte).  The
 * workgroups (at most as many as the device holds at once) run pass 1, meet
 * at a grid barrier once the global maximum is complete ("NVFP4 Streaming
 * Design", Numerical Constraint: no block is packed before the global
 * reduction, and the two phases may be joined around a grid-wide barrier),
 * and run pass 2, which takes the y of
 * the rows each workgroup visited last from registers and LDS instead of
 * reading x again.  Writes *tensor_scale, *amax_out (may be NULL), qdata and
 * sfa as the two calls do; uses the same workspace.  The barrier needs every
 * workgroup's pass 1, not every workgroup's presence: workgroups that have
 * waited 100 us (nvfp4_set_barrier_help_us) compute the pass 1 of workgroups that could not start (their
 * CUs held by other kernels, for instance another single launch waiting at
 * its own barrier), so concurrent launches complete; the workgroups that
 * start late find the barrier passed.  A wait past the bound of
 * nvfp4_set_barrier_timeout_us (1 s by default) gives a NaN tensor scale and
 * amax, scale code 0x7F and zero codes in every block, for that call only,
 * and adds one to the workspace's timeout count
 * (NVFP4_WORKSPACE_TIMEOUT_COUNT_OFFSET).
 * Calls that can overlap in time must use different workspaces.  Each call
 * takes its barrier tag from the host when it is enqueued, so a call captured
 * into a HIP graph would replay one tag and find the previous replay's words
 * already arrived: under graph capture use nvfp4_modulate_quantize_noalloc
 * (its words are cleared by a kernel on every call) or the two calls
 * nvfp4_modulate_absmax + nvfp4_modulate_pack (whose words return to zero).
 * When D > 16384, or x spans 4 GiB or more, it enqueues the two passes
 * instead.
 * Same requirements as nvfp4_modulate_absmax and nvfp4_modulate_pack
 * together. */
nvfp4_status nvfp4_modulate_quantize(const uint16_t* x, int64_t M, int64_t D, int64_t ldx,
                                     const nvfp4_segments* seg, void* workspace, float* tensor_scale,
                                     float* amax_out, uint8_t* qdata, uint8_t* sfa, int64_t M_pad,
                                     void* stream);

/* nvfp4_modulate_quantize for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): the same results, byte for byte, with no workspace argument.
 * The grid barrier's words live in a fixed 16,640-byte array inside the
 * library's code object, one copy per device (held until the process ends);
 * every shape nvfp4_modulate_quantize accepts fits it.  The call enqueues a
 * small kernel that zeroes those words, then the producer, on `stream`; it
 * calls no allocator.  Because the words are cleared by a kernel, a call
 * captured into a graph replays correctly (make one call outside capture
 * first: it looks up the array's address and the grid size).  All calls on one device share the array: calls that
 * can overlap in time on one device (two streams without ordering between
 * them) race and must not be made.  Same arguments, requirements and errors
 * as nvfp4_modulate_quantize, without the workspace. */
nvfp4_status nvfp4_modulate_quantize_noalloc(const uint16_t* x, int64_t M, int64_t D, int64_t ldx,
                                             const nvfp4_segments* seg, float* tensor_scale, float* amax_out,
                                             uint8_t* qdata, uint8_t* sfa, int64_t M_pad, void* stream);

/* The plain quantizer: nvfp4_modulate_quantize with y = x (no modulation), for
 * activations that need none (the attention-output projection's input,
 * "NVFP4 Streaming Design", P0/P2: the widths 5376, 7168, 14336) and for
 * prepacking weights.  Same launch structure, outputs, workspace,
 * requirements and graph-capture caveat, without the segment table. */
nvfp4_status nvfp4_quantize(const uint16_t* x, int64_t M, int64_t D, int64_t ldx, void* workspace,
                            float* tensor_scale, float* amax_out, uint8_t* qdata, uint8_t* sfa, int64_t M_pad,
                            void* stream);

/* Pass 1 of the SwiGLU producer ("FC2 NVFP4 Library Scheduling", Exact
 * Operation and Current Baseline: exact BF16 SwiGLU fused into NVFP4
 * production).  h = bf16(bf16(silu(g)) * u) with silu(g) = g / (1 + exp(-g))
 * in binary32 with a correctly rounded exp; g = gate[r*ld + c],
 * u = up[r*ld + c] for c < F.  For one [M, 2F] gate/up tensor pass
 * gate = GU, up = GU + F, ld = 2F.  Writes tensor scale and amax as
 * nvfp4_modulate_absmax.  Requirements: F % 16 == 0, ld >= F, ld % 8 == 0,
 * gate and up 16-byte aligned. */
nvfp4_status nvfp4_swiglu_absmax(const uint16_t* gate, const uint16_t* up, int64_t M, int64_t F,
                                 int64_t ld, void* workspace, float* tensor_scale, float* amax_out,
                                 void* stream);

/* Pass 2 of the SwiGLU producer: recomputes h and writes qdata [M_pad, F/2]
 * and sfa [M_pad, F/16] with the device *tensor_scale; pad rows zero. */
nvfp4_status nvfp4_swiglu_pack(const uint16_t* gate, const uint16_t* up, int64_t M, int64_t F,
                               int64_t ld, const float* tensor_scale, uint8_t* qdata, uint8_t* sfa,
                               int64_t M_pad, void* stream);

/* Both SwiGLU passes in one call (same results as nvfp4_swiglu_absmax
 * followed by nvfp4_swiglu_pack, byte for byte): after the silu table fill,
 * one launch runs pass 1, a grid barrier and pass 2, keeping h of the rows
 * each workgroup visited last in registers, as nvfp4_modulate_quantize does
 * (same workspace, the same barrier with helping, the same bound, and the
 * same caveat under graph capture: use the two calls there).  When
 * F > 16384, or gate/up spans
 * 4 GiB or more, it enqueues the two passes instead.  Same arguments,
 * requirements and errors as the two calls together. */
nvfp4_status nvfp4_swiglu_quantize(const uint16_t* gate, const uint16_t* up, int64_t M, int64_t F,
                                   int64_t ld, void* workspace, float* tensor_scale, float* amax_out,
                                   uint8_t* qdata, uint8_t* sfa, int64_t M_pad, void* stream);

/* Block-scaled GEMM ("FC2 NVFP4 Library Scheduling", Exact Operation;
 * "NVFP4 Streaming Design", P0: FP32 global-scale product applied before the
 * BF16 conversion):
 *   out[m][n] = bf16(RN(alpha * sum_k A[m][k] * W[n][k])),  m < M, n < N
 *   A = e2m1(qa) * e4m3(sfa), W = e2m1(qw) * e4m3(sfw),
 *   alpha = RN(*a_scale * *w_scale)  (both device floats)
 * qa [M_pad, K/2], sfa [M_pad, K/16] (rows >= M are read as padding and
 * ignored), qw [N, K/2], sfw [N, K/16], out [M, ldo] bf16.  The K sum is
 * accumulated in binary32 in an order of the kernel's choosing.
 * Requirements: K % 64 == 0, N % 16 == 0, ldo >= N, ldo % 4 == 0,
 * M_pad >= M, qa/qw 16-byte aligned, sfa/sfw 4-byte aligned, out 8-byte
 * aligned; N * K/2 < 2^32 (the packed weight under 4 GiB), K <= 2^25,
 * M_pad < 2^31.  The activation may exceed 4 GiB: the rows are then computed
 * in chunks of floor((2^32 - 1) / (K/2)) rounded down to a multiple of 256, one
 * launch sequence per chunk in stream order. */
nvfp4_status nvfp4_gemm(const uint8_t* qa, const uint8_t* sfa, const float* a_scale, int64_t M,
                        int64_t M_pad, const uint8_t* qw, const uint8_t* sfw, const float* w_scale,
                        int64_t N, int64_t K, uint16_t* out, int64_t ldo, void* stream);

/* Bytes of device workspace nvfp4_gemm_ws uses for an [M,K] x [N,K] product
 * (0 when it has nothing to split; for an activation in several row chunks,
 * the largest chunk's need).  Depends on the shape only. */
size_t nvfp4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K);

/* nvfp4_gemm with a caller-owned workspace of at least
 * nvfp4_gemm_workspace_bytes(M, N, K) bytes (16-byte aligned; may be NULL when
 * that is 0).  The output tiles are computed in waves of 256 workgroups; when
 * the last wave would fill at most a third of the chip, its tiles are each
 * computed as several K ranges by separate workgroups whose binary32 partial
 * sums land in the workspace, then added in K order and scaled by alpha.  The
 * result satisfies the same contract as nvfp4_gemm (only the binary32
 * summation order differs).  The workspace holds no state between calls;
 * calls sharing it must not overlap.  Like nvfp4_gemm it enqueues kernels
 * only (no memset, no allocation), so a call can be captured into a HIP graph
 * and replayed with new operands in the same buffers.  Same requirements and errors as
 * nvfp4_gemm, plus NVFP4_ERR_INVALID_ARGUMENT for a missing or short
 * workspace. */
nvfp4_status nvfp4_gemm_ws(const uint8_t* qa, const uint8_t* sfa, const float* a_scale, int64_t M,
                           int64_t M_pad, const uint8_t* qw, const uint8_t* sfw, const float* w_scale,
                           int64_t N, int64_t K, uint16_t* out, int64_t ldo, void* workspace,
                           size_t workspace_bytes, void* stream);

/* Per-segment gates of the residual epilogue: segment s covers output rows
 * [row_start[s], row_start[s+1]) (count+1 HOST entries, 0 .. M, strictly
 * increasing, 1 <= count <= NVFP4_MAX_SEGMENTS) and uses the DEVICE bf16 gate
 * row gate[s * ld .. s * ld + N). */
typedef struct {
    int32_t count;
    const int64_t* row_start;
    const uint16_t* gate;
    int64_t ld;
} nvfp4_row_gates;

/* nvfp4_gemm_ws followed by the exact residual epilogue ("NVFP4 Streaming
 * Design", P4: the GEMM result rounded to BF16, scaled by the gate, added to
 * the residual and rounded to BF16 again), fused into the GEMM's store:
 *   o   = bf16(RN(alpha * sum_k A[m][k] * W[n][k]))   (the nvfp4_gemm output)
 *   out = bf16(RN(residual[m][n] + bf16(RN(gate[s][n] * o))))
 * with s the segment of row m; residual is bf16 [M, ldr].  out may be the
 * residual itself (same pointer and stride: each element is read before it is
 * written, by the same thread); otherwise the two must not overlap.  Same
 * requirements and workspace as nvfp4_gemm_ws, plus: gate and residual 8-byte
 * aligned, gates->ld and ldr >= N and multiples of 4; a bad gate table returns
 * NVFP4_ERR_SEGMENTS. */
nvfp4_status nvfp4_gemm_gate_residual(const uint8_t* qa, const uint8_t* sfa, const float* a_scale, int64_t M,
                                      int64_t M_pad, const uint8_t* qw, const uint8_t* sfw, const float* w_scale,
                                      int64_t N, int64_t K, const nvfp4_row_gates* gates, const uint16_t* residual,
                                      int64_t ldr, uint16_t* out, int64_t ldo, void* workspace,
                                      size_t workspace_bytes, void* stream);

/* ---- Packed-tile ring ---------------------------------------------------
 * "NVFP4 Streaming Design", P2 (N-group reuse): instead of materializing the
 * whole packed activation, a bounded ring of packed row slots; one tensor
 * scale from the full activation is reused by every chunk, each chunk of rows
 * is packed into a slot and multiplied by the whole weight, and the slot is
 * recycled.  The pages chose 2048-row chunks (18 full ones and a last one of
 * 946 rows at 37,810 rows) and reported the ring slower than the
 * materialized path at block level on their GPU; here it is an opt-in entry
 * point with the same results as nvfp4_modulate_quantize followed by
 * nvfp4_gemm_ws, so the two can be compared. */

/* Bytes of one ring slot: chunk_rows rows of QDATA (K/2 bytes each) followed
 * by chunk_rows rows of SFA (K/16 bytes each).  0 for an invalid argument
 * (chunk_rows and K must be positive multiples of 64). */
size_t nvfp4_ring_slot_bytes(int64_t chunk_rows, int64_t K);

/* Bytes of GEMM workspace nvfp4_modulate_gemm_ring needs: two K-split
 * workspaces (one per GEMM stream) for the larger of a full and the last
 * chunk.  0 when no chunk's GEMM splits (or for an invalid argument). */
size_t nvfp4_ring_gemm_workspace_bytes(int64_t M, int64_t chunk_rows, int64_t N, int64_t K);

/* Modulation producer and GEMM through a ring of `slots` packed slots:
 *   1. pass 1 over all M rows of x [M, K]: *tensor_scale, *amax_out (may be
 *      NULL), as nvfp4_modulate_absmax (same workspace rules);
 *   2. for chunk c (rows [c*chunk_rows, min(M, (c+1)*chunk_rows))): pass 2 of
 *      its rows into slot c % slots (rows past the chunk's last row up to the
 *      next multiple of 64 are zero), then the GEMM of that slot against the
 *      packed weight qw [N, K/2], sfw [N, K/16] with alpha = RN(*tensor_scale
 *      * *w_scale), written to out rows [c*chunk_rows, ...) (bf16 [M, ldo]).
 * The slot bytes of chunk c equal rows c*chunk_rows .. of the QDATA/SFA that
 * nvfp4_modulate_quantize writes; the outputs satisfy nvfp4_gemm's contract
 * and, when chunk_rows is a multiple of 256, equal nvfp4_gemm_ws's bit for bit
 * except in tiles that either call computes as K-split pieces.
 * Streams: pass 1 and the even chunks' GEMMs run on `stream`; the packs and
 * the odd chunks' GEMMs on two streams the library creates once per device
 * (default priority), ordered by events: a pack waits for the GEMM that last
 * read its slot, a GEMM for its chunk's pack, and `stream` waits for all of it
 * before its next work, so the call is stream-ordered for the caller.  No
 * workgroup waits on another.  The ring (16-byte aligned, at least
 * slots * nvfp4_ring_slot_bytes(chunk_rows, K) bytes) and gemm_workspace
 * (nvfp4_ring_gemm_workspace_bytes) are caller-owned and must not be shared
 * with calls that may overlap; calls on one device are enqueued one at a time
 * (a host lock).
 * Requirements: those of nvfp4_modulate_absmax, nvfp4_modulate_pack and
 * nvfp4_gemm_ws; 1 <= slots <= 64; chunk_rows a multiple of 64 with
 * chunk_rows * K/2 < 2^32. */
nvfp4_status nvfp4_modulate_gemm_ring(const uint16_t* x, int64_t M, int64_t K, int64_t ldx,
                                      const nvfp4_segments* seg, void* workspace, float* tensor_scale,
                                      float* amax_out, uint8_t* ring, int32_t slots, int64_t chunk_rows,
                                      const uint8_t* qw, const uint8_t* sfw, const float* w_scale, int64_t N,
                                      uint16_t* out, int64_t ldo, void* gemm_workspace, size_t gemm_workspace_bytes,
                                      void* stream);

/* ---- Rotary positions, the 8-bit key/value cache and attention over it ----
 * What lies between the QKV projection and the quantizer of the attention
 * output's projection: rotate the queries (nvfp4_rope), write keys and values
 * into a paged cache of 8-bit codes (nvfp4_kv_write, rotating the keys on the
 * way where asked), and attend over the cache (nvfp4_kv_attention).  All of
 * them enqueue kernels only, keep no state between calls, and replay correctly
 * under graph capture. */

/* Heads [rows, heads, dim] in device memory, bf16, unit stride along dim: head
 * h of row m starts at data + m * row_stride + h * head_stride (elements, both
 * multiples of 8 and not negative, at most 2^38; data 16-byte aligned; neither
 * (rows - 1) * row_stride nor (heads - 1) * head_stride past 2^60).  A third of a
 * QKV product and [heads, rows, dim] are both of this form.  As an output no two
 * heads may overlap: row_stride >= (heads - 1) * head_stride + dim with
 * head_stride >= dim, or head_stride >= (rows - 1) * row_stride + dim with
 * row_stride >= dim. */
typedef struct {
    uint16_t* data;
    int64_t row_stride;
    int64_t head_stride;
} nvfp4_heads;

/* Rotary positions with 1 to 4 axes (a token's place, or time, height and
 * width).  A head's first 2 * sum(pairs) dims are rotated; the pairs are shared
 * out over the axes in order, axis a taking pairs[a] of them.  Pair i is dims
 * (2i, 2i + 1), or with split != 0 dims (i, i + sum(pairs)).  Pair i of axis a
 * (its first being i0) turns by the angle whose (cos, sin) is
 * table[a][positions[m][a]][i - i0], binary32:
 *   y1 = bf16(RN(RN(x1 cos) - RN(x2 sin))),  y2 = bf16(RN(RN(x2 cos) + RN(x1 sin))).
 * pairs[a] >= 1, sum(pairs) a multiple of 8 and at most dim / 2.  table[a] is a
 * DEVICE array [rows[a]][pairs[a]][2] (8-byte aligned, rows[a] >= 1), positions
 * a DEVICE int32 array [M][axes] with row stride ld_positions >= axes.  A
 * position outside [0, rows[a]) gives NaN; nothing is read for it. */
#define NVFP4_ROPE_MAX_AXES 4
typedef struct {
    int32_t axes;
    int32_t split;
    int32_t pairs[NVFP4_ROPE_MAX_AXES];
    int64_t rows[NVFP4_ROPE_MAX_AXES];
    const float* table[NVFP4_ROPE_MAX_AXES];
    const int32_t* positions;
    int64_t ld_positions;
} nvfp4_rope_params;

/* The usual table of one axis: (cos, sin) of p * theta^(-j / pairs) for
 * positions p < rows and j < pairs, formed in binary64 and rounded to binary32.
 * rows >= 1, pairs >= 1, rows * pairs < 2^28, theta > 0 and finite. */
nvfp4_status nvfp4_rope_table(float* table, int64_t rows, int32_t pairs, double theta, void* stream);

/* Rotates x [M, heads, dim] into out; dims past the rotated ones are copied.
 * out may be x itself (same data and strides); otherwise they must not overlap.
 * dim a multiple of 16, at most 512; 1 <= M <= 2^23; a bad rope table returns
 * NVFP4_ERR_SHAPE. */
nvfp4_status nvfp4_rope(const nvfp4_heads* x, int64_t M, int32_t heads, int32_t dim, const nvfp4_rope_params* rope,
                        const nvfp4_heads* out, void* stream);

/* A pool of cache blocks.  A block holds 64 positions of every key/value head:
 * for each head one E4M3 code per value and, apart for keys and values, one
 * power of two, held as the byte b that stands for 2^(b - 127).  The power is
 * the smallest with amax <= 448 * 2^(b - 127) over the block's finite values
 * (b >= 1); a code is the nearest E4M3 (ties to even) of value / 2^(b - 127),
 * or a NaN code where the value is not finite; with b = 247, the largest that
 * occurs, codes stop at 240, so that code * power is finite.  A power of two leaves E4M3's
 * relative precision as it is and makes code * power exact in bf16.
 *   k [blocks][heads][dim / 16][64][16]: dims 16c..16c+15 of position t at [c][t]
 *   v [blocks][heads][4][dim][16]: position t = 32u + 16e + 8m + 4h + j (e, m, h
 *     in {0, 1}, j < 4) of dim d at [2u + h][d][8e + 4m + j]
 *   k_power, v_power [blocks][heads]
 * dim 64 or 128; k and v 16-byte aligned.  A block needs no initial value. */
#define NVFP4_KV_BLOCK 64
typedef struct {
    uint8_t* k;
    uint8_t* v;
    uint8_t* k_power;
    uint8_t* v_power;
    int64_t blocks;
    int32_t heads;
    int32_t dim;
} nvfp4_kv_cache;

/* `count` sequences, all arrays DEVICE int32.  Sequence b has new rows
 * [row_start[b], row_start[b + 1]) of the M rows of a call (count + 1 entries,
 * nondecreasing; a sequence may have none, and rows outside all sequences are
 * neither read nor written), which are its last positions: with lens[b]
 * positions in all, the new ones among them, row row_start[b] + i is position
 * lens[b] - n + i.  Position p lies in cache block table[b][p / 64]
 * (table row stride ld_table >= table_blocks, entries of unused blocks are not
 * read).  1 <= count <= 2^20.  The arrays' contents are not checked by the host:
 * whatever they hold, no access leaves the arrays, M rows and pool given. */
typedef struct {
    int64_t count;
    const int32_t* row_start;
    const int32_t* lens;
    const int32_t* table;
    int64_t ld_table;
    int64_t table_blocks;
} nvfp4_kv_sequences;

/* Quantises the M rows of k and v [M, heads, dim] and writes them to their
 * positions; with a rope the keys are rotated first, as nvfp4_rope does.  A
 * block that already holds positions of the sequence before the new ones keeps
 * them: its power becomes the larger of the old and what the new values need,
 * and where it grew the held codes are re-encoded, E4M3(code * 2^(old - new)).
 * Bytes of positions after the last are left as they were, but for the values'
 * in a block that new values give the largest power, b = 247: they become 0,
 * since what an earlier use of the block left there may not be finite with it.  Rows whose block
 * does not exist (an entry outside the pool, a length that the table cannot
 * hold, a position before 0) are skipped.  No block may be written twice in one
 * call, by two sequences or by one whose table names it twice (the bytes that it
 * would hold are not defined).  1 <= M <= 2^23. */
nvfp4_status nvfp4_kv_write(const nvfp4_kv_cache* cache, const nvfp4_kv_sequences* seqs, int64_t M,
                            const nvfp4_heads* k, const nvfp4_heads* v, const nvfp4_rope_params* rope, void* stream);

/* Reads the positions of the M rows back: k and v [M, heads, dim] = code *
 * power, exact in bf16.  A row before position 0 is 0; one whose block does not
 * exist, NaN.  k and v must not overlap; sequences may share blocks. */
nvfp4_status nvfp4_kv_read(const nvfp4_kv_cache* cache, const nvfp4_kv_sequences* seqs, int64_t M,
                           const nvfp4_heads* k, const nvfp4_heads* v, void* stream);

/* Attention of the queries q [M, q_heads, dim] over their sequences' cached
 * keys and values; query head g reads key/value head g / (q_heads / heads).
 *   out[m][g] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * q.k_j - max)
 * over positions j below the row's limit: lens[b] with causal_block = 0; with
 * causal_block = c >= 1 the end of the row's own run of c positions, at most
 * lens[b] (c = 1: a row sees itself and what is before it).  A row that sees
 * nothing gives 0.  Whatever a hidden position holds has no effect; a NaN that
 * is seen, a query that is not finite, a block outside the pool or a length
 * that the table cannot hold gives NaN.
 * Products and sums are binary32.  The keys' codes are multiplied as they are;
 * a query is split into two E4M3 numbers that together hold each bf16 element
 * to its last bit, or to 2^-21 of the row's largest element where that is
 * more.  Probabilities are rounded to bf16 for the product with the values, and
 * the output once to bf16.  (The sums run against a reference that may lie a few
 * powers of two below the maximum and is itself a binary32 number: values above
 * 2^96, or scaled scores above 2^26, can overflow them, and so can q.k past
 * binary32 before it is scaled.)  The order of the sums depends on the sizes and
 * max_len only: the same call gives the same bytes.
 * max_len is the host's bound on the lengths, used to decide how many rows a
 * workgroup takes and how far the keys of few rows are shared out over
 * workgroups (results for longer sequences are right all the same).  Both are
 * decided once for all sequences of a call: single tokens over long contexts are
 * faster apart from prompts.  The workspace needs
 * nvfp4_kv_attention_workspace_bytes(...) bytes for the same sizes (16-byte
 * aligned; may be NULL when that is 0); calls that can overlap must not share
 * it.  scale > 0, and scale * log2(e) finite in binary32; causal_block, max_len
 * >= 0; q_heads a multiple of cache->heads, M * q_heads <= 2^28; out may be q
 * itself. */
size_t nvfp4_kv_attention_workspace_bytes(int64_t M, int64_t count, int32_t q_heads, int32_t heads, int32_t dim,
                                          int64_t max_len);
nvfp4_status nvfp4_kv_attention(const nvfp4_heads* q, int64_t M, int32_t q_heads, const nvfp4_kv_cache* cache,
                                const nvfp4_kv_sequences* seqs, float scale, int32_t causal_block, int64_t max_len,
                                const nvfp4_heads* out, void* workspace, size_t workspace_bytes, void* stream);

/* ---- Around the cache ------------------------------------------------------
 * What a serving step does besides: norms of the heads, the tables that the
 * cache's calls take, attention that sees a part of the past, and attention over
 * a prefix that the sequences of a batch share.  As above: kernels only, no state
 * between calls, and replays under graph capture are right. */

/* Root-mean-square norms of query and key heads, with rotary positions:
 *   n_i = x_i w_i / sqrt(mean_j x_j^2 + eps),  j over the head's dim elements,
 *   y1 = n1 cos - n2 sin,  y2 = n2 cos + n1 sin  for the rotated pairs, y = n else,
 * in binary32, rounded once to bf16.  Squares that leave binary32 do no harm; an
 * element that is not finite does what the formula says.  q [M, q_heads, dim] and
 * k [M, k_heads, dim] with weights [dim] (bf16, 16-byte aligned; NULL: ones), both
 * in one launch; k_heads = 0: no keys (k, k_out NULL).  rope as in nvfp4_rope, or
 * NULL for no rotation.  Each output may be its own input (same data and strides);
 * otherwise no two of them overlap.  2^-126 <= eps <= 1; dim a multiple of 16, at
 * most 512; 1 <= M <= 2^23. */
nvfp4_status nvfp4_norm_rope(const nvfp4_heads* q, int32_t q_heads, const uint16_t* q_weight, const nvfp4_heads* k,
                             int32_t k_heads, const uint16_t* k_weight, int64_t M, int32_t dim, float eps,
                             const nvfp4_rope_params* rope, const nvfp4_heads* q_out, const nvfp4_heads* k_out,
                             void* stream);

/* The block tables of `count` requests and a stack of the pool's free blocks,
 * DEVICE int32.  table[b][j] is request b's cache block of positions 64 j .. 64 j +
 * 63 (row stride ld_table >= table_blocks); the stack's top is free_blocks[n - 1]
 * where n, at most `capacity`, is held apart.  1 <= count <= 2^20; 1 <= capacity <=
 * 2^30. */
typedef struct {
    int64_t count;
    int32_t* table;
    int64_t ld_table;
    int64_t table_blocks;
    int32_t* free_blocks;
    int64_t capacity;
} nvfp4_kv_tables;

/* Gives every request its next rows, positions and blocks.  Request b holds past[b]
 * positions and asks for more[b] (below 0: none).  In order of b:
 *   n = more[b], cut to the rows left of M and to a length below 2^31;
 *   row_start[b] = the rows of the requests before, row_start[count] all of them;
 *   lens[b] = past[b] + n;
 *   blocks ceil(past / 64) .. ceil(lens / 64) - 1 of its table (as far as the table
 *   goes) are taken from the top of the stack; where that is empty, the entry
 *   becomes -1 and *missing, the number of these, grows.
 * *free_left is the stack's size after it; the stack's own entries stay as they are.
 * The m-th row's position goes to positions[m] (int32) and its slot, block * 64 +
 * position % 64, to slots[m] (int64; -1 where there is no block); rows of no request
 * get -1 in both.  Either may be NULL.  row_start, lens, table and positions are what
 * nvfp4_kv_write, nvfp4_rope and nvfp4_kv_attention take: nothing of a step's tables
 * passes the host.  (slots are for a program's own kernels: no call here takes them.)  lens may be past and free_left may be free_count (a step in
 * place); otherwise outputs must not overlap one another or the inputs.  *free_count
 * is taken as at least 0 and at most capacity.  1 <= M <= 2^23.  The workspace needs
 * nvfp4_kv_extend_workspace_bytes(count) bytes (16-byte aligned). */
size_t nvfp4_kv_extend_workspace_bytes(int64_t count);
nvfp4_status nvfp4_kv_extend(const nvfp4_kv_tables* tables, const int32_t* past, const int32_t* more,
                             const int32_t* free_count, int64_t M, int32_t* row_start, int32_t* lens, int32_t* free_left,
                             int32_t* missing, int32_t* positions, int64_t* slots, void* workspace,
                             size_t workspace_bytes, void* stream);

/* Takes the blocks of finished requests back: of each b with done[b] != 0, in order,
 * the entries keep .. ceil(lens[b] / 64) - 1 of its table that are not negative go on
 * top of the stack (what would pass its capacity is dropped), and lens_out[b] = 0;
 * the other lengths are copied.  *free_left is the stack's size after it.  The table
 * stays as it is.  keep: the first entries of every table that are not the request's
 * own (a shared prefix).  lens_out may be lens and free_left may be free_count.  The
 * workspace needs nvfp4_kv_release_workspace_bytes(count) bytes (16-byte aligned; may
 * be NULL when that is 0).
 * A length of 0 says that a request holds no block.  Where its table still names the
 * kept ones, the next request in its place has to begin behind them: extended from 0 it
 * would put blocks of its own over the prefix's entries, which no release with that
 * `keep` gives back.  nvfp4_kv_release_to_prefix is for that: lens_out[b] of finished
 * requests becomes 64 * keep (at most 64 * table_blocks). */
size_t nvfp4_kv_release_workspace_bytes(int64_t count);
nvfp4_status nvfp4_kv_release(const nvfp4_kv_tables* tables, const int32_t* lens, const int32_t* done, int64_t keep,
                              const int32_t* free_count, int32_t* lens_out, int32_t* free_left, void* workspace,
                              size_t workspace_bytes, void* stream);
nvfp4_status nvfp4_kv_release_to_prefix(const nvfp4_kv_tables* tables, const int32_t* lens, const int32_t* done, int64_t keep,
                                        const int32_t* free_count, int32_t* lens_out, int32_t* free_left, void* workspace,
                                        size_t workspace_bytes, void* stream);

/* nvfp4_kv_attention through a window: of the positions below its limit, the row at
 * position p sees those above p - window and the first `sinks`; the others' blocks
 * are not read.  causal_block bounds what a row sees ahead of it, as there (with 0 all
 * of its sequence).  window >= 1, sinks >= 0.  What hidden positions hold has no
 * effect.  The sum that divides is of the probabilities as they were rounded to bf16,
 * where nvfp4_kv_attention adds them before: a key that has all the weight gives its
 * value as it is.  Everything else as nvfp4_kv_attention has it.  The workspace needs
 * nvfp4_kv_attention_window_workspace_bytes(...) bytes for the same sizes (16-byte
 * aligned; may be NULL when that is 0). */
size_t nvfp4_kv_attention_window_workspace_bytes(int64_t M, int64_t count, int32_t q_heads, int32_t heads, int32_t dim,
                                                 int32_t causal_block, int32_t window, int32_t sinks, int64_t max_len);
nvfp4_status nvfp4_kv_attention_window(const nvfp4_heads* q, int64_t M, int32_t q_heads, const nvfp4_kv_cache* cache,
                                       const nvfp4_kv_sequences* seqs, float scale, int32_t causal_block, int32_t window,
                                       int32_t sinks, int64_t max_len, const nvfp4_heads* out, void* workspace,
                                       size_t workspace_bytes, void* stream);

/* nvfp4_kv_attention of sequences whose first 64 * shared_blocks positions are the
 * same: the blocks shared[0 .. shared_blocks) (DEVICE int32) stand for the first
 * entries of every sequence's table, which are not read.  All rows of the batch are
 * taken against them together, so that a long prefix is read and multiplied in tiles
 * of many sequences' rows, and against their own sequence's further positions apart;
 * the two are joined by their maxima and sums, so that a row's result is that of one
 * softmax.  The new rows of every sequence lie behind the prefix: rows of one with
 * lens[b] - n < 64 * shared_blocks give NaN.  max_len bounds the lengths, prefix
 * included.  1 <= shared_blocks <= (2^31 - 1) / 64; the tables hold the prefix too
 * (lens[b] <= 64 * table_blocks).  The rounded probabilities are what is summed, as
 * through a window.  Everything else as nvfp4_kv_attention has it.  The
 * workspace needs nvfp4_kv_attention_shared_workspace_bytes(...) bytes for the same
 * sizes (16-byte aligned). */
size_t nvfp4_kv_attention_shared_workspace_bytes(int64_t M, int64_t count, int32_t q_heads, int32_t heads, int32_t dim,
                                                 int64_t shared_blocks, int64_t max_len);
nvfp4_status nvfp4_kv_attention_shared(const nvfp4_heads* q, int64_t M, int32_t q_heads, const nvfp4_kv_cache* cache,
                                       const nvfp4_kv_sequences* seqs, const int32_t* shared, int64_t shared_blocks,
                                       float scale, int32_t causal_block, int64_t max_len, const nvfp4_heads* out,
                                       void* workspace, size_t workspace_bytes, void* stream);

/* Rows of no sequence become 0.  The attention calls leave them as they were, so that a
 * call whose rows are not all in use (a captured step that is made for its largest)
 * leaves there what the output held before, and nvfp4_norm_rope gives NaN in rows at
 * position -1; nvfp4_quantize takes one scale from all M rows, these among them.  out
 * [M, heads, dim]: rows before row_start[0] and from row_start[count] on (DEVICE int32
 * [count + 1]) are written, no others.  dim a multiple of 16, at most 512; 1 <= M <=
 * 2^23; M * heads <= 2^28; 1 <= count <= 2^20. */
nvfp4_status nvfp4_kv_clear_rest(const nvfp4_heads* out, int64_t M, int32_t heads, int32_t dim, const int32_t* row_start,
                                 int64_t count, void* stream);

/* ---- Single-step entry points ------------------------------------------
 * Elementwise versions of single producer steps, running the very device
 * functions the producer kernels use, so that each step can be checked over
 * its whole input domain.  All arrays are device memory of n elements. */

/* a1: y[i] = bf16(bf16(bf16(x*bf16(scale+1))) + shift)
 * ("NVFP4 Modulation Producer Fusion", Exactness Contract). */
nvfp4_status nvfp4_step_modulate(const uint16_t* x, const uint16_t* scale, const uint16_t* shift,
                                 uint16_t* y, int64_t n, void* stream);
/* a6: h[i] = bf16(bf16(silu(g)) * u) ("FC2 NVFP4 Library Scheduling"). */
nvfp4_status nvfp4_step_swiglu(const uint16_t* g, const uint16_t* u, uint16_t* h, int64_t n,
                               void* stream);
/* a3: sf[i] = E4M3(RN(RN(a16[i] / 6) / *s_g)) with a16 given as bf16 bits
 * ("NVFP4 Streaming Design", Numerical Constraint, step 3). */
nvfp4_status nvfp4_step_block_scale(const uint16_t* a16, const float* s_g, uint8_t* sf, int64_t n,
                                    void* stream);
/* a4: code[i] = E2M1(RN(y[i] / RN(float(sf[i]) * *s_g))), 0 when sf[i] is 0
 * or the NaN code ("NVFP4 Streaming Design", Numerical Constraint, step 4). */
nvfp4_status nvfp4_step_element_code(const uint16_t* y, const uint8_t* sf, const float* s_g,
                                     uint8_t* code, int64_t n, void* stream);
/* E2M1 encoding of binary32 values (the conversion behind a4):
 * code[i] = E2M1(v[i]) with ties to the even code and saturation at +-6. */
nvfp4_status nvfp4_step_e2m1(const float* v, uint8_t* code, int64_t n, void* stream);
/* E4M3 encoding of non-negative binary32 values (the conversion behind a3). */
nvfp4_status nvfp4_step_e4m3(const float* t, uint8_t* code, int64_t n, void* stream);

const char* nvfp4_status_string(nvfp4_status s);
int nvfp4_last_hip_error(void);

#ifdef __cplusplus
}
#endif
#endif /* NVFP4_H */
