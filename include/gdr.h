/*
 * gdr.h -- C ABI of libgdr: the gated delta rule on AMD Instinct MI355X (gfx950).
 *
 * The method.  For each sequence and head a state S (dv rows x dk columns,
 * fp32, dk contiguous) evolves token by token as
 *
 *     S_t = alpha_t * S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T
 *     o_t = S_t q_t                      (the state after the update)
 *     alpha_t = exp(g_t)
 *
 * (the gated delta rule of GDN-style linear attention).  Two forms are
 * provided: a one-token decode step that updates the state in place, and a
 * chunked ("CP", chunk-parallel) prefill over packed variable-length
 * sequences.  The chunked form follows the structure described on the
 * FlashInfer PR #3866 page ("CP delta-rule precompute optimisation for
 * ultra-low parallelism"): every chunk c gets a local state L_c and a
 * transfer matrix M_c in parallel, then a sequential fixup
 *     fixed[c] = fixed[c-1] * M_c + L_c
 * produces the state at the end of each chunk (section "code changes 2",
 * accumulate_state_fragment: the state multiplies M from the left;
 * init_state_tile: with an initial state the scan starts at chunk 0, without
 * one the first fixed state is L_0 and the scan starts at chunk 1), and the
 * outputs of chunk c are computed from fixed[c-1].
 *
 * Conventions shared by every entry point:
 *   - All tensor pointers are DEVICE pointers, owned by the caller, dense
 *     row-major (C order), 16-byte aligned.  The library never allocates,
 *     frees or synchronises; work is enqueued on `stream` (a hipStream_t,
 *     NULL = the default stream) and buffers must stay alive until the stream
 *     has passed the call.  No call reads a host copy of device data, so every
 *     call may be captured in a HIP graph.
 *   - Validation happens on the host before any launch.  A failing check
 *     returns GDR_ERR_INVALID_ARG or GDR_ERR_UNSUPPORTED, launches nothing and
 *     writes nothing; gdr_last_error() then holds a message (per thread).
 *     A failed launch returns GDR_ERR_HIP.  No C++ exception crosses the ABI.
 *   - Device-side integer inputs (cu_seqlens, chunk_offsets) are not
 *     inspected on the host (that would need a synchronisation).  They must be
 *     non-decreasing, start at 0 and end at T_total (resp. the chunk count);
 *     kernels clamp every index they derive from them to the buffer sizes
 *     given, so bad values give wrong results but no out-of-bounds access.
 *   - Supported shapes of the gated delta rule: (dk, dv) in {(64, 64),
 *     (128, 128)}; chunk in {16, 64}.
 *   - Dtypes: q, k, v are bf16 or fp32 (in_dtype); o is bf16 or fp32
 *     (out_dtype; bf16 is round-to-nearest-even of the fp32 result).  g, beta,
 *     states, L, M and fixed states are always fp32.
 *   - Calls are thread-safe.  The only global state is a per-device property
 *     cache filled on first use.
 */
#ifndef GDR_H_
#define GDR_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  GDR_OK = 0,
  GDR_ERR_INVALID_ARG = 1, /* NULL pointer, misalignment, bad size */
  GDR_ERR_UNSUPPORTED = 2, /* shape or dtype outside the supported set */
  GDR_ERR_HIP = 3          /* a HIP runtime call or launch failed */
} gdr_status;

typedef enum { GDR_BF16 = 0, GDR_FP32 = 1 } gdr_dtype;

/* hipStream_t, kept opaque so that this header needs no HIP headers. */
typedef void* gdr_stream_t;

/*
 * gdr_decode_step -- one token of the recurrence for N independent
 * (sequence, head) states, updated IN PLACE.
 *
 * The decode step is the recurrence above with T = 1.  Its kernel streams
 * each fp32 state row straight from HBM into registers with 16-byte loads and
 * back, with no LDS staging: the state has no reuse (the FlashInfer PR #7156
 * page, "Cake GDP kernel optimisation: less shared memory, direct register
 * loads", code analysis 1, describes the same change for a split-V T=1 step).
 *
 *   q, k      [N, H, dk]      in_dtype
 *   v         [N, H, dv]      in_dtype
 *   g, beta   [N, H]          fp32; alpha = exp(g); g and beta are used as
 *                             given (no clamping)
 *   state     [N, H, dv, dk]  fp32, read and overwritten with S_t
 *   o         [N, H, dv]      out_dtype, o = S_t q
 *   N, H      > 0
 * q, k, v, g, beta and o must not overlap `state`.
 */
gdr_status gdr_decode_step(const void* q, const void* k, const void* v,
                           const float* g, const float* beta,
                           float* state, void* o,
                           int N, int H, int dk, int dv,
                           gdr_dtype in_dtype, gdr_dtype out_dtype,
                           gdr_stream_t stream);

/*
 * gdr_decode_mtp -- T decode tokens for each of N x H (sequence, head) states
 * (multi-token decode, e.g. verifying T draft tokens).
 *
 * The FlashInfer PR #7156 page ("Cake GDP kernel optimisation: less shared
 * memory, direct register loads", introduction) optimises the T = 1 variant of
 * a multi-token ("MTP") decode kernel; this entry point is the general T.
 * Token t of sequence n applies the recurrence to the state after token t-1
 * (state_in for t = 0), and its output uses the updated state.  The result is
 * that of gdr_chunk_prefill over N packed sequences of T tokens, and T = 1 is
 * gdr_decode_step (bit for bit).  The state is read once and written once
 * whatever T is.  Without `inter`, T >= 2 tokens are applied in chunks of 8
 * (the last may be shorter) of the chunked form on the matrix cores, other T
 * token by token; the two agree to rounding (1e-3 for bf16 inputs, 1e-5 for
 * fp32 inputs, against the token-by-token recurrence), and each is
 * deterministic.
 *
 *   q, k       [N, T, H, dk]     in_dtype (row n*T + t is token t of sequence n)
 *   v          [N, T, H, dv]     in_dtype
 *   g, beta    [N, T, H]         fp32; alpha = exp(g), used as given
 *   state_in   [N, H, dv, dk]    fp32 input states
 *   state_out  [N, H, dv, dk]    fp32 final states; may equal state_in (updated
 *                                in place); NULL: no final state is written
 *   o          [N, T, H, dv]     out_dtype
 *   inter      [N, T, H, dv, dk] fp32 or NULL: the state after every token
 *                                (inter[n][T-1] is the final state), e.g. to
 *                                restart from the last accepted draft token
 *   N, H > 0; 1 <= T <= 64
 * q, k, v, g, beta, o and inter must not overlap state_in or state_out.
 */
gdr_status gdr_decode_mtp(const void* q, const void* k, const void* v,
                          const float* g, const float* beta,
                          const float* state_in, float* state_out, void* o,
                          float* inter, int N, int T, int H, int dk, int dv,
                          gdr_dtype in_dtype, gdr_dtype out_dtype,
                          gdr_stream_t stream);

/*
 * gdr_max_chunks -- host-only upper bound on the number of chunks of a packed
 * batch of N sequences with T_total tokens: T_total / chunk + N (every
 * sequence adds at most one partial chunk).  Returns -1 on bad arguments.
 * Chunk-indexed buffers (L, M, fixed, chunk_indices) hold this many slots.
 */
int gdr_max_chunks(int T_total, int N, int chunk);

/*
 * gdr_chunk_layout -- varlen chunk layout, device to device (bit-exact).
 *
 *   cu_seqlens     [N+1] int32   token offsets of the packed sequences
 *   chunk_offsets  [N+1] int32   out: chunk_offsets[0] = 0,
 *                  chunk_offsets[n+1] = chunk_offsets[n] + ceil(len_n / chunk)
 *   chunk_indices  [max_chunks, 2] int32  out: row chunk_offsets[n] + j holds
 *                  (n, j); rows past the real chunk count hold (-1, -1)
 *   max_chunks     rows of chunk_indices (>= gdr_max_chunks(T_total, N, chunk))
 * Chunk j of sequence n covers tokens [cu[n] + j*chunk, min(cu[n] + (j+1)*chunk, cu[n+1])).
 * Chunks never straddle a sequence boundary (the FlashInfer PR #3866 page
 * handles variable-length batches with per-sequence chunk counts and zeroes
 * the slots past a sequence's valid chunks, zero_invalid_slots; here chunks
 * are packed, so there are no invalid slots inside the range).
 */
gdr_status gdr_chunk_layout(const int32_t* cu_seqlens, int N, int chunk,
                            int32_t* chunk_offsets, int32_t* chunk_indices,
                            int max_chunks, gdr_stream_t stream);

/*
 * gdr_chunk_prefill_workspace_bytes -- device workspace that gdr_chunk_prefill
 * needs for inputs of in_dtype when L_out, M_out and fixed_out are all NULL,
 * for whichever schedule the call takes (an upper bound for every other case).
 * Returns 0 on bad arguments (also for a shape or dtype gdr_chunk_prefill
 * refuses).
 */
size_t gdr_chunk_prefill_workspace_bytes(int T_total, int N, int H, int dk, int dv,
                                         int chunk, gdr_dtype in_dtype);

/*
 * gdr_chunk_prefill -- chunked prefill over packed variable-length sequences.
 *
 *   q, k        [T_total, H, dk]  in_dtype
 *   v           [T_total, H, dv]  in_dtype
 *   g, beta     [T_total, H]      fp32
 *   cu_seqlens  [N+1] int32       device; sequence n is tokens [cu[n], cu[n+1])
 *   state_in    [N, H, dv, dk]    fp32 initial states, or NULL for zero states
 *   state_out   [N, H, dv, dk]    fp32 final states (may equal state_in)
 *   o           [T_total, H, dv]  out_dtype
 *   L_out       [max_chunks, H, dv, dk] fp32 or NULL: local state of every chunk
 *               (the chunk run from a zero state): L_out[c][h][i][j] = L_c[i][j]
 *   M_out       [max_chunks, H, dk, dk] fp32 or NULL: transfer matrix of every
 *               chunk, M_out[c][h][a][b] = M_c[a][b], in the orientation of
 *               the recurrence: S_end = S_start M_c + L_c, i.e.
 *               S_end[i][b] = sum_a S_start[i][a] M_c[a][b] + L_c[i][b]
 *               (M_c = gamma_c I - W^T diag(D) K, the product of the chunk's
 *               per-token maps alpha_t (I - beta_t k_t k_t^T) in token order)
 *   fixed_out   [max_chunks, H, dv, dk] fp32 or NULL: state at the end of every
 *               chunk
 *   (max_chunks = gdr_max_chunks(T_total, N, chunk); chunk slot
 *    chunk_offsets[n] + j belongs to chunk j of sequence n; slots past the real
 *    chunk count are not written)
 *   T_total >= 0, N > 0, H > 0; chunk in {16, 64}; in_dtype bf16 or fp32 at
 *   either chunk size
 *   workspace   device scratch of workspace_bytes bytes (see
 *               gdr_chunk_prefill_workspace_bytes); may be NULL only when the
 *               bound is 0; its contents on entry do not matter
 * Sequences of length 0 are allowed: their final state is the initial state
 * (or zero).  q, k, v, g, beta and o must not overlap each other or the
 * state/L/M/fixed buffers.  All work is enqueued on `stream`, in one of the
 * following schedules, with the same results up to rounding order:
 *   - chunk-parallel: layout, chunk-local L/M, fixup over the chunks of each
 *     sequence (two-level for long sequences with few heads), chunk outputs,
 *     final states.  Taken for fp32 inputs or chunk 16 (fp32 inputs keep
 *     every product at fp32 precision);
 *   - sequential scan: layout, per-chunk factors T = (I + A)^{-1} and
 *     P = (Q K^T) (.) Gamma, then one pass per (sequence, head, block of state
 *     rows) that applies the UT transform and the fixup in factored form
 *     (S M_c + L_c = gamma_C S + (diag(D) T diag(beta) (V - diag(gamma) K S^T))^T K,
 *     without forming M, L, W or Ut) and writes the outputs, the final states
 *     and, when given, fixed_out.  Taken for bf16 inputs at chunk 64; for long
 *     sequences at low parallelism as a segmented scan: one pass over
 *     segments of whole chunks carrying two chains per segment, from zero
 *     (segment local states) and from the identity with v = 0 (segment
 *     transfer matrices), the segment-level fixup, and a final pass from every
 *     segment's true start.  When L_out or
 *     M_out is given, the chunk-local kernel of the chunk-parallel form writes
 *     them in parallel, before the scan.  The scan holds T and P as one fp16
 *     plane each (scaled by 16), and beta (V - diag(gamma) K S^T) / 16 and
 *     U / 16 as two fp16 planes each: entries of beta (v - gamma S k) or of U
 *     beyond about 1e6 in magnitude overflow to non-finite results (keys are
 *     expected L2-normalised, as the method assumes).
 */
gdr_status gdr_chunk_prefill(const void* q, const void* k, const void* v,
                             const float* g, const float* beta,
                             const int32_t* cu_seqlens, int N,
                             const float* state_in, float* state_out, void* o,
                             float* L_out, float* M_out, float* fixed_out,
                             int T_total, int H, int dk, int dv, int chunk,
                             gdr_dtype in_dtype, gdr_dtype out_dtype,
                             void* workspace, size_t workspace_bytes,
                             gdr_stream_t stream);

/*
 * gdr_chunk_prefill_noalloc -- gdr_chunk_prefill without a workspace, for
 * callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc).
 *
 * Arguments, layouts, schedules and results are those of gdr_chunk_prefill
 * (bit for bit: the same kernels run), minus workspace and workspace_bytes.
 * The workspace is instead a static device array of the library, 128 MiB
 * (134,217,728 bytes) on each GPU it runs on, held from the first call on that
 * GPU until the process ends.  A call that needs more than that (see
 * gdr_chunk_prefill_workspace_bytes; e.g. 4 sequences x 4096 tokens x 16 heads
 * at d = 128 needs about 55 MB) returns GDR_ERR_UNSUPPORTED with a message
 * and launches nothing.  Nothing is allocated or freed, here or on later
 * calls.  All calls on one GPU share its array, which keeps the last call's
 * contents (no call depends on them): calls that may overlap on one GPU, from
 * two streams or two threads, race and must be serialised by the caller.
 */
gdr_status gdr_chunk_prefill_noalloc(const void* q, const void* k, const void* v,
                                     const float* g, const float* beta,
                                     const int32_t* cu_seqlens, int N,
                                     const float* state_in, float* state_out, void* o,
                                     float* L_out, float* M_out, float* fixed_out,
                                     int T_total, int H, int dk, int dv, int chunk,
                                     gdr_dtype in_dtype, gdr_dtype out_dtype,
                                     gdr_stream_t stream);

/*
 * gdr_state_fixup -- the inter-chunk fixup alone.
 *
 *   L             [n_chunks, H, dv, dk] fp32 local states, L[c][h][i][j] = L_c[i][j]
 *   M             [n_chunks, H, dk, dk] fp32 transfer matrices in the
 *                 orientation of the recurrence, M[c][h][a][b] = M_c[a][b]
 *                 (the same layout as gdr_chunk_prefill's M_out)
 *   state_in      [N, H, dv, dk] fp32, or NULL (no initial state)
 *   chunk_offsets [N+1] int32 device: sequence n owns chunk slots
 *                 [chunk_offsets[n], chunk_offsets[n+1])
 *   fixed         [n_chunks, H, dv, dk] fp32 out:
 *                 fixed[c0] = state_in[n] M_c0 + L_c0   (c0 = first chunk of n)
 *                           = L_c0                      (state_in == NULL)
 *                 fixed[c]  = fixed[c-1] M_c + L_c      (later chunks of n)
 *   n_chunks      slots in L, M and fixed; chunk ids at or past it are ignored
 * The FlashInfer PR #3866 page ("CP delta-rule precompute optimisation for
 * ultra-low parallelism", code changes 2) describes this scan: the state
 * multiplies M_c from the left, and without an initial state the first chunk's
 * state is its local state.  Here it runs one workgroup per (sequence, head,
 * block of state rows) on the matrix cores with the state and M_c split into
 * three bf16 planes each (fp32 precision), and loads chunk c+1's M and L while
 * chunk c is multiplied.  fixed must not overlap L, M or state_in.
 */
gdr_status gdr_state_fixup(const float* L, const float* M, const float* state_in,
                           const int32_t* chunk_offsets, int N, float* fixed,
                           int n_chunks, int H, int dk, int dv, gdr_stream_t stream);

/*
 * Linear attention with a decay for each head -- the recurrence of retention
 * and of scalar-gate state-space layers, the gated delta rule without its
 * delta term:
 *
 *     S_t = alpha_t * S_{t-1} + v_t k_t^T,   o_t = scale * S_t q_t
 *     alpha_t = exp(g)
 *
 * g is one value for each token and head (GDR_DECAY_TOKEN) or one for each
 * head (GDR_DECAY_HEAD, the same at every token).  g <= 0 is expected, and g
 * below -110, -inf among it, counts as -110: a decay of exactly zero in fp32.
 * Value head h reads query and key head h / (H / Hk), with H a multiple of Hk.
 *
 * Beyond the conventions above, for gdr_linear_*:
 *   - (dk, dv) may be any of {64, 128} x {64, 128}.
 *   - q, k and v may be slices of wider token rows: q_stride, k_stride and
 *     v_stride are the elements from one token's row to the next, 0 for dense
 *     ([T, heads, d] contiguous).  The heads of one token are always
 *     contiguous, and a stride is a multiple of 16 bytes, not below the heads'
 *     width and at most 2^24 elements.
 *   - cu_seqlens[N] may be below T_total: rows behind the last sequence are
 *     neither read nor written.
 *   - N <= 65536, H <= 65535, N * H <= 4000000 and T_total * H < 2^31.
 *   - An infinity or NaN in a token's q, k or v may make the outputs of its
 *     own chunk of 64 tokens non-finite as well as those after it; other
 *     sequences are not affected.
 *   - Every result is deterministic: no atomics.
 *   - Calls that may run at the same time need workspaces of their own.
 *   - Long sequences are cut into segments that run side by side, by the average
 *     length of the batch: one sequence far longer than four times that average is
 *     walked as a whole, and is faster in a call of its own.
 */
typedef enum { GDR_DECAY_TOKEN = 0, GDR_DECAY_HEAD = 1 } gdr_decay;

/*
 * gdr_linear_decode -- one token for N x H states, updated IN PLACE.
 *
 *   q, k      [N, Hk, dk]     in_dtype, rows q_stride / k_stride apart
 *   v         [N, H, dv]      in_dtype, rows v_stride apart
 *   g         [N, H] or [H]   fp32, by `decay`
 *   state     [N, H, dv, dk]  fp32, read and overwritten with S_t
 *   o         [N, H, dv]      out_dtype
 *   N, H, Hk  > 0, H % Hk == 0
 * No tensor may overlap `state`.
 */
gdr_status gdr_linear_decode(const void* q, const void* k, const void* v, const float* g,
                             float* state, void* o, int N, int H, int Hk, int dk, int dv,
                             int64_t q_stride, int64_t k_stride, int64_t v_stride, float scale,
                             gdr_decay decay, gdr_dtype in_dtype, gdr_dtype out_dtype,
                             gdr_stream_t stream);

/*
 * gdr_linear_prefill -- prompts: packed variable-length sequences.
 *
 *   q, k        [T_total, Hk, dk]  in_dtype, rows q_stride / k_stride apart
 *   v           [T_total, H, dv]   in_dtype, rows v_stride apart
 *   g           [T_total, H] or [H] fp32, by `decay`
 *   cu_seqlens  [N+1] int32        device; sequence n is tokens [cu[n], cu[n+1])
 *   state_in    [N, H, dv, dk]     fp32, or NULL for zero states
 *   state_out   [N, H, dv, dk]     fp32 final states; may equal state_in; NULL:
 *                                  not written.  A sequence of length 0 passes
 *                                  its initial state on
 *   o           [T_total, H, dv]   out_dtype
 *   workspace   gdr_linear_prefill_workspace_bytes(...) bytes of device scratch
 *               (NULL when that is 0); its contents do not matter
 * o must not overlap any input.
 */
gdr_status gdr_linear_prefill(const void* q, const void* k, const void* v, const float* g,
                              const int32_t* cu_seqlens, int N, const float* state_in,
                              float* state_out, void* o, int T_total, int H, int Hk, int dk,
                              int dv, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                              float scale, gdr_decay decay, gdr_dtype in_dtype,
                              gdr_dtype out_dtype, void* workspace, size_t workspace_bytes,
                              gdr_stream_t stream);

/* Device workspace of gdr_linear_prefill; 0 also on bad arguments. */
size_t gdr_linear_prefill_workspace_bytes(int T_total, int N, int H, int dk, int dv,
                                          gdr_dtype in_dtype);

/*
 * gdr_linear_backward -- gradients of gdr_linear_prefill.  With d_o the
 * gradient of o and dstate_out that of state_out, and R_t the gradient of S_t,
 *     R_t  = scale d_o_t q_t^T + alpha_{t+1} R_{t+1}
 *     dq_t = scale S_t^T d_o_t,  dk_t = R_t^T v_t,  dv_t = R_t k_t
 *     dg_t = alpha_t <R_t, S_{t-1}>,  dstate_in = alpha_1 R_1
 *
 *   q, k, v, g, cu_seqlens, state_in   as given to gdr_linear_prefill
 *   d_o          [T_total, H, dv]   in_dtype, dense
 *   dstate_out   [N, H, dv, dk]     fp32, or NULL for zero
 *   dq, dk_out   [T_total, Hk, dk]  grad_dtype: summed over the value heads that
 *                                   share the head, in fp32
 *   dv_out       [T_total, H, dv]   grad_dtype
 *   dg           fp32, the shape of g, or NULL.  For GDR_DECAY_HEAD the sum over
 *                all tokens.  Where g is below -110 the gradient is that of a
 *                decay of zero: 0.  dg is formed by sums over the tokens behind, so
 *                that its error is relative to the largest values of its
 *                sequence and head (about 1e-6 of them), not to its own: at a nearly
 *                closed gate (g of -15, say) between open ones, whose true gradient
 *                is far smaller than that, dg is rounding
 *   dstate_in    [N, H, dv, dk]     fp32, or NULL
 *   workspace    gdr_linear_backward_workspace_bytes(...) bytes
 * Where heads are shared (H above Hk), T_total * Hk * dk is at most 2^34 - 1024.
 * No output may overlap an input or another output (dstate_in not dstate_out).
 */
gdr_status gdr_linear_backward(const void* q, const void* k, const void* v, const float* g,
                               const int32_t* cu_seqlens, int N, const float* state_in,
                               const void* d_o, const float* dstate_out, void* dq, void* dk_out,
                               void* dv_out, float* dg, float* dstate_in, int T_total, int H,
                               int Hk, int dk, int dv, int64_t q_stride, int64_t k_stride,
                               int64_t v_stride, float scale, gdr_decay decay,
                               gdr_dtype in_dtype, gdr_dtype grad_dtype, void* workspace,
                               size_t workspace_bytes, gdr_stream_t stream);

/* Device workspace of gdr_linear_backward; 0 also on bad arguments. */
size_t gdr_linear_backward_workspace_bytes(int T_total, int N, int H, int Hk, int dk, int dv,
                                           gdr_dtype in_dtype);

/*
 * gdr_block_norm -- the norms around a block, fused with its gate and its
 * scaled residual.  Per row of D values, with rms(a) = sqrt(mean(a^2) + eps):
 *
 *     u = x / rms(x) * w_after            (x itself without w_after)
 *     u = u * act(gate)                   (where gate is given)
 *     h = residual + scale * u            (scale * u without residual)
 *     y = h / rms(h) * w_before           (where w_before is given)
 *
 * w_after is the norm after the block that produced x (for the outputs o of
 * the recurrences: rows = tokens * heads, D = dv), w_before the norm before
 * the next block.  All arithmetic is fp32 and y comes from the unrounded h.
 * A row of zeros gives zeros (eps > 0 keeps rms above zero; eps = 0 is the
 * caller's choice).
 *
 *   x, gate, residual  [rows, D]   in_dtype; gate and residual may be NULL
 *   w_after, w_before  [D]         w_dtype; may be NULL
 *   h, y               [rows, D]   out_dtype; h may be NULL where y is given;
 *                                  y is given exactly when w_before is.  h or y
 *                                  may be the buffer of x, gate or residual when
 *                                  the dtypes agree (not both the same one)
 *   act                GDR_GATE_SILU: z sigmoid(z), GDR_GATE_SIGMOID: sigmoid(z)
 *   1 <= D <= 16384, 0 <= rows <= 2^28, rows * D < 2^33
 * For D a multiple of 8 every row is read with 16-byte loads; other D take
 * single-element accesses.
 */
typedef enum { GDR_GATE_SILU = 0, GDR_GATE_SIGMOID = 1 } gdr_gate;

gdr_status gdr_block_norm(const void* x, const void* w_after, const void* gate,
                          const void* residual, const void* w_before, void* h, void* y,
                          int64_t rows, int D, float scale, float eps, gdr_gate act,
                          gdr_dtype in_dtype, gdr_dtype w_dtype, gdr_dtype out_dtype,
                          gdr_stream_t stream);

/*
 * gdr_block_norm_backward -- gradients of gdr_block_norm.
 *
 *   x, w_after, gate, residual, w_before   as given to gdr_block_norm (residual
 *                is read only with w_before, where h is formed again)
 *   dh           [rows, D]  in_dtype: gradient of h, or NULL for zero
 *   dy           [rows, D]  in_dtype: gradient of y, given exactly when w_before is
 *   dx           [rows, D]  out_dtype
 *   dgate        [rows, D]  out_dtype; NULL: not written
 *   dresidual    [rows, D]  out_dtype; NULL: not written
 *   dw_after, dw_before  [D] fp32, sums over all rows; NULL: not written
 *   workspace    gdr_block_norm_backward_workspace_bytes(rows, D) bytes (needed
 *                only when a dw is asked for): the sums of single workgroups,
 *                added in a fixed order by a second kernel (deterministic)
 * No output may overlap an input or another output.
 */
gdr_status gdr_block_norm_backward(const void* x, const void* w_after, const void* gate,
                                   const void* residual, const void* w_before, const void* dh,
                                   const void* dy, void* dx, void* dgate, void* dresidual,
                                   float* dw_after, float* dw_before, int64_t rows, int D,
                                   float scale, float eps, gdr_gate act, gdr_dtype in_dtype,
                                   gdr_dtype w_dtype, gdr_dtype out_dtype, void* workspace,
                                   size_t workspace_bytes, gdr_stream_t stream);

/* Device workspace of gdr_block_norm_backward; 0 also on bad arguments. */
size_t gdr_block_norm_backward_workspace_bytes(int64_t rows, int D);

/*
 * gdr_block_norm8 -- gdr_block_norm with its result in 8 bits, for the product
 * that follows (gdr_product8).  y (with w_before) or h (without) leaves as e4m3
 * (OCP, torch.float8_e4m3fn) with one fp32 scale for each 128 consecutive values
 * of a row, the last block of a row being shorter where D is no multiple of 128:
 *
 *     y_scale = max|y| / 448,  y8 = e4m3(y / y_scale)   (round to nearest even)
 *
 * from the unrounded fp32 values, the quotient as a product with 448 / max|y|: a value
 * within 2^-22 of the middle between two e4m3 numbers may become either.  A block whose values are all below 2^-100 in
 * magnitude, zeros among them, is stored as zeros with a scale of 0.  A NaN stays
 * a NaN in its place; an infinity makes its block's scale infinite and itself a
 * NaN, so that none of the block reads as a finite number.
 *
 *   x, w_after, gate, residual, w_before, act   as gdr_block_norm's
 *   h         [rows, D]              out_dtype, or NULL: not written.  May be the
 *                                    buffer of x, gate or residual when the dtypes
 *                                    agree
 *   y8        [rows, D]              e4m3
 *   y_scale   [rows, ceil(D / 128)]  fp32
 *   D a multiple of 16, otherwise the limits of gdr_block_norm.  y8 and y_scale
 *   must not overlap anything else.
 */
gdr_status gdr_block_norm8(const void* x, const void* w_after, const void* gate,
                           const void* residual, const void* w_before, void* h, void* y8,
                           float* y_scale, int64_t rows, int D, float scale, float eps,
                           gdr_gate act, gdr_dtype in_dtype, gdr_dtype w_dtype,
                           gdr_dtype out_dtype, gdr_stream_t stream);

/*
 * gdr_product8 -- the product of rows in 8 bits with weights in 8 bits:
 *
 *     out[m][n] = sum_b a_scale[m][b] w_scale[n / 128][b] sum_{k in block b} a[m][k] w[n][k]
 *
 * over blocks b of 128 consecutive k.  With fp32 results products are exact and every sum
 * is fp32.  With bf16 results the matrix cores' 8-bit instruction forms a block's sum: it
 * keeps the products of 8 consecutive k as multiples of 2^-13 of the largest one's power of
 * two and adds the rest in fp32.  What that loses is below 7 2^-13 of the sum of the products'
 * absolute values, 1.5e-5 of it for normal data; sums that cancel feel it more, and are what
 * fp32 results are for.
 *
 * There is no gradient entry.  That of a is this product with w transposed and laid out in
 * blocks of 128 x 128 again; that of w sums over rows, for which nothing here makes 8 bits.
 *
 *   a        [M, K]                           e4m3, as gdr_block_norm8 writes it
 *   a_scale  [M, ceil(K / 128)]               fp32
 *   w        [N, K]                           e4m3
 *   w_scale  [ceil(N / 128), ceil(K / 128)]   fp32: one for each 128 x 128 of w
 *   out      [M, N]                           out_dtype
 *   M >= 0, N > 0, K > 0 a multiple of 16; M, N <= 2^24, K <= 2^22, M * N < 2^36
 * A row of a, or of w, touches its own row, or column, of out only, NaN and
 * infinite scales among them.  The two scales of a block are multiplied first: their
 * product has to be a number that fp32 holds.  out must not overlap an input.
 * Deterministic.
 */
gdr_status gdr_product8(const void* a, const float* a_scale, const void* w, const float* w_scale,
                        void* out, int M, int N, int K, gdr_dtype out_dtype, gdr_stream_t stream);

/* Most rows M that gdr_product8 takes with N columns; 0 on a bad N. */
int gdr_product8_max_rows(int N);

/*
 * The gated linear recurrence with a decay for each channel -- a recurrence whose
 * state is a vector (gated recurrent units without a nonlinearity in time, the
 * recurrent layers of hybrid models).  Per sequence and channel
 *
 *     h_t = a_t h_{t-1} + b_t
 *     a_t = exp(g_t) (GDR_CHANNEL_LOG) or sigmoid(g_t) (GDR_CHANNEL_LOGIT)
 *     b_t = x_t, or (1 - a_t) x_t with `complement`
 *
 * Conventions of gdr_channel_*, beyond those above:
 *   - x, g, h and their gradients are rows of D channels, any D from 1 to 2^20.
 *     x, h, dh and dx share io_dtype, g and dg have g_dtype.  States are fp32.
 *   - x and g may be slices of wider token rows: x_stride and g_stride are the
 *     elements from one row to the next, 0 for dense, at least D and at most 2^24.
 *     Rows are fastest where D and both strides are multiples of 8 (of 4 with
 *     io_dtype GDR_FP32).
 *   - g <= 0 is expected of GDR_CHANNEL_LOG (a decay); -110 or less, -infinity among
 *     it, is a decay of exactly zero.  1 - a is formed without cancellation.
 *   - cu_seqlens[N] may be below T_total: rows behind the last sequence are not
 *     written, and what they hold does not matter.
 *   - N <= 2^20, N * D < 2^31, and T_total and D such that a launch holds them:
 *     T_total / 64 + 1 times D / 64 + 1 below 2^24.
 *   - An infinity or NaN in x or g spreads to later tokens of its own sequence and
 *     channel (earlier ones in the gradient), and nowhere else.
 *   - Every result is deterministic: sums are formed in one order, whatever the
 *     order in which workgroups run.
 *   - Calls that may run at the same time need workspaces of their own, two captured
 *     graphs among them: a workspace holds what workgroups of one call tell each other.
 */
typedef enum { GDR_CHANNEL_LOG = 0, GDR_CHANNEL_LOGIT = 1 } gdr_channel_gate;

/*
 * gdr_channel_decode -- one token of N sequences, state updated IN PLACE.
 *
 *   x, g    [N, D]   rows x_stride / g_stride apart
 *   state   [N, D]   fp32, read and overwritten with h_t
 *   h       [N, D]   io_dtype; may be x's buffer where x is dense
 */
gdr_status gdr_channel_decode(const void* x, const void* g, float* state, void* h, int N, int D,
                              int64_t x_stride, int64_t g_stride, gdr_channel_gate gate,
                              int complement, gdr_dtype io_dtype, gdr_dtype g_dtype,
                              gdr_stream_t stream);

/*
 * gdr_channel_prefill -- prompts: packed variable-length sequences.
 *
 *   x, g        [T_total, D]   rows x_stride / g_stride apart
 *   cu_seqlens  [N+1] int32    device; sequence n is tokens [cu[n], cu[n+1])
 *   state_in    [N, D] fp32, or NULL for zero states
 *   state_out   [N, D] fp32 final states; may equal state_in; NULL: not written.
 *               A sequence of length 0 passes its initial state on
 *   h           [T_total, D]   io_dtype; may be x's buffer where x is dense
 *   workspace   gdr_channel_prefill_workspace_bytes(...) bytes of device scratch
 *               (NULL when that is 0); its contents do not matter
 * No other overlap of outputs with inputs or each other.
 */
gdr_status gdr_channel_prefill(const void* x, const void* g, const int32_t* cu_seqlens, int N,
                               const float* state_in, float* state_out, void* h, int T_total,
                               int D, int64_t x_stride, int64_t g_stride, gdr_channel_gate gate,
                               int complement, gdr_dtype io_dtype, gdr_dtype g_dtype,
                               void* workspace, size_t workspace_bytes, gdr_stream_t stream);

/* Device workspace of gdr_channel_prefill; 0 also on bad arguments. */
size_t gdr_channel_prefill_workspace_bytes(int T_total, int D);

/*
 * gdr_channel_backward -- gradients of gdr_channel_prefill.  With r_t the gradient
 * of h_t, from h's own and from later tokens,
 *     r_t  = dh_t + a_{t+1} r_{t+1}       (dstate_out for the one after the last)
 *     dx_t = r_t, or (1 - a_t) r_t with `complement`
 *     dg_t = a' r_t (h_{t-1} [- x_t with `complement`]),  a' = a, or a (1 - a) of logits
 *     dstate_in = a_1 r_1
 *
 *   x, g, cu_seqlens, state_in   as given to gdr_channel_prefill (x is read with
 *               `complement` only, and may be NULL without)
 *   h           [T_total, D]   io_dtype, as gdr_channel_prefill wrote it: dg takes
 *               h_{t-1} from it, so that its relative error is that of h's rounding
 *   dh          [T_total, D]   io_dtype
 *   dstate_out  [N, D] fp32, or NULL for zero
 *   dx, dg      [T_total, D]   io_dtype and g_dtype, dense
 *   dstate_in   [N, D] fp32, or NULL: not written
 *   workspace   gdr_channel_backward_workspace_bytes(...) bytes
 * No output may overlap an input or another output.
 */
gdr_status gdr_channel_backward(const void* x, const void* g, const void* h,
                                const int32_t* cu_seqlens, int N, const float* state_in,
                                const void* dh, const float* dstate_out, void* dx, void* dg,
                                float* dstate_in, int T_total, int D, int64_t x_stride,
                                int64_t g_stride, gdr_channel_gate gate, int complement,
                                gdr_dtype io_dtype, gdr_dtype g_dtype, void* workspace,
                                size_t workspace_bytes, gdr_stream_t stream);

/* Device workspace of gdr_channel_backward; 0 also on bad arguments. */
size_t gdr_channel_backward_workspace_bytes(int T_total, int D);

/* Static text for a status code. */
const char* gdr_status_string(gdr_status s);

/* Detail of the last failure on the calling thread ("" if none). */
const char* gdr_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* GDR_H_ */
