/*
 * ssd_diag.h -- C ABI of libssd's diagonal selective scan and of what serves
 * it: state maps built on the device from request lengths, the short causal
 * convolution over packed requests and its gradient, the scan in dense,
 * packed and backward form, and the single-token state update.
 *
 * The recurrence is that of ssd.h ("Hybrid Architectures for Language
 * Models", summary page, section 2 Background: h_t = Abar h_{t-1} + Bbar x_t,
 * y_t = C h_t + D x_t) with a decay of its own for every channel and state
 * element, where ssd.h's chunked scan has one per head:
 *
 *   dt[t][e]   = softplus(dt_raw[t][e] + dt_bias[e])
 *   h_t[e][n]  = exp(dt[t][e] A[e][n]) h_{t-1}[e][n] + dt[t][e] u[t][e] B[t][g][n]
 *   y[t][e]    = (sum_n h_t[e][n] C[t][g][n] + D[e] u[t][e]) * SiLU(z[t][e])
 *
 * Notation: E channels, N state elements per channel, G groups of B/C
 * (channel e reads group g = e / (E / G)), T packed tokens, k conv width.
 *
 * Row counts (b * L; T and nseq together) are at most 2^31 - 65537, else
 * SSD_ERR_UNSUPPORTED.
 *
 * The conventions are those of ssd.h (caller-owned device memory, no
 * allocation, no synchronisation, no global state, work enqueued on
 * `stream`, return values), with these shared by the calls below:
 *   - u, dt_raw, z, y, dy, conv rows and their gradients have the element
 *     type `dtype`, rows of E adjacent elements at a row stride of their own
 *     (elements; a multiple of 8, at least E); E and E / G are multiples of
 *     8, pointers to rows 16-byte aligned.
 *   - B, C have the element type `dtype`, token t, group g, n at
 *     B[t*bc_stride + g*N + n]; any element-aligned pointer and any stride of
 *     at least G*N (they are usually columns of a projection's rows).
 *   - NaN in a row spoils what the formulas say and nothing else.  An
 *     infinite u, B or dt_raw may give NaN where they give an infinity.
 *   - A [E][N], D [E], dt_bias [E], conv weights (16-byte aligned, as A) and
 *     states are float32;
 *     sums, states and gradients accumulate in float32.  A is expected <= 0
 *     (-inf: a state that forgets at once).
 *   - N is a multiple of 4, at most 64 (else SSD_ERR_UNSUPPORTED above 64).
 *
 * Slots.  A serving loop keeps the requests' states (and conv caches) in a
 * pool of `nslots` slots, each one request's state after some token.  A
 * request of p tokens held has its tokens in blocks of `block_tokens`; block
 * j's slot, table[r][j], holds the state after token min(p, (j+1) *
 * block_tokens) - 1.  With blocks longer than any request, that is one slot
 * per request; with shorter ones every block's end leaves its state behind,
 * and a later request that begins with the same whole blocks starts from
 * there (its table names the same slots; whole blocks are only read).
 * ssd_state_map builds what the packed calls read:
 *   cu_seqlens [n+1] int32  request r's new tokens are rows cu[r] .. cu[r+1]-1
 *   seq_of     [T]   int32  the request of each row, -1 behind the last
 *   pos_of     [T]   int32  the row's place in its request, held tokens counted
 *   slot_of    [T]   int64  slot * block_tokens + place in the block, -1 behind
 *                           (also where a paged cache of per-token entries
 *                           has this token)
 *   init_slot  [n]   int32  the slot of the held tokens' state, -1 for none
 * The packed calls start sequence r from slot init_slot[r] (from zero where
 * that is -1) and write a state at every row that is the last of its block
 * or of its sequence, to the slot of its block.  Rows behind cu[nseq] are
 * not written (outputs there stay as they were) and no result depends on what
 * they hold; slots that no
 * row's block ends in stay as they were.  Maps that ssd_state_map made
 * without an error are sound.  For any other map, each call checks on the
 * device what memory safety needs (ranges of rows, sequences and slots),
 * leaves out the sequence or the slot concerned and sets *status to
 * SSD_ERR_INVALID_ARG; that no slot is written by two sequences of a call,
 * nor read by one and written by another, is then the caller's to ensure.
 */
#ifndef SSD_DIAG_H_
#define SSD_DIAG_H_

#include "ssd.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The map of a batch of requests, built on the device.
 *
 *   lens, ctx  [n] int32    new tokens of each request; tokens it holds
 *   table      [n][max_blocks] int32   block j < ceil(ctx/block_tokens) of
 *                           request r has slot table[r][j]; the rest is ignored.
 *                           The call reads the last of these (the state to start
 *                           from); entries before it are copied as they are, so
 *                           the slots of earlier states may be given back.
 *   free_list  [nfree] int32, free_head [1] int32   slots free_list[*free_head
 *                           ..] are unused; the call takes as many as the new
 *                           tokens open blocks, in the order of requests and blocks
 *   T          rows of the packed batch; sum(lens) <= T
 *   cu_seqlens .. init_slot as above, written
 *   table_out  [n][max_blocks], written: table with the new blocks' slots
 *   free_head_out [1], written: *free_head + slots taken
 *              (each may be its input, for an update in place)
 *   seq_of, pos_of and slot_of are 16-byte aligned
 *   workspace  ssd_state_map_workspace_bytes(n) bytes, no initial contents
 *   status     device int32, REQUIRED; the caller zeroes it before the call
 * Everything is checked on the device: lengths negative or beyond int32,
 * more than T tokens, a table too narrow, too few free slots, a slot outside
 * [0, nslots), a slot that two requests would write (the same unfinished
 * block twice, a free slot taken twice, a free slot that is also the state
 * that a request of the batch starts from), a slot that one would start from
 * while another writes it.  On any of these *status
 * is SSD_ERR_INVALID_ARG, the map is that of a batch without tokens
 * (cu_seqlens zero, the others -1), the table is copied unchanged and no
 * slot is taken.  n == 0 or T == 0 is allowed.  nslots is at most 1500000
 * (else SSD_ERR_UNSUPPORTED).
 */
SSD_API size_t ssd_state_map_workspace_bytes(int n);
SSD_API ssd_status_t ssd_state_map(const int32_t* lens, const int32_t* ctx, const int32_t* table,
                                   const int32_t* free_list, const int32_t* free_head, int n, int max_blocks,
                                   int nfree, int T, int block_tokens, int nslots, int32_t* cu_seqlens,
                                   int32_t* seq_of, int32_t* pos_of, int64_t* slot_of, int32_t* init_slot,
                                   int32_t* table_out, int32_t* free_head_out, void* workspace,
                                   size_t workspace_bytes, int32_t* status, cudaStream_t stream);

/*
 * ssd_conv1d_silu over packed requests, its caches in slots.
 *
 *   x      [T][.] dtype, row t's E channels at x[t*x_stride]; out likewise
 *          (must not overlap x)
 *   w [E][k], bias [E] (may be NULL)  float32
 *   cache  [nslots][E][k] dtype: column j of a slot holds the input k - j
 *          tokens before the slot's state ends (as ssd_conv1d_silu's cache)
 * The left context of a sequence is its init slot's cache (zero without
 * one).  Single tokens per request are the decode step's conv.
 * 2 <= k <= 4 (else SSD_ERR_UNSUPPORTED).  status REQUIRED.
 */
SSD_API ssd_status_t ssd_conv1d_silu_varlen(const void* x, int64_t x_stride, void* out, int64_t out_stride,
                                            const float* w, const float* bias, void* cache,
                                            const int32_t* cu_seqlens, const int32_t* seq_of,
                                            const int64_t* slot_of, const int32_t* init_slot, int nseq, int T,
                                            int E, int k, int block_tokens, int nslots, ssd_dtype_t dtype,
                                            int32_t* status, cudaStream_t stream);

/*
 * Gradients through ssd_conv1d_silu (a dense batch).
 *
 *   x [b][L][E], w [E][k], bias [E] or NULL, conv_state [b][E][k] dtype or
 *          NULL: the forward call's inputs (the cache as it was before)
 *   dout [b][L][E] dtype
 *   dx   [b][L][E] dtype, written
 *   dw [E][k], dbias [E] float32, written (dbias may be NULL: not wanted)
 *   dconv_state [b][E][k] dtype, written, may be NULL (not wanted)
 *   workspace  ssd_conv1d_silu_bwd_workspace_bytes(...) bytes
 * The rewritten cache holds copies of inputs; a gradient with respect to it
 * adds to dx's last rows and is the caller's.  Deterministic.  b == 0 or
 * L == 0 writes zeros to dw, dbias and dconv_state.
 */
SSD_API size_t ssd_conv1d_silu_bwd_workspace_bytes(int b, int L, int E, int k);
SSD_API ssd_status_t ssd_conv1d_silu_bwd(const void* x, const float* w, const float* bias, const void* conv_state,
                                         const void* dout, void* dx, float* dw, float* dbias, void* dconv_state,
                                         int b, int L, int E, int k, ssd_dtype_t dtype, void* workspace,
                                         size_t workspace_bytes, cudaStream_t stream);

/*
 * The diagonal scan of a dense batch.
 *
 *   u, dt_raw [b][L] rows at u_stride, dt_stride; z [b][L] rows at z_stride,
 *          or NULL (no gate); B, C [b][L] rows at bc_stride
 *   dt_bias, D [E] float32, may be NULL (zero)
 *   init_state [b][E][N] float32, may be NULL (zero)
 *   y      [b][L][E] dtype, written; must not overlap inputs
 *   final_state [b][E][N] float32, may be NULL; may be init_state
 *   workspace  ssd_diag_scan_fwd_workspace_bytes(b, L, E, N, G) bytes, no
 *              initial contents: 0 where no sequence is cut (batches that fill
 *              the device by themselves, sequences no longer than a piece).
 *              ssd_diag_scan_workspace_bytes(b, b*L, E, N, G) is never less
 * L == 0 copies init_state (or zeros) into final_state.
 */
SSD_API size_t ssd_diag_scan_fwd_workspace_bytes(int b, int L, int E, int N, int G);
SSD_API ssd_status_t ssd_diag_scan_fwd(const void* u, int64_t u_stride, const void* dt_raw, int64_t dt_stride,
                                       const void* z, int64_t z_stride, const void* B, const void* C,
                                       int64_t bc_stride, const float* A, const float* dt_bias, const float* D,
                                       const float* init_state, void* y, float* final_state, int b, int L, int E,
                                       int N, int G, ssd_dtype_t dtype, void* workspace, size_t workspace_bytes,
                                       cudaStream_t stream);

/*
 * The diagonal scan of packed requests, their states in slots.
 *
 *   u, dt_raw, z, B, C as above with T rows; y [T][E] dtype
 *   states [nslots][E][N] float32, read and written by slot
 *   workspace  ssd_diag_scan_workspace_bytes(nseq, T, E, N, G) bytes (0 for
 *              batches that fill the device by themselves): for any lengths
 *              that the map may hold
 *   status REQUIRED
 */
SSD_API size_t ssd_diag_scan_workspace_bytes(int nseq, int rows, int E, int N, int G);
SSD_API ssd_status_t ssd_diag_scan_fwd_varlen(const void* u, int64_t u_stride, const void* dt_raw,
                                              int64_t dt_stride, const void* z, int64_t z_stride, const void* B,
                                              const void* C, int64_t bc_stride, const float* A,
                                              const float* dt_bias, const float* D, float* states, void* y,
                                              const int32_t* cu_seqlens, const int32_t* seq_of,
                                              const int64_t* slot_of, const int32_t* init_slot, int nseq, int T,
                                              int E, int N, int G, int block_tokens, int nslots,
                                              ssd_dtype_t dtype, void* workspace, size_t workspace_bytes,
                                              int32_t* status, cudaStream_t stream);

/*
 * Gradients through ssd_diag_scan_fwd, given dy = dLoss/dy and dfinal =
 * dLoss/d(final_state).
 *
 *   inputs as the forward call's; dy [b][L][E] dtype; dfinal [b][E][N]
 *          float32 or NULL (zero)
 *   du, ddt_raw, dz [b][L][E] dtype, written (dz exactly when z is given)
 *   dB, dC [b][L][G][N] dtype, written (summed over each group's channels)
 *   dA [E][N], dD, ddt_bias [E] float32, written (summed over the batch)
 *   dinit  [b][E][N] float32, written, may be NULL (not wanted)
 *   workspace  ssd_diag_scan_bwd_workspace_bytes(...) bytes, no initial
 *          contents: a float32 state every 4 tokens (b*L*E*N bytes: 671 MB for
 *          8 x 2048 tokens of 2560 channels, N = 16) and partial sums
 * Deterministic: no atomics.  b == 0 or L == 0 zeroes dA, dD and ddt_bias
 * and copies dfinal (or zeros) into dinit.
 */
SSD_API size_t ssd_diag_scan_bwd_workspace_bytes(int b, int L, int E, int N, int G);
SSD_API ssd_status_t ssd_diag_scan_bwd(const void* u, int64_t u_stride, const void* dt_raw, int64_t dt_stride,
                                       const void* z, int64_t z_stride, const void* B, const void* C,
                                       int64_t bc_stride, const float* A, const float* dt_bias, const float* D,
                                       const float* init_state, const void* dy, const float* dfinal, void* du,
                                       void* ddt_raw, void* dz, void* dB, void* dC, float* dA, float* dD,
                                       float* ddt_bias, float* dinit, int b, int L, int E, int N, int G,
                                       ssd_dtype_t dtype, void* workspace, size_t workspace_bytes,
                                       cudaStream_t stream);

/*
 * One token per request: the recurrence once, from slot init_slot[r] to the
 * slot of the token's block, r = seq_of[i] for row i.  The map's arrays may
 * all be NULL: row i is then state i, in place (nslots >= rows).
 *
 *   u, dt_raw, z, B, C rows as above; y [rows][E] dtype, written
 *   states [nslots][E][N] float32
 *   status REQUIRED with a map
 * A request with more than one row in the call is refused on the device
 * (*status; its rows are left out).
 */
SSD_API ssd_status_t ssd_diag_state_update(float* states, const void* u, int64_t u_stride, const void* dt_raw,
                                           int64_t dt_stride, const void* z, int64_t z_stride, const void* B,
                                           const void* C, int64_t bc_stride, const float* A, const float* dt_bias,
                                           const float* D, void* y, const int32_t* cu_seqlens,
                                           const int32_t* seq_of, const int64_t* slot_of,
                                           const int32_t* init_slot, int nseq, int rows, int E, int N, int G,
                                           int block_tokens, int nslots, ssd_dtype_t dtype, int32_t* status,
                                           cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SSD_DIAG_H_ */
