/*
 * dspark.h -- C ABI of the GB300 (sm_103a) DSpark ancestral draft-block
 * sampler.
 *
 * The method (brb-nv/TensorRT-LLM PR #21, "2. Golden sampling semantics";
 * brb-nv/TensorRT-LLM PR #27, "2. One fused kernel per draft position"):
 * for request b and draft position k = 0..K-1,
 *     l_k   = base_k + bias(d_{k-1}),   bias(d) = U[d] @ Wb   (rank-r head)
 *     s_k   = l_k / T                   (float32 IEEE division)
 *     d_k   = argmax_v (s_k[v] + g[v])  (Gumbel-max; g from Philox noise
 *                                        keyed by (seed, offset, k))
 *     q_k   = softmax(s_k)              (the proposal, written after the
 *                                        block from the same float32 l_k)
 * with d_{-1} = d0[b], the last accepted token.  Greedy requests take
 * d_k = argmax_v s_k[v] and store a one-hot proposal.  CUDA-graph padding
 * rows draw from the bias alone.  Verification is standard token-level
 * rejection sampling (PR #21, "2. Golden sampling semantics").
 *
 * Noise (reading of PR #27, "2. One fused kernel per draft position"):
 * Philox4x32-10 with key = (seed lo, seed hi) and counter
 * (v >> 2, k | stream << 16, offset lo, offset hi), word v & 3; stream 0
 * feeds the draft, 1 the acceptance uniforms, 2 the residual / bonus draws.
 * g = -log(-log1p(-w)), w = (x + 0.5) * 2^-32.  Ties go to the lowest index;
 * a NaN or -inf score never wins, and a row where nothing wins (every score
 * NaN or -inf) yields token 0.
 *
 * Conventions for every entry point:
 *   - All tensors are dense, row-major, and live in device memory unless
 *     stated otherwise.  The caller owns every buffer; the library does not
 *     allocate, free, print or trap, and does not synchronise except in the
 *     calls documented as synchronising (the measurement variants
 *     dspark_draft_block_profile and dspark_draft_block_timeline, and
 *     dspark_read_device_error).
 *   - Calls are asynchronous on `stream` and, except those three, may be
 *     captured in a CUDA graph (their work is kernel launches and memsets on
 *     `stream`).
 *   - Argument checks run on the host before any launch; a failing check
 *     returns a status and enqueues nothing.  A launch failure returns
 *     DSPARK_ERR_CUDA (from cudaGetLastError).
 *   - Results are bitwise deterministic given the inputs on a given GPU
 *     model (fixed reduction order, counter-based noise).
 */
#ifndef DSPARK_H_
#define DSPARK_H_

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#if defined(__GNUC__)
#define DSPARK_API __attribute__((visibility("default")))
#else
#define DSPARK_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { DSPARK_F32 = 0, DSPARK_BF16 = 1 } dspark_dtype;

typedef enum {
  DSPARK_OK = 0,
  DSPARK_ERR_INVALID_ARG = 1, /* null pointer, non-positive size, bad T,
                                 misaligned pointer, out-of-range token */
  DSPARK_ERR_UNSUPPORTED = 2, /* valid but outside the supported shapes */
  DSPARK_ERR_WORKSPACE = 3,   /* workspace missing or too small */
  DSPARK_ERR_CUDA = 4,        /* a CUDA runtime call or launch failed */
  DSPARK_ERR_DEVICE = 5       /* a kernel recorded an error in the workspace
                                 (a bounded wait ran out); see
                                 dspark_read_device_error */
} dspark_status;

/* Supported shapes: 1 <= B <= 1024, 1 <= K <= 64, 1 <= V <= 2^26,
 * 16 <= r <= 256 with r % 16 == 0.  (PR #27, Results: B x 7 x 200064
 * logits and a rank-256 head sit inside these limits.) */
#define DSPARK_MAX_B 1024
#define DSPARK_MAX_K 64
#define DSPARK_MAX_R 256
#define DSPARK_MAX_V (1 << 26)

/*
 * Bytes of device workspace dspark_draft_block needs for these sizes
 * (0 if the sizes are unsupported).  The workspace holds a device error
 * word (its first 4 bytes), the decision keys the position kernels share
 * across CTAs, per-chunk softmax statistics (two buffers, so consecutive
 * positions do not overwrite each other's) and per-row (max, sum-exp) of
 * every position.  Its contents need not be initialised: every call first
 * clears the error word and the keys (one 2-D memset on `stream`), and
 * every other word is written before it is read.  Two calls in flight at
 * the same time must not share a workspace.
 */
DSPARK_API size_t dspark_draft_workspace_bytes(int B, int K, int V, int r);

/*
 * dspark_draft_block -- ancestral drafting of one K-token block for B
 * requests (PR #27, "2. One fused kernel per draft position").
 *
 *   base_logits  [B,K,V] base_dtype (F32 or BF16); read only, never modified
 *                (PR #27, Test Coverage: the drafter's logits are left as
 *                they are).  Rows of padding requests may hold anything,
 *                NaN included.
 *   U            [V,r] w_dtype;  Wb [r,V] w_dtype (F32 or BF16, both the
 *                same dtype).  bias(d) = U[d] @ Wb, accumulated in float32.
 *   d0           [B] int32, the last accepted token of each request, in
 *                [0, V).  An entry outside that range is replaced by 0 and
 *                the workspace's device error word is set to 1 (read it with
 *                dspark_read_device_error).
 *   seed, offset [B] uint64 each: the request's noise key and draft slot.
 *                A new offset draws anew (PR #27, Test Coverage).
 *   T            temperature, finite and > 0 (the same for every request).
 *   greedy       [B] uint8 or NULL: nonzero = greedy request (argmax chain,
 *                one-hot proposal, no noise consumed).  NULL = all sampled.
 *   pad_row      [B] uint8 or NULL: nonzero = CUDA-graph padding row; its
 *                base logits are ignored and l = bias (PR #27: padding rows
 *                draw from the bias alone).
 *   tokens       [B,K] int32 out: the drafted tokens d_k.
 *   logits       [B,K,V] float32 out: the biased logits l_k.
 *   draft_probs  [B,K,V] float32 out: the proposals q_k.
 *   workspace    device scratch of at least
 *                dspark_draft_workspace_bytes(B,K,V,r) bytes, 256-byte
 *                aligned.
 * Alignment: every device pointer must be at least 16-byte aligned
 * (DSPARK_ERR_INVALID_ARG otherwise).
 * Launches on `stream`, after one 2-D memset of the error word and the
 * decision keys: with a bf16 head, r a multiple of 16 up to 256 and
 * V % 8 == 0 the tensor-core kernel, K positions and one pick per request
 * group (ceil(B / 96) groups of near-equal size, each a chain over the same
 * heads), then one proposal writer; otherwise the FFMA kernel, K positions
 * and K picks, then the writer.  No host synchronisation; graph capturable.
 */
DSPARK_API dspark_status dspark_draft_block(
    const void* base_logits, dspark_dtype base_dtype, const void* U,
    const void* Wb, dspark_dtype w_dtype, const int32_t* d0,
    const uint64_t* seed, const uint64_t* offset, float T,
    const uint8_t* greedy, const uint8_t* pad_row, int B, int K, int V, int r,
    int32_t* tokens, float* logits, float* draft_probs, void* workspace,
    size_t workspace_bytes, cudaStream_t stream);

/*
 * dspark_draft_block_profile -- measurement variant of dspark_draft_block:
 * the same argument checks and the same launch sequence, with a pair of CUDA
 * events recorded on `stream` around every launch.  It then synchronises
 * `stream` and returns, per kernel class, the summed event time and the
 * number of launches:
 *   stage_ms[3], stage_launches[3]  (host arrays) -- [0] the position
 *   kernels (K per request group), [1] the pick kernels (one after each
 *   group's last position on the tensor-core path, one after every position
 *   on the FFMA path), [2] the proposal writer.  The events between launches remove the overlap of
 *   consecutive positions (programmatic dependent launch); see
 *   dspark_draft_block_timeline for times in the block's own schedule.
 * Outputs are identical to dspark_draft_block's.  Because it synchronises
 * and creates events, it must not be captured in a CUDA graph.
 */
DSPARK_API dspark_status dspark_draft_block_profile(
    const void* base_logits, dspark_dtype base_dtype, const void* U,
    const void* Wb, dspark_dtype w_dtype, const int32_t* d0,
    const uint64_t* seed, const uint64_t* offset, float T,
    const uint8_t* greedy, const uint8_t* pad_row, int B, int K, int V, int r,
    int32_t* tokens, float* logits, float* draft_probs, void* workspace,
    size_t workspace_bytes, float* stage_ms, int* stage_launches,
    cudaStream_t stream);

/*
 * dspark_draft_block_timeline -- measurement variant of dspark_draft_block
 * that keeps the block's own schedule (positions chained by programmatic
 * dependent launch, no event between them).  It captures one
 * dspark_draft_block launch sequence from `stream` into a CUDA graph, with
 * event nodes at its start, between the position chain (the memset, the K
 * position kernels and their picks) and the proposal writer, and at its
 * end; it then replays the graph `replays` (>= 1) times, synchronising
 * after each replay, and returns the mean duration of each segment:
 *   chain_ms[1], proposal_ms[1] (host) -- milliseconds per replay.
 * `stream` must be a created stream (not the legacy NULL stream; status
 * DSPARK_ERR_INVALID_ARG) that is not already capturing.  Outputs are
 * identical to dspark_draft_block's.  It creates three events, a graph and
 * its executable (the driver allocates for them) and destroys them before
 * returning; it synchronises and must not itself be captured.
 */
DSPARK_API dspark_status dspark_draft_block_timeline(
    const void* base_logits, dspark_dtype base_dtype, const void* U,
    const void* Wb, dspark_dtype w_dtype, const int32_t* d0,
    const uint64_t* seed, const uint64_t* offset, float T,
    const uint8_t* greedy, const uint8_t* pad_row, int B, int K, int V, int r,
    int32_t* tokens, float* logits, float* draft_probs, void* workspace,
    size_t workspace_bytes, int replays, float* chain_ms, float* proposal_ms,
    cudaStream_t stream);

/*
 * dspark_draft_block_per_request -- dspark_draft_block with a temperature
 * per request and slot-indexed proposals, as a serving batch needs them
 * (PR #27, "2. One fused kernel per draft position": the proposal writer
 * stores q_k into the slot-indexed draft_probs; the temperature of a draft
 * is its request's sampling temperature).
 *
 *   temperature  [B] float32, device, 4-byte aligned: request b's T.  A
 *                value that is not finite and positive counts as 1 and sets
 *                the device error word to 3 (DSPARK_ERR_DEVICE via
 *                dspark_read_device_error).
 *   draft_probs  [num_slots, K, V] float32 when slot is given, else [B,K,V].
 *   slot         [B] int32 device (4-byte aligned) or NULL: request b's
 *                proposals are written to draft_probs[slot[b]]; slots of
 *                different requests must differ; a slot outside
 *                [0, num_slots) writes nothing for that request and sets the
 *                device error word to 4.  Slots of no request are left as
 *                they are.
 *   num_slots    rows of draft_probs (ignored when slot is NULL).
 * Every other argument, the workspace (dspark_draft_workspace_bytes) and the
 * errors are those of dspark_draft_block; tokens and logits stay [B,K] and
 * [B,K,V].  With equal temperatures T the outputs are bitwise those of
 * dspark_draft_block with T.
 */
DSPARK_API dspark_status dspark_draft_block_per_request(
    const void* base_logits, dspark_dtype base_dtype, const void* U,
    const void* Wb, dspark_dtype w_dtype, const int32_t* d0,
    const uint64_t* seed, const uint64_t* offset, const float* temperature,
    const uint8_t* greedy, const uint8_t* pad_row, int B, int K, int V, int r,
    int32_t* tokens, float* logits, float* draft_probs, const int32_t* slot,
    int num_slots, void* workspace, size_t workspace_bytes,
    cudaStream_t stream);

/*
 * dspark_draft_block_noalloc -- dspark_draft_block for callers that cannot
 * allocate device memory: code that is handed only its input and output
 * buffers by a host runtime that owns all device memory (an inference
 * server that sizes every allocation at start-up and forbids allocation
 * afterwards), or that runs where cudaMalloc must not be called.  There is
 * no counterpart in the pages; it is the same launch sequence as
 * dspark_draft_block with the workspace replaced by library-owned scratch.
 *
 * Arguments and outputs are those of dspark_draft_block without
 * `workspace` / `workspace_bytes`.  The scratch is one file-scope device
 * array of DSPARK_NOALLOC_SCRATCH_BYTES bytes (2 MiB), held on every GPU
 * that loads the library until the process exits; sizes whose workspace
 * (dspark_draft_workspace_bytes) exceeds it are rejected with
 * DSPARK_ERR_WORKSPACE before any launch (B <= 101 fits at K = 7).
 * The call allocates nothing: no cudaMalloc, cudaFree or allocating library
 * routine.  Each call made outside stream capture looks up the scratch's
 * device address on the current device (so a device reset or a new primary
 * context is followed); a call made during a capture uses the address the
 * last uncaptured call on that device found, so the first call on a device
 * must come before any capture, and a capture must not outlive a device
 * reset.  Every call on a device shares the one scratch array and it keeps
 * the last call's contents (each call clears the device error word and the
 * decision keys it starts with); calls that overlap on the GPU, from any
 * stream or thread, race on it and must be serialised by the caller.  Device-side error codes
 * of this variant stay in the scratch and are not reported.
 */
#define DSPARK_NOALLOC_SCRATCH_BYTES (2u << 20)
DSPARK_API dspark_status dspark_draft_block_noalloc(
    const void* base_logits, dspark_dtype base_dtype, const void* U,
    const void* Wb, dspark_dtype w_dtype, const int32_t* d0,
    const uint64_t* seed, const uint64_t* offset, float T,
    const uint8_t* greedy, const uint8_t* pad_row, int B, int K, int V, int r,
    int32_t* tokens, float* logits, float* draft_probs, cudaStream_t stream);

/*
 * dspark_draft_host_workspace_bytes -- device workspace of
 * dspark_draft_block_host: that of dspark_draft_block plus room for the
 * per-request inputs and the tokens (0 if the sizes are unsupported).
 */
DSPARK_API size_t dspark_draft_host_workspace_bytes(int B, int K, int V, int r);

/*
 * dspark_draft_block_host -- dspark_draft_block with its inputs in host
 * memory and the drafted tokens returned to host memory; the call issues
 * the copies itself.
 *
 *   base_logits_host [B,K,V] base_dtype in host memory.  Page-locked memory
 *                lets the copies run asynchronously (with pageable memory
 *                each copy synchronises).
 *   d0_host, seed_host, offset_host [B]; greedy_host, pad_row_host [B] or
 *                NULL: host memory, meanings as in dspark_draft_block.
 *   U, Wb        device, as in dspark_draft_block (resident weights).
 *   base_dev     device [B,K,V] base_dtype buffer that receives the drafter
 *                logits (16-byte aligned; read by this call's kernels).
 *   tokens_host  [B,K] int32 host out, copied on `stream` after the block.
 *   logits, draft_probs  device [B,K,V] float32 outputs.
 *   workspace    device, dspark_draft_host_workspace_bytes(B,K,V,r) bytes,
 *                256-byte aligned.
 *   stream       the compute stream; copy_stream a second stream for the
 *                drafter-logit copies (must differ from stream).
 * Position k's drafter logits (B rows of V values, one 2-D copy) travel on
 * copy_stream while earlier positions compute on stream.  Position k waits
 * for its own copy only, and each position's proposals are written as soon
 * as its softmax statistics exist (after the next position on the
 * tensor-core path, after its pick otherwise), so the block's work hides
 * behind the copies.  The copies start after all
 * work issued to `stream` before the call.  Outputs are identical to
 * dspark_draft_block's.  Host buffers must stay valid until `stream` has
 * passed the end of the call.  The call creates and destroys K+1 CUDA
 * events.  It may be captured in a CUDA graph: its event waits join
 * copy_stream to the capture of `stream`.
 */
DSPARK_API dspark_status dspark_draft_block_host(
    const void* base_logits_host, dspark_dtype base_dtype, const void* U,
    const void* Wb, dspark_dtype w_dtype, const int32_t* d0_host,
    const uint64_t* seed_host, const uint64_t* offset_host, float T,
    const uint8_t* greedy_host, const uint8_t* pad_row_host, int B, int K,
    int V, int r, void* base_dev, int32_t* tokens_host, float* logits,
    float* draft_probs, void* workspace, size_t workspace_bytes,
    cudaStream_t stream, cudaStream_t copy_stream);

/*
 * dspark_verify_standard -- standard token-level rejection sampling of the
 * drafts (PR #21, "2. Golden sampling semantics": the default rule), for B
 * requests.
 *
 *   draft_probs  [B,K,V] float32: the proposals q_k the drafts came from.
 *   target_probs [B,K+1,V] float32: the target's p_k for the drafted prefix;
 *                row K is the bonus distribution.
 *   tokens       [B,K] int32 drafts, each in [0, V) (a token outside it makes
 *                that request report accepted_len = -1).
 *   seed, offset [B] uint64 (streams 1 and 2 of the counter layout above).
 *   accepted_len [B] int32 out: number of accepted drafts, 0..K.
 *   emitted_token[B] int32 out: the token emitted after the accepted prefix
 *                (the residual draw at the first rejection, or the bonus
 *                draw from p_K when all K are accepted).
 * Draft k is accepted iff float(u_k * q_k[d_k]) < p_k[d_k] with
 * u_k = ((x >> 9) + 0.5) * 2^-23 from stream 1 word 0 at position k.  The
 * residual is max(p_k - q_k, 0) (p_k itself if that is all zero); draws are
 * Gumbel-max over log(weight) with stream 2 noise at the drawing position.
 */
DSPARK_API dspark_status dspark_verify_standard(const float* draft_probs,
                                     const float* target_probs,
                                     const int32_t* tokens,
                                     const uint64_t* seed,
                                     const uint64_t* offset, int B, int K,
                                     int V, int32_t* accepted_len,
                                     int32_t* emitted_token,
                                     cudaStream_t stream);

/*
 * dspark_verify_block -- block verification of the drafts (PR #21, "2.
 * Golden sampling semantics": the block value of rejection_sample_method,
 * the block verification of Sun et al., 2024), for B requests.  Arguments,
 * layouts, outputs and errors are those of dspark_verify_standard.
 * With d_k = tokens[b,k], q_k = draft_probs[b,k], p_k = target_probs[b,k]:
 *   w_0 = 1, w_{k+1} = min(w_k * (p_k[d_k] / q_k[d_k]), 1) in float32
 *   (a NaN weight counts as 0);
 *   h_i = r_i / (r_i + 1 - w_i) for i = 1..K-1, with
 *   r_i = sum_x max(w_i p_i(x) - q_i(x), 0) (1 when r_i = 1 - w_i = 0);
 *   h_K = w_K;
 *   accepted_len = the largest i in 1..K with u_{i-1} <= h_i (0 if none),
 *   u_k the uniform of the standard rule;
 *   emitted_token: Gumbel-max with stream 2 noise at position accepted_len
 *   over p_K when accepted_len = K, else over max(w p - q, 0) at that
 *   position (over p itself if that is all zero).
 * The sums r_i run in float32 in a fixed order (results are reproducible
 * call to call).  The call reads the K-1 rows p_1..p_{K-1} and q_1..q_{K-1}
 * in full.  On average it accepts at least as many drafts as the standard
 * rule, and it is lossless.
 */
DSPARK_API dspark_status dspark_verify_block(const float* draft_probs,
                                  const float* target_probs,
                                  const int32_t* tokens, const uint64_t* seed,
                                  const uint64_t* offset, int B, int K, int V,
                                  int32_t* accepted_len, int32_t* emitted_token,
                                  cudaStream_t stream);

/*
 * dspark_sample_workspace_bytes -- device workspace of
 * dspark_sample_temperature for R rows of V logits (0 if unsupported).
 */
DSPARK_API size_t dspark_sample_workspace_bytes(int R, int V);

/*
 * dspark_sample_temperature -- temperature-only sampling of target rows
 * (PR #27, "1. Temperature-only sampling runs no filter": softmax and
 * sampling, no top-k, top-p or min-p).
 *
 *   logits       [R,V] float32 device: one row per sample.
 *   temperature  [R] float32 device (4-byte aligned) or NULL: per-row T (a
 *                value that is not finite and positive counts as 1 and sets
 *                the device error word to 3); NULL uses T (finite, > 0).
 *   greedy       [R] uint8 or NULL: 1 = argmax of s, one-hot probabilities.
 *   seed, offset [R] uint64: the row's noise key and counter words.
 *   position     [R] int32 (4-byte aligned) or NULL (0): the counter's
 *                position word, in [0, 65535] (outside: 0 is used and the
 *                device error word is set to 5).
 *   tokens       [R] int32 out; probs [R,V] float32 out, or NULL to skip.
 *   workspace    dspark_sample_workspace_bytes(R, V) bytes, 256-byte aligned.
 * Row i: s = l / T_i (float32 IEEE), token = argmax of s + g with g from
 * noise stream 3 (word v & 3 of Philox4x32-10 block (v >> 2,
 * position | 3 << 16, offset lo, offset hi) under key seed), the lowest
 * index on ties, NaN never winning (a row where nothing wins gives token 0);
 * probs = softmax(s).  R <= 65535.  Three launches on `stream` (two when
 * probs is NULL), graph capturable; results are reproducible call to call.
 */
DSPARK_API dspark_status dspark_sample_temperature(
    const float* logits, const float* temperature, float T,
    const uint8_t* greedy, const uint64_t* seed, const uint64_t* offset,
    const int32_t* position, int R, int V, int32_t* tokens, float* probs,
    void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* ------------------------------------------------ the paged key/value cache
 *
 * The steps around the draft block that read and write a model's (or a
 * drafter's) key/value cache: room for a step's tokens is reserved, each
 * layer's queries and keys are normalised and rotated and the keys and
 * values stored, the drafted tokens attend over the cache, and after
 * verification the accepted path is moved together and the pages behind it
 * are freed.  A sequence can be forked: its full pages are shared.
 *
 * The caller owns every array.  A cache of S = max_seqs sequences:
 *   pool         [layers][2][num_pages][kv_heads][page_size][head_dim] dtype,
 *                keys in plane 0 of a layer and values in plane 1; 16-byte
 *                aligned.
 *   block_table  [max_seqs][max_pages] int32: entry i of a row is the page of
 *                tokens i * page_size .. of that sequence; -1 behind the held
 *                pages.
 *   page_count   [max_seqs] int32: pages that a sequence holds.
 *   ref_count    [num_pages] int32: sequences that hold a page.
 *   free_list    [num_pages] int32: a stack of the free pages; pages are
 *                taken from its top.
 *   control      [DSPARK_CACHE_CONTROL_WORDS] int32, 16-byte aligned: [0] the
 *                device error word (dspark_read_device_error reads and clears
 *                it; calls on a cache set it and never clear it), [1] the
 *                number of free pages, [2] a counter that every call leaves
 *                at 0; scratch from word 64 on.
 * Lengths are the caller's: `length` [B] int32 is the number of committed
 * tokens of each sequence of a call.  `seq` [B] int32 (or NULL: 0..B-1)
 * names the sequences, each at most once in a call.
 * Limits: 1 <= layers <= 1024, page_size <= 4096, head_dim a multiple of 8
 * up to 256, kv_heads <= 1024, max_seqs * max_pages < 2^31, num_pages < 2^31,
 * max_pages * page_size <= 2^30, B <= 1024.  The pool is addressed in 64 bits.
 *
 * Sequences, pages, positions and paths that are out of range are seen on
 * the device: the entry is skipped as its call says and the error word is
 * set (2: a bounded wait inside the attention ran out, its result is not to
 * be used; 6: a seq outside [0, max_seqs); 7: a length or page outside what the
 * sequence holds; 8: no free page left, or more pages than a table row has;
 * 9: an accepted path or length that is not one; 10: a position outside the
 * rotation table; 11: a fork whose child is a parent, or twice a child; 12: a
 * group of sequences that is none, or whose prefix one of them does not have).
 * Calls on one cache must follow one another (one stream, or ordered by the
 * caller); calls on different caches are independent. */
typedef struct {
  void* pool;
  dspark_dtype dtype;
  int layers, num_pages, kv_heads, page_size, head_dim;
  int max_seqs, max_pages;
  int32_t* block_table;
  int32_t* page_count;
  int32_t* ref_count;
  int32_t* free_list;
  int32_t* control;
} dspark_cache;

#define DSPARK_CACHE_MAX_B 1024
#define DSPARK_CACHE_CONTROL_WORDS (64 + 2 * DSPARK_CACHE_MAX_B)
#define DSPARK_TREE_MAX_TOKENS 64
#define DSPARK_TREE_MAX_GROUP 32

/*
 * dspark_cache_init -- an empty cache: no sequence holds a page, every page
 * is free (page 0 on top of the stack), the error word is 0.  The pool is
 * left as it is.  One launch, graph capturable.
 */
DSPARK_API dspark_status dspark_cache_init(const dspark_cache* cache,
                                           cudaStream_t stream);

/*
 * dspark_cache_reserve -- pages for `tokens` (>= 0) more tokens of each of B
 * sequences: afterwards sequence seq[b] holds at least
 * ceil((length[b] + tokens) / page_size) pages.  Pages are taken in the order
 * of b and, within a sequence, of its tokens.  A sequence whose table row is
 * too short, or for which too few pages are free, gets none (error 8), and
 * the others are served.  One launch.
 */
DSPARK_API dspark_status dspark_cache_reserve(const dspark_cache* cache,
                                              const int32_t* seq,
                                              const int32_t* length,
                                              int tokens, int B,
                                              cudaStream_t stream);

/*
 * dspark_cache_release -- the B sequences give up all their pages.  Pages
 * that no sequence holds any more go back on the stack, the last one first
 * (so reserving and releasing the same sequences leaves the stack as it
 * was).  One launch.
 */
DSPARK_API dspark_status dspark_cache_release(const dspark_cache* cache,
                                              const int32_t* seq, int B,
                                              cudaStream_t stream);

/*
 * dspark_cache_fork -- sequence child[b] becomes a copy of the first
 * length[b] tokens of sequence parent[b], in every layer: the full pages are
 * shared, and the tokens of a page that is partly filled are copied to a page
 * of the child's own.  Pages that the child held before are given up first.
 * Several children may have the same parent; a child that is also a parent
 * of the call, or is named twice, makes the whole call do nothing (error 11).
 * A child whose parent holds fewer than length[b] tokens (error 7), or for
 * which no page is free (error 8), ends up empty.  Shared pages are full, so
 * nothing writes to them as long as a sequence's length does not shrink; one
 * that is to be cut back is forked at the shorter length instead.  Two
 * launches.
 */
DSPARK_API dspark_status dspark_cache_fork(const dspark_cache* cache,
                                           const int32_t* parent,
                                           const int32_t* child,
                                           const int32_t* length, int B,
                                           cudaStream_t stream);

/*
 * dspark_cache_accept -- keeps the accepted ones of the `tokens` tokens that
 * follow the committed ones: n = accepted_len[b] + extra of them stay (none
 * if accepted_len[b] < 0, verification's report of a bad request).
 *
 *   path         [B, path_width] int32 or NULL: the i-th kept token is the
 *                one at length[b] + path[b][i], strictly increasing in i and
 *                below `tokens`; it moves to length[b] + i, keys and values,
 *                in every layer.  NULL: the kept tokens are the first n.
 *   accepted_len [B] int32, as the verification calls write it.
 *   extra        tokens kept besides the accepted drafts (1 when the tokens
 *                start with the last emitted one).
 *   new_length   [B] int32 out (may be `length`): length[b] + n.
 * Pages behind the kept tokens are given up as dspark_cache_release does.  A
 * path that is not one, or n > path_width or tokens, keeps nothing (error 9).
 * One launch.
 */
DSPARK_API dspark_status dspark_cache_accept(
    const dspark_cache* cache, const int32_t* seq, const int32_t* length,
    const int32_t* accepted_len, const int32_t* path, int path_width,
    int extra, int tokens, int B, int32_t* new_length, cudaStream_t stream);

/*
 * dspark_cache_append -- the queries and keys of T new tokens of each of B
 * sequences, normalised for each head and rotated by their positions, in one
 * pass; keys and values go to the cache of `layer`, token t of sequence b to
 * place length[b] + t (whose page must be held: dspark_cache_reserve).
 *
 *   q            [B,T,heads,D], k and v [B,T,kv_heads,D], the cache's dtype,
 *                D = head_dim; a token's heads are dense, and consecutive
 *                tokens lie q_stride, k_stride, v_stride elements apart (so
 *                the three may be parts of one projection's output).
 *                16-byte aligned, strides multiples of 8 elements.
 *   q_weight, k_weight  [D] float32 or NULL: y = x / sqrt(mean(x^2) + eps) * w
 *                over each head (NULL: no normalisation).
 *   cos_sin      [max_position][rot_dim] float32: rot_dim / 2 cosines, then
 *                the sines.  The first rot_dim (even, <= D) dims are rotated:
 *                pairs (i, i + rot_dim / 2), or (2 i, 2 i + 1) when
 *                `interleaved`: (a, b) -> (a c - b s, b c + a s).
 *   position     [B,T] int32 rows of cos_sin.
 *   token_count  [B] int32 or NULL (T): tokens of sequence b (below 0: none,
 *                above T: T); later rows of
 *                q_out and later places of the cache are left as they are.
 *   q_out        [B,T,heads,D] dense.  It may be q when that is dense; else it
 *                must not overlap a token's rows of q, k or v.
 * Everything runs in float32 and is rounded once; values are copied.  A token
 * whose page is not held is not stored (error 7); one with a position outside
 * the table is not rotated (error 10).  One launch, B * T < 2^24.
 */
DSPARK_API dspark_status dspark_cache_append(
    const dspark_cache* cache, int layer, const int32_t* seq,
    const int32_t* length, const int32_t* token_count, const void* q,
    int64_t q_stride, const void* k, int64_t k_stride, const void* v,
    int64_t v_stride, const float* q_weight, const float* k_weight, float eps,
    const float* cos_sin, int max_position, int rot_dim, int interleaved,
    const int32_t* position, int B, int T, int heads, void* q_out,
    cudaStream_t stream);

/* Device workspace of dspark_tree_attention (0 if unsupported). */
DSPARK_API size_t dspark_tree_workspace_bytes(int B, int T, int heads,
                                              int kv_heads, int head_dim);

/*
 * dspark_tree_attention -- attention of T drafted tokens of each of B
 * sequences over the cache of `layer`, the drafted tokens' own keys and values
 * included (they lie behind the committed ones, see dspark_cache_append).
 *
 *   q            [B,T,heads,D] dense, the cache's dtype, 16-byte aligned.
 *                heads = group * kv_heads; query head h reads key head
 *                h / group.
 *   mask         uint64 words or NULL: bit j of word t says that token t sees
 *                drafted token j: the ancestors of t in a tree of drafts and
 *                t itself, all tokens in a block that sees itself whole.
 *                mask_stride words lie between two sequences (0: one tree for
 *                all).  NULL: token t sees tokens 0..t.
 *   token_count  [B] int32 or NULL (T): drafted tokens of sequence b (below 0:
 *                none, above T: T).  Later
 *                rows of out and lse are left as they are, later keys are not
 *                read.
 *   window       0, or the number of positions that a token sees: token t
 *                sees committed token j if position[b][t] - j < window.  The
 *                mask alone rules the drafted tokens: with a NULL mask and a
 *                window below T a token sees drafted ones beyond the window, and
 *                a caller that wants them hidden leaves their bits out.
 *   position     [B,T] int32 or NULL (length[b] + t), used with a window; a
 *                position below length[b] counts as length[b].
 *   scale        of the scores q.k, finite.
 *   out          [B,T,heads,D] dense: sum_j p_j v_j, p = softmax(scale q.k)
 *                over the visible tokens; zeros for a token that sees none.
 *                Must not overlap q.
 *   lse          [B,T,heads] float32 or NULL: log(sum_j exp(scale q.k_j)),
 *                -inf for a token that sees none.
 *   workspace    dspark_tree_workspace_bytes(...) bytes, 256-byte aligned; its
 *                contents need not be initialised.  Two calls in flight at
 *                the same time must not share it.
 * Scores, softmax statistics and sums are float32.  The tensor cores multiply
 * weights rounded to bfloat16 (relative error 2^-8 at most each, the sum of the
 * weights being that of the unrounded ones); the FFMA kernel multiplies float32
 * weights, also of bfloat16 inputs.  Keys and values of
 * places that a token does not see never reach its result, whatever they
 * hold.  A sequence whose length or pages are out of range is not computed
 * (error 6 or 7; its rows are left as they are); a table entry that names no
 * page reads as zeros (error 7).  A call with 2^31 tiles of keys or more (128
 * keys a tile on the tensor cores, 64 or 32 on the FFMA kernel), over all
 * sequences, key heads and groups of query rows, is not computed (error 7).
 * 1 <= T <= 64, group <= 32.  bfloat16 with head_dim 64 or 128 and a page size
 * that is a power of two from 8 on runs on the tensor cores, everything else
 * on the FFMA kernel.  Two launches, graph capturable, no synchronisation.
 */
DSPARK_API dspark_status dspark_tree_attention(
    const dspark_cache* cache, int layer, const int32_t* seq,
    const int32_t* length, const int32_t* token_count, const void* q,
    const uint64_t* mask, int64_t mask_stride, const int32_t* position,
    int window, float scale, int B, int T, int heads, void* out, float* lse,
    void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* ------------------------------------------- reading part of the cache
 *
 * A long context costs a query its whole length.  The calls below let it read
 * less: dspark_cache_bounds keeps the smallest and largest keys of every full
 * page, dspark_select_pages chooses pages for each query by them, and
 * dspark_sparse_attention attends over the chosen ones; and
 * dspark_prefix_attention reads what several sequences share (dspark_cache_fork)
 * once for all of them.
 *
 * The caller owns the bounds: [layers][num_pages][kv_heads][2][head_dim] of the
 * cache's dtype, 16-byte aligned, the smallest keys and then the largest.  They
 * are kept by page, so sequences that share a page share its bounds.  A page
 * counts as full, and is chosen, when all its tokens are committed. */

/*
 * dspark_cache_bounds -- the bounds, in every layer, of the pages that the
 * sequences have filled between `start` [B] and `length` [B] committed tokens:
 * those whose last token lies in [start, length).  A call behind each
 * dspark_cache_accept or prompt, with the lengths before and after it, keeps
 * them; a length below its start fills nothing.  Other bounds are left as they
 * are.  A NaN among a page's keys makes the bounds of its dimension NaN.  A
 * sequence that holds fewer than `length` tokens is left out (error 7), and so are
 * all where they have filled 2^31 pages or more.  One launch.
 */
DSPARK_API dspark_status dspark_cache_bounds(const dspark_cache* cache,
                                             const int32_t* seq,
                                             const int32_t* start,
                                             const int32_t* length, int B,
                                             void* bounds, cudaStream_t stream);

/* Device workspace of dspark_select_pages (0 if unsupported). */
DSPARK_API size_t dspark_select_workspace_bytes(const dspark_cache* cache, int B,
                                                int T, int shared);

/*
 * dspark_select_pages -- for each drafted token and key head (or, with
 * `shared`, for all of a sequence's tokens together) the `count` full pages of
 * the sequence whose keys can have the largest products with the queries.
 *
 *   q            [B,T,heads,D] dense, the cache's dtype, 16-byte aligned.
 *   bounds       of every layer, as dspark_cache_bounds keeps them.
 *   token_count  [B] int32 or NULL (T), as in dspark_tree_attention: lists of
 *                later tokens are left as they are, and a shared list goes by
 *                the tokens that there are.
 *   first, last  so many of the sequence's first and of its last full pages
 *                are always taken; they count.  first + last <= count.
 *   pages        [B,T,kv_heads,count] int32 out ([B,1,kv_heads,count] with
 *                `shared`): the pages' numbers within the sequence (tokens
 *                page * page_size ..), ascending, then -1 where the sequence
 *                has fewer full pages.
 * A page's score is the largest, over the query heads of the key head (and over
 * the tokens with `shared`), of sum_d max(q_d min_d, q_d max_d): no product of
 * q with a key of the page exceeds it.  (For attention with scale > 0.)  The
 * choice is that of exact scores: where float32 leaves it open, pages are
 * scored more exactly (off by 2^-46 of the largest that sums of their terms can
 * be).  Equal scores go to the lower page; a score that is not a number counts as
 * infinite.
 * 1 <= T <= 64, group <= 32.  A sequence whose length is out of range is left out
 * (error 6 or 7); a table entry that names no page has the lowest score (error
 * 7).  Two launches, graph capturable; the same result on every run.  The
 * workspace's contents need not be initialised; two calls in flight at the
 * same time must not share it.
 */
DSPARK_API dspark_status dspark_select_pages(
    const dspark_cache* cache, int layer, const int32_t* seq,
    const int32_t* length, const int32_t* token_count, const void* q,
    const void* bounds, int count, int first, int last, int shared, int B, int T,
    int heads, int32_t* pages, void* workspace, size_t workspace_bytes,
    cudaStream_t stream);

/* Device workspace of dspark_sparse_attention (0 if unsupported). */
DSPARK_API size_t dspark_sparse_workspace_bytes(const dspark_cache* cache, int B,
                                                int T, int heads, int count);

/*
 * dspark_sparse_attention -- attention of T drafted tokens of each of B
 * sequences over part of the cache of `layer`: the full pages that a list
 * names, the committed tokens behind the last full page, and the drafted tokens
 * that the mask allows.
 *
 *   pages        [B,T,kv_heads,count] int32, or [B,1,kv_heads,count] with
 *                `shared`: for each key head the pages of a token (or of all
 *                tokens), by their numbers within the sequence, as
 *                dspark_select_pages writes them.  Any order; entries below 0 are
 *                passed over, and a page named twice counts once.  An entry at
 *                or behind the sequence's full pages is passed over too (error
 *                7).  Lists of tokens behind the last one are not read.
 * All else is as for dspark_tree_attention: q, mask, token_count, scale, out, lse,
 * what a token sees that sees nothing, the workspace, the roundings, the shapes
 * that run on the tensor cores (here with every head_dim up to 128 that is a
 * multiple of 16: those but 64 and 128 have their weights rounded to bfloat16
 * here, and not in dspark_tree_attention), and the errors.  Keys and values that a token
 * does not see never reach its result, those of pages that only other tokens'
 * lists name among them.  count * T <= 2^24.  Three launches, graph capturable, no
 * synchronisation.
 */
DSPARK_API dspark_status dspark_sparse_attention(
    const dspark_cache* cache, int layer, const int32_t* seq,
    const int32_t* length, const int32_t* token_count, const void* q,
    const int32_t* pages, int count, int shared, const uint64_t* mask,
    int64_t mask_stride, float scale, int B, int T, int heads, void* out,
    float* lse, void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Device workspace of dspark_prefix_attention (0 if unsupported). */
DSPARK_API size_t dspark_prefix_workspace_bytes(int B, int T, int heads,
                                                int kv_heads, int head_dim);

/*
 * dspark_prefix_attention -- dspark_tree_attention without a window for
 * sequences that share prefixes: the shared keys and values are read once for
 * all the sequences of a group, not once for each.
 *
 *   group_start  [groups + 1] int32: group g is rows group_start[g] ..
 *                group_start[g + 1] - 1 of the call, not decreasing; rows in no
 *                group are attended by themselves.  1 <= groups <= B.
 *   prefix       [groups] int32: committed tokens that the group's sequences
 *                share.  They are read through the pages of the group's first
 *                row, which the other rows need not hold themselves; their
 *                table entries there are not looked at.
 * A row whose sequence has fewer committed tokens than its group's prefix is
 * attended by itself, as all rows are where group_start is no such list, and a
 * group's where its first row has fewer or does not hold them (error 12).  Results do
 * not depend on it where the pages hold the same tokens, but for roundings.  All
 * else is as for dspark_tree_attention, but that the shapes that run on the tensor
 * cores, with their rounding of the weights, are dspark_sparse_attention's; partial
 * results of both kinds are float32.  B * T * heads < 2^31.  Three or four launches, graph capturable, no
 * synchronisation.
 */
DSPARK_API dspark_status dspark_prefix_attention(
    const dspark_cache* cache, int layer, const int32_t* seq,
    const int32_t* length, const int32_t* token_count, const void* q,
    const int32_t* group_start, const int32_t* prefix, int groups,
    const uint64_t* mask, int64_t mask_stride, float scale, int B, int T,
    int heads, void* out, float* lse, void* workspace, size_t workspace_bytes,
    cudaStream_t stream);

/*
 * dspark_noise_words -- diagnostic: writes the n raw Philox words the
 * sampler uses for elements 0..n-1 of (seed, offset, position k, stream),
 * i.e. out[v] = word (v & 3) of Philox4x32-10(counter (v >> 2,
 * k | stream << 16, offset lo, offset hi), key (seed lo, seed hi)), and
 * gumbel[v] = the float32 Gumbel variate the draft kernel derives from it
 * (gumbel may be NULL).  out/gumbel are device pointers.
 */
DSPARK_API dspark_status dspark_noise_words(uint64_t seed, uint64_t offset, int k,
                                 int stream_id, int n, uint32_t* out,
                                 float* gumbel, cudaStream_t stream);

/*
 * dspark_noise_words_folded -- the same diagnostic computed the way the
 * position, verification and sampler kernels compute their noise: the parts
 * of Philox4x32-10's first two rounds that depend only on the key and the
 * fixed counter words (k | stream << 16, offset lo, offset hi) are folded
 * into per-request constants, and the round keys are precomputed.  Its
 * words must equal dspark_noise_words' (and the published Philox4x32-10's)
 * bit for bit; arguments and errors are those of dspark_noise_words.
 */
DSPARK_API dspark_status dspark_noise_words_folded(uint64_t seed, uint64_t offset,
                                        int k, int stream_id, int n,
                                        uint32_t* out, float* gumbel,
                                        cudaStream_t stream);

/*
 * dspark_read_device_error -- copies the device error word of `workspace`
 * to the host (synchronising `stream`) and clears it.  Returns DSPARK_OK if
 * no kernel of the last call on this workspace recorded an error,
 * DSPARK_ERR_DEVICE (and *code != 0) if one did.  Every draft-block and
 * sampler call clears the word when it starts, so the code describes the
 * last call only; the calls on a cache never clear its word (control), which
 * this call reads likewise: their codes 2 and 6 to 12 are described there.
 * Codes: 1 a d0 outside [0, V) (token 0 used), 2 a bounded
 * wait inside a kernel ran out, 3 a per-request temperature that is not
 * finite and positive (1 used), 4 a proposal slot outside [0, num_slots),
 * 5 a sampler position outside [0, 65535] (0 used).  Synchronises
 * `stream`.
 */
DSPARK_API dspark_status dspark_read_device_error(void* workspace, int* code,
                                       cudaStream_t stream);

/* Human-readable name of a status. */
DSPARK_API const char* dspark_status_string(dspark_status status);

/* Library version, "major.minor.patch". */
DSPARK_API const char* dspark_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DSPARK_H_ */
