/*
 * Exact IO-aware softmax attention for NVIDIA GB300 (sm_103a): C ABI.
 *
 * What is computed (per batch b and head h, with s = `scale`):
 *   S = s Q K^T, masked;  P = softmax_rows(S);  O = P V;  LSE = logsumexp_rows(S)
 * and, for an upstream gradient dO of O,
 *   D = rowsum(dO * O), dV = P^T dO, dP = dO V^T, dS = P * (dP - D),
 *   dQ = s dS K, dK = s dS^T Q.
 *
 * How it is computed follows the FlashAttention practice record ("Why
 * recomputation is cheaper here than storing", Anthology of the SOTA): score
 * tiles live only in on-chip memory and are consumed at once with a running
 * row maximum and normaliser, the N x N matrix is never written to HBM, and the
 * backward pass rebuilds every S/P tile from Q, K, V and the saved per-row
 * statistics. Those statistics are the running maximum m and normaliser l of
 * "FlashAttention Algorithm > Recomputation Strategy" (section "What Gets
 * Stored vs Recomputed"), folded here into one value LSE = m + ln l.
 *
 * Conventions shared by every entry point (the _qk, _varlen and _split entry
 * points below state how their shapes differ):
 *  - Tensors Q, K, V, O, dO, dQ, dK, dV are contiguous [B, H, N, d] bf16 in
 *    device memory, d innermost; every base pointer 16-byte aligned.
 *    LSE is contiguous [B, H, N] fp32 (natural log). kv_len, when given, is
 *    a device int32 [B]: key j of batch b is valid iff j < kv_len[b].
 *  - d must be 64 or 128. N >= 0 (any value; N = 0 is a no-op). B, H >= 1.
 *    causal = 1 keeps key j for query i iff j <= i (with N_q query and N_k key
 *    rows, fa_forward_qk: iff j <= i + N_k - N_q).
 *  - All memory is owned by the caller. The library allocates nothing and
 *    frees nothing; outputs are fully overwritten.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default
 *    stream). A non-OK return means nothing was launched, except FA_ERR_CUDA
 *    after a failed launch.
 *  - Inside the kernels every wait is bounded; a wait that runs out records
 *    FA_ERR_TIMEOUT in a per-device status word that
 *    fa_get_last_device_status() reads (fa_get_last_device_status_detail()
 *    also says where). An argument that only the kernels can
 *    check (a packed sequence longer than max_seqlen) records
 *    FA_ERR_DEVICE_CHECK there; so does a failed bounds check in the
 *    bounds-checked build of this library (fa_debug.h). A recorded check does
 *    not affect other calls; a recorded timeout makes kernels give up at their
 *    next long wait until the word is read.
 *  - Entry points are reentrant; calls that share output buffers race.
 */
#ifndef IO_AWARE_EXACT_FA_H
#define IO_AWARE_EXACT_FA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define FA_API __attribute__((visibility("default")))
#else
#define FA_API
#endif

typedef struct CUstream_st* fa_stream_t; /* identical to cudaStream_t */

typedef enum {
  FA_OK = 0,
  FA_ERR_INVALID_ARG = 1,  /* null pointer, negative size, bad flag, too-small workspace */
  FA_ERR_UNSUPPORTED = 2,  /* d not in {64, 128}, B*H > 65535, or N beyond 32-bit indexing */
  FA_ERR_MISALIGNED = 3,   /* a tensor base pointer not 16-byte aligned */
  FA_ERR_CUDA = 4,         /* a CUDA runtime/driver call failed */
  FA_ERR_TIMEOUT = 5,      /* (device status) a bounded wait inside a kernel ran out */
  FA_ERR_DEVICE_CHECK = 6  /* (device status) an in-kernel consistency check failed */
} fa_status;

/* Forward pass: O and LSE from Q, K, V.
 * Defined by the practice record's account of the tiled kernel (scores kept on
 * chip and consumed immediately, blockwise running-maximum softmax) and by the
 * handbook's list of what is stored for the backward pass (O plus the per-row
 * running statistics). Returns an fa_status. */
FA_API int fa_forward(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N, int d,
               float scale, int causal, fa_stream_t stream);

/* As fa_forward, with optional key padding: kv_len is NULL or a device int32
 * [B] of valid key counts (values are clamped to [0, N]). A query row with no
 * valid key gets O = 0 and LSE = -inf. */
FA_API int fa_forward_ex(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N, int d,
                  float scale, int causal, const int32_t* kv_len, fa_stream_t stream);

/* As fa_forward_ex, with query and key lengths that may differ: q and o are
 * [B, H, Nq, d], k and v [B, H, Nk, d], lse [B, H, Nq]; kv_len values are
 * clamped to [0, Nk]. With causal = 1 the queries stand for the last Nq
 * positions of the keys' sequence: query row i keeps key j iff
 * j <= i + Nk - Nq (for Nq = Nk the pages' rule j <= i; the pages state only
 * that case). When Nq > Nk the first Nq - Nk rows keep no key and get O = 0,
 * LSE = -inf. Nq = 0 with Nk > 0 or the reverse returns FA_ERR_UNSUPPORTED;
 * both 0 is FA_OK with nothing to do. fa_forward_ex(.., N, ..) is exactly
 * fa_forward_qk(.., N, N, ..). */
FA_API int fa_forward_qk(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int Nq,
                         int Nk, int d, float scale, int causal, const int32_t* kv_len, fa_stream_t stream);

/* Forward pass over packed sequences of different lengths (variable-length
 * batches with no padding): B sequences, each its own attention problem with
 * N = len_b query and key rows (the pages' masks per sequence: causal j <= i).
 *  - Layout: q, k, v, o are [H, T, d] bf16 with every head's rows of all
 *    sequences packed back to back; lse is [H, T] fp32. Sequence b has rows
 *    [cu_seqlens[b], cu_seqlens[b + 1]) of every head.
 *  - cu_seqlens: device int32 [B + 1], non-decreasing, cu_seqlens[0] = 0,
 *    cu_seqlens[B] = T. max_seqlen: host upper bound of every length; it sizes
 *    the grid. A longer sequence is not fully computed and records
 *    FA_ERR_DEVICE_CHECK in the device status word.
 *  - A sequence of length 0 writes nothing. */
FA_API int fa_forward_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                             const int32_t* cu_seqlens, int B, int H, int T, int max_seqlen, int d, float scale,
                             int causal, fa_stream_t stream);

/* Backward of fa_forward_varlen: q, k, v, o, dO, dq, dk, dv are [H, T, d] bf16,
 * lse [H, T] fp32, sequences as in the forward call (same cu_seqlens,
 * max_seqlen, scale and causal). workspace: fa_backward_varlen_workspace_size
 * bytes, 256-byte aligned, contents on entry irrelevant. A sequence longer
 * than max_seqlen records FA_ERR_DEVICE_CHECK. */
FA_API int fa_backward_varlen(const void* q, const void* k, const void* v, const void* o, const void* dO,
                              const float* lse, void* dq, void* dk, void* dv, const int32_t* cu_seqlens, int B, int H,
                              int T, int max_seqlen, int d, float scale, int causal, void* workspace,
                              size_t workspace_bytes, fa_stream_t stream);

/* Workspace bytes of fa_backward_varlen: per head, -D and a base-2 LSE for
 * T + 4 B + 256 rows (each sequence's rows start on a 16-byte boundary) and
 * an fp32 dQ accumulator of T rows rounded up to 128. 0 for invalid arguments. */
FA_API size_t fa_backward_varlen_workspace_size(int B, int H, int T, int d);

/* Forward pass for inference shapes: few query rows over many keys, where one
 * CTA per (head, query-tile pair) leaves most SMs idle (the pages: inference
 * workloads are mostly memory-bound). The key tiles of each work item are cut
 * into n_split near-equal shares run by separate CTAs. Each writes its share's O
 * (divided by its own normaliser, fp32) and LSE into `workspace`. A second
 * kernel joins the shares with the running-maximum rescaling that the tiled
 * softmax applies between key blocks. Shapes, masks and results as
 * fa_forward_qk. With Nq <= 8 (decode) a streaming kernel on the CUDA cores
 * runs instead (one query row would waste a 128-row tensor-core tile). It
 * takes the 128-key tiles of all heads as one sequence. With n_split = 1 each
 * CTA takes ceil(B * H / min(#SMs, 256)) whole heads and writes their O and LSE
 * directly (no second kernel, the workspace is not touched). With n_split > 1
 * each of G = min(#SMs, 256, n_split * B * H) CTAs takes an equal run of the
 * sequence; a head whose tiles all fall to one CTA is written directly, the
 * partial results of a head split between CTAs go to the workspace and a
 * second kernel joins them. That second kernel runs whenever kv_len is given
 * (the tile counts are on the device) or some CTA's run starts inside a head.
 *  - lse may be NULL: then no LSE is written.
 *  - workspace: at least fa_forward_split_workspace_size(B, H, Nq, d, n_split)
 *    bytes, 256-byte aligned; its contents on entry do not matter.
 *  - n_split >= 1 (more than 1024 returns FA_ERR_UNSUPPORTED). With
 *    n_split = 1, Nq > 8 and lse non-NULL this is fa_forward_qk and the
 *    workspace is not touched. */
FA_API int fa_forward_split(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int Nq,
                            int Nk, int d, float scale, int causal, const int32_t* kv_len, int n_split,
                            void* workspace, size_t workspace_bytes, fa_stream_t stream);

/* Workspace bytes of fa_forward_split: 2 * n_split * B * H * Nq rows of d + 1 fp32
 * (the decode kernel uses 2 G * Nq of them, G <= n_split * B * H).
 * Returns 0 for invalid arguments. */
FA_API size_t fa_forward_split_workspace_size(int B, int H, int Nq, int d, int n_split);

/* The library's choice of n_split for a shape on the current device. For
 * Nq <= 8 (the decode kernel): 1 (whole heads a CTA) when 2 * B * H >= SMs, else
 * ceil(SMs / (B * H)), at most 64, so that the decode kernel runs one CTA per SM.
 * Otherwise it is 1 when B * H * ceil(Nq / 256) work items
 * already reach the SM count, else the largest count whose CTAs fit in two
 * waves (floor(2 * SMs / items)), capped at ceil(Nk / 128) / 4 (four key tiles
 * a share) and at 64. */
FA_API int fa_forward_split_count(int B, int H, int Nq, int Nk, int d);

/* Bytes of device workspace fa_backward needs: per (b, h), D and a base-2
 * copy of LSE for every query row and an fp32 dQ accumulator, each padded to
 * a multiple of 128 rows. Linear in N. Returns 0 for unsupported d. */
FA_API size_t fa_backward_workspace_size(int B, int H, int N, int d);

/* Backward pass: dQ, dK, dV from Q, K, V, O, dO and the LSE saved by the
 * forward pass. No N x N input exists: every S and P tile is recomputed from
 * Q, K and LSE, as the practice record and the handbook ("What Gets Stored vs
 * Recomputed", and the closing paragraph of that section: tiles rebuilt with
 * the forward's tiling, gradients computed per block and accumulated) describe.
 * `workspace` is caller-owned device memory of at least
 * fa_backward_workspace_size(B, H, N, d) bytes, 256-byte aligned; its
 * contents on entry do not matter. `scale` and `causal` must equal the
 * forward call's. */
FA_API int fa_backward(const void* q, const void* k, const void* v, const void* o, const void* dO, const float* lse,
                void* dq, void* dk, void* dv, int B, int H, int N, int d, float scale, int causal, void* workspace,
                size_t workspace_bytes, fa_stream_t stream);

/* As fa_backward, with the same optional key padding as fa_forward_ex. */
FA_API int fa_backward_ex(const void* q, const void* k, const void* v, const void* o, const void* dO, const float* lse,
                   void* dq, void* dk, void* dv, int B, int H, int N, int d, float scale, int causal,
                   const int32_t* kv_len, void* workspace, size_t workspace_bytes, fa_stream_t stream);

/* Backward of fa_forward_qk: q, o, dO, dq are [B, H, Nq, d], k, v, dk, dv
 * [B, H, Nk, d], lse [B, H, Nq]; the same masking as the forward call. The
 * workspace is fa_backward_workspace_size(B, H, Nq, d) bytes (it holds
 * per-query-row data only). fa_backward_ex(.., N, ..) is exactly
 * fa_backward_qk(.., N, N, ..). */
FA_API int fa_backward_qk(const void* q, const void* k, const void* v, const void* o, const void* dO,
                          const float* lse, void* dq, void* dk, void* dv, int B, int H, int Nq, int Nk, int d,
                          float scale, int causal, const int32_t* kv_len, void* workspace, size_t workspace_bytes,
                          fa_stream_t stream);

/* One stage of fa_backward_ex, same arguments; running stages 0, 1, 2 in
 * order on one stream is exactly fa_backward_ex. Exposed so that each kernel
 * can be timed on its own.
 *   0: -D = -rowsum(dO * O) and -LSE in base 2 per query row, into the workspace;
 *      zeroes the fp32 dQ accumulator.
 *   1: the recomputing kernel: dK and dV written, dQ accumulated in fp32.
 *   2: the fp32 dQ accumulator rounded to bf16 into dq.
 * Any other stage value returns FA_ERR_INVALID_ARG. */
FA_API int fa_backward_stage(int stage, const void* q, const void* k, const void* v, const void* o, const void* dO,
                             const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                             float scale, int causal, const int32_t* kv_len, void* workspace,
                             size_t workspace_bytes, fa_stream_t stream);

/* One stage of fa_backward_qk (stages as for fa_backward_stage). */
FA_API int fa_backward_stage_qk(int stage, const void* q, const void* k, const void* v, const void* o,
                                const void* dO, const float* lse, void* dq, void* dk, void* dv, int B, int H,
                                int Nq, int Nk, int d, float scale, int causal, const int32_t* kv_len,
                                void* workspace, size_t workspace_bytes, fa_stream_t stream);

/* Backward pass for callers that cannot allocate device memory: no workspace
 * argument. The pages have no counterpart of this entry point; it exists for
 * callers that are handed only their input and output buffers and may not
 * call cudaMalloc (for example a runtime that reserves all device memory up
 * front and gives a plugin nothing else). Instead of a caller's workspace it
 * uses one fixed scratch array compiled into the library, of
 * fa_backward_noalloc_max_bytes() bytes (32 MiB) on every GPU that loads the
 * library, held until the process exits.
 *  - Same arguments and results as fa_backward_ex without the workspace; the
 *    same argument checks come first, in the same order.
 *  - A valid shape whose workspace (fa_backward_workspace_size) exceeds the
 *    array returns FA_ERR_UNSUPPORTED before anything runs;
 *    fa_last_error_detail() then says how many bytes it needed.
 *  - Allocates nothing. The first call on each device (and context) looks up
 *    the array's device address (cudaGetSymbolAddress) with that device
 *    current; make that first call before any stream capture. A device
 *    ordinal of 64 or more returns FA_ERR_UNSUPPORTED.
 *  - All calls on a device share the one array: calls whose kernels overlap on
 *    the GPU (other streams, other host threads) race and corrupt each other's
 *    gradients. Serialise them. Each call re-initialises what it needs. */
FA_API int fa_backward_noalloc(const void* q, const void* k, const void* v, const void* o, const void* dO,
                               const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                               float scale, int causal, const int32_t* kv_len, fa_stream_t stream);

/* Size in bytes of the scratch array fa_backward_noalloc uses. */
FA_API size_t fa_backward_noalloc_max_bytes(void);

/* ---------------------------------------------------------------- serving
 * Attention of whole prompts and of drafted tokens over a cache in pages, and
 * the cache's own work. The pages state attention for equal heads over whole
 * rows only; these entry points compute the same softmax(s Q K^T) V, with
 * grouped heads, packed token-major rows and masks as stated at each.
 *
 * Conventions of these entry points, besides those above:
 *  - Types: FA_BF16 or FA_FP16, the same for every tensor of a call.
 *  - Grouped heads: Hq query heads share Hkv key/value heads, Hq a multiple of
 *    Hkv and Hq / Hkv <= 128; query head h reads key/value head h / (Hq / Hkv).
 *  - Rounding: scores, maxima, sums, LSE and O are fp32, O is rounded once to the
 *    type; the probabilities are rounded to the type before their product with V
 *    (each by half a step, eps / 2 of itself; in fp16 below 2^-23 of the row's
 *    largest by up to 2^-34 of that one), the sum that divides O is not.
 *  - Tokens of all sequences are packed back to back: sequence b has the tokens
 *    [cu[b], cu[b + 1]), cu a device int32 [B + 1], non-decreasing from 0. cu[B]
 *    may be less than T: the rows behind it are neither read for a result nor
 *    written. cu is read on the device only, so that a captured call can be
 *    replayed with other lengths.
 *  - A value that only the kernels can check (an offset that decreases or passes
 *    T, a length that passes the page table, a page id outside the cache) records
 *    FA_ERR_DEVICE_CHECK in the device status word. Nothing outside the given
 *    tensors is read or written; what the call says below happens instead.
 *    Where offsets decrease, rows that two sequences claim hold either's result.
 *  - Each entry point is called once on a device before it is captured there. */
typedef enum { FA_BF16 = 0, FA_FP16 = 1 } fa_dtype;

/* Rows of [T, H, d] tokens: d contiguous, strides in elements, both positive
 * multiples of 8 (the rows of a wider projection, say); data 16-byte aligned. */
typedef struct {
  void* data;
  int64_t token_stride, head_stride;
} fa_rows;

/* A cache in pages: K and V of shape [n_pages, Hkv, page_size, d], d contiguous,
 * with the same strides (elements, positive multiples of 8; any order of the
 * other dimensions), 16-byte aligned. page_size is 16, 32, 64, 128 or 256.
 * table: device int32, row b (table_stride entries apart, table_width of them
 * used) lists the pages of sequence b: token i lies in page
 * table[b][i / page_size] at place i % page_size. */
typedef struct {
  void *k, *v;
  int64_t page_stride, head_stride, token_stride;
  int32_t n_pages, page_size;
  const int32_t* table;
  int64_t table_stride;
  int32_t table_width;
} fa_pages;

/* Causal attention of whole prompts: token i of a sequence attends to the tokens
 * j <= i of the same sequence. q and o are [T, Hq, d], k and v [T, Hkv, d], lse
 * [Hq, T] fp32 (NULL: not written). Sequences may have any length, 0 and 1 too.
 * What lies in rows of k and v behind a sequence's end (other sequences, padding)
 * does not reach its results, whatever it holds; a NaN or infinity in V of a token
 * of the sequence itself may reach earlier tokens of the same key/value head, those
 * less than 128 + 128 Hkv / Hq (rounded down) before it.
 * Decreasing offsets or ones past T record FA_ERR_DEVICE_CHECK; the sequence is
 * then cut to the tokens that exist. */
FA_API int fa_forward_prompt(const fa_rows* q, const fa_rows* k, const fa_rows* v, const fa_rows* o, float* lse,
                             const int32_t* cu_seqlens, int B, int T, int Hq, int Hkv, int d, int dtype, float scale,
                             fa_stream_t stream);

/* Attention of drafted tokens ("nodes") over a cache in pages and over each
 * other. Sequence b has lens[b] tokens in the cache (device int32 [B]) and the
 * nodes [cu[b], cu[b + 1]), whose queries, keys and values are the packed rows
 * q [T, Hq, d], k and v [T, Hkv, d]; the nodes are not in the cache. Every node
 * attends to all lens[b] cached tokens, and
 *  - mask = NULL: to the nodes j <= i of its sequence (a chain; one node is plain
 *    decoding, many are a further part of a prompt);
 *  - mask given: to the nodes whose bits are set: mask is a device uint32
 *    [T, mask_words], bit j % 32 of word j / 32 of a node's row is node j of its
 *    sequence (fa_tree_mask makes it from parents). Any bits may be set; those at
 *    or past the sequence's number of nodes, and nodes past 32 mask_words, count
 *    as not set.
 * A NaN or infinity in V of a node may reach nodes of its sequence, of the same
 * key/value head, that do not see it.
 * A node that sees nothing gets O = 0 and LSE = -inf. o is [T, Hq, d], lse
 * [Hq, T] fp32 (NULL: not written). A sequence without nodes writes nothing, and
 * its length and pages are not looked at. What lies in the cache past lens[b]
 * does not reach the results, whatever it holds.
 * A length outside [0, table_width * page_size] is taken as the nearest one
 * inside, a page id outside [0, n_pages) as a page of zeros, and either records
 * FA_ERR_DEVICE_CHECK.
 * workspace: fa_forward_tree_workspace_size bytes, 256-byte aligned, contents on
 * entry irrelevant; calls that may overlap need one each. */
FA_API int fa_forward_tree(const fa_rows* q, const fa_rows* k, const fa_rows* v, const fa_rows* o, float* lse,
                           const fa_pages* cache, const int32_t* lens, const int32_t* cu_nodes, const uint32_t* mask,
                           int mask_words, int B, int T, int Hq, int Hkv, int d, int dtype, float scale,
                           void* workspace, size_t workspace_bytes, fa_stream_t stream);

/* Workspace bytes of fa_forward_tree on the current device: two partial results
 * of 256 rows, and 32 bytes, for each SM. 0 for an unsupported d. */
FA_API size_t fa_forward_tree_workspace_size(int d);

/* Which nodes a node of a tree sees: itself and its ancestors. parents: device
 * int32 [T], for each node its parent's index within its sequence, less than its
 * own, or negative for a root. mask: device uint32 [T, mask_words] as
 * fa_forward_tree reads it. A parent at or past the node's own index counts as a
 * root and records FA_ERR_DEVICE_CHECK; so does a sequence of more than
 * 32 mask_words nodes, whose bits past them are left out. */
FA_API int fa_tree_mask(const int32_t* parents, const int32_t* cu_nodes, uint32_t* mask, int mask_words, int B, int T,
                        fa_stream_t stream);

/* Writes tokens into their pages: token i of sequence b goes to position
 * start[b] + i of the cache (start: device int32 [B]). k and v are [Tkv, Hkv, d];
 * the token's row is cu[b] + i, or rows[cu[b] + i] where rows (device int32, T
 * entries) is given: the accepted nodes of a draft, say. T: the rows of k and v
 * without rows, the entries of rows with it. A token whose position, page id or
 * row lies outside is left out and records FA_ERR_DEVICE_CHECK. Tokens that name
 * the same place race. */
FA_API int fa_cache_append(const fa_rows* k, const fa_rows* v, const fa_pages* cache, const int32_t* start,
                           const int32_t* cu, const int32_t* rows, int B, int T, int Tkv, int Hkv, int d,
                           fa_stream_t stream);

/* The page tables of a cache with `planes` planes (K and V of every layer) that
 * share them: plane x lies plane_stride elements after plane 0, each of shape
 * [n_pages, Hkv, page_size, d], contiguous, 16-bit elements, 16-byte aligned. */
typedef struct {
  void* data;
  int64_t plane_stride;
  int32_t planes, n_pages, Hkv, page_size, d;
  int32_t* table;  /* [slots, table_width] pages of each slot */
  int32_t* lens;   /* [slots] tokens of each slot */
  int32_t slots, table_width;
} fa_pool;

/* Every slot s becomes the first min(new_lens[s], lens[src[s]]) tokens of slot
 * src[s] as it was before the call, with pages for new_lens[s] tokens: src[s] = s
 * keeps, trims (a shorter new_lens), frees (0) or grows a slot; another src forks
 * it, and a permutation reorders beams. Pages that only hold kept tokens are
 * shared. The page in which the next token would be written, where some of its
 * tokens are kept, is the slot's own afterwards: it stays if src[s] = s and no
 * other slot keeps it, else its kept tokens are copied (in every plane) to a new
 * page. New pages come from those free before the call, lowest id first, in the
 * order of the slots. A page is in use while some slot's table lists it among the
 * first ceil(lens / page_size) entries; nothing else records that.
 * table and lens are updated in place, table entries behind a slot's pages become
 * -1. info: device int32 [2], the pages needed and the pages free; where more are
 * needed than free, nothing else is changed. A src outside [0, slots), a length
 * (old or new) outside [0, table_width * page_size] or a listed page id outside
 * [0, n_pages) records FA_ERR_DEVICE_CHECK, info becomes {-1, -1}, and nothing
 * else is changed. workspace: fa_cache_workspace_size bytes, 256-byte aligned. */
FA_API int fa_cache_update(const fa_pool* pool, const int32_t* src, const int32_t* new_lens, int32_t* info,
                           void* workspace, size_t workspace_bytes, fa_stream_t stream);

/* Moves the pages in use to the lowest ids: with n of them in use, the r-th page
 * in use at or past n (by id) moves, in every plane, to the r-th page below n that
 * is free, and the tables follow; entries behind a slot's pages are left as they
 * are. info: device int32 [2], the pages in use and the pages moved. Lengths and
 * page ids outside their ranges as for fa_cache_update. */
FA_API int fa_cache_compact(const fa_pool* pool, int32_t* info, void* workspace, size_t workspace_bytes,
                            fa_stream_t stream);

/* Workspace bytes of fa_cache_update and fa_cache_compact. 0 for invalid sizes. */
FA_API size_t fa_cache_workspace_size(int n_pages, int slots, int table_width);

/* ---- a cache in 8 bits
 * K and V of a cache in pages (fa_pages) as e4m3, strides in elements, positive
 * multiples of 16, with a positive fp32 scale for each block of `block` tokens of a
 * page and head (16, 32, 64, 128 or 256, at most the page size): an element stands
 * for its value times scale[page * page_stride + head * head_stride + i], i = place
 * in the page / block. The same strides for k and v. */
typedef struct {
  float *k, *v;
  int64_t page_stride, head_stride;
  int32_t block;
} fa_scales;

/* fa_forward_tree over a cache in 8 bits: the queries, the nodes' keys and values
 * and O are of the type `dtype`, the cached ones e4m3 with their blocks' scales.
 * As there otherwise, but for what is said here.
 *  - Rounding: scores and sums are fp32. An element of a query takes part with its bits
 *    down to 2^-21 of its row's largest; in bf16 with many rows that of a query, or of a
 *    node's key or value, with those down to 2^-38 of the largest of the rows it is taken
 *    with (32 at most). A probability times the scale of its value's block is rounded
 *    once, by half a step of the type at most, or by 2^-32 (in bf16 with few rows 2^-30) of
 *    the product of the row's largest probability and the sequence's and head's largest
 *    such scale, whichever is more. With many rows that concerns nodes' values too: their
 *    scale is 1, or in bf16 the power of two that brings the largest element of 32 rows
 *    from [2^14, 2^15) to what it is. Which of the kernels runs follows from B, T,
 *    Hq / Hkv, d and dtype alone: a batch that is mostly sequences without nodes is best
 *    given without those.
 *  - A NaN in the cache reaches the rows that see it. Scales have to be positive, normal
 *    and finite; others give undefined results, of their own sequence and head only. From
 *    2^80 on (keys and values from 2^88 on) sums may pass fp32's range: the row is then
 *    infinite or NaN. An infinity in a query makes the row NaN, as scores of -inf alone do.
 * workspace: fa_forward_tree_8bit_workspace_size bytes, 256-byte aligned. */
FA_API int fa_forward_tree_8bit(const fa_rows* q, const fa_rows* k, const fa_rows* v, const fa_rows* o, float* lse,
                                const fa_pages* cache, const fa_scales* scales, const int32_t* lens,
                                const int32_t* cu_nodes, const uint32_t* mask, int mask_words, int B, int T, int Hq,
                                int Hkv, int d, int dtype, float scale, void* workspace, size_t workspace_bytes,
                                fa_stream_t stream);

/* Workspace bytes of fa_forward_tree_8bit on the current device. 0 for an unsupported d. */
FA_API size_t fa_forward_tree_8bit_workspace_size(int d);

/* fa_cache_append into a cache in 8 bits: k and v of the type `dtype`. How a token is
 * held: in a block none of whose tokens lies before the call's first one there, the
 * scale becomes 2^i with the least i >= -118 that brings the largest magnitude of the
 * block's new tokens (of that head, of K or of V) to 448 at most. Where tokens lie
 * before it they stay, and the scale s becomes 2^i s with the least such i >= 0; for
 * i > 0 their elements are rounded again, to 2^-i of themselves. (A scale there that
 * is no positive, normal number is taken as none; those elements stay as they are.) An
 * element is rounded once, from its value times the reciprocal of the scale, to the
 * nearest e4m3, ties to even. NaN and infinities become NaN and count for no scale.
 * Other elements of the pages and other blocks' scales are left as they are. A
 * sequence's blocks that the call touches must belong to no other sequence of it. */
FA_API int fa_cache_append_8bit(const fa_rows* k, const fa_rows* v, const fa_pages* cache, const fa_scales* scales,
                                const int32_t* start, const int32_t* cu, const int32_t* rows, int B, int T, int Tkv,
                                int Hkv, int d, int dtype, fa_stream_t stream);

/* The rotation of queries and keys by the angles of their positions. angles: fp32,
 * `positions` rows of `dim` values (row_stride apart, a multiple of 4; 16-byte aligned):
 * the cosines of the position's dim / 2 angles, then their sines. dim is a multiple
 * of 16, at most d. With pair j of a head being elements (j, j + dim / 2), or
 * (2j, 2j + 1) if interleaved,
 *   (x1, x2) -> (x1 cos - x2 sin, x2 cos + x1 sin)
 * in fp32, each product and sum rounded; elements from dim on stay. at: device int32
 * [T], each token's position for the angles, or NULL: its position in the cache. */
typedef struct {
  const float* angles;
  int64_t row_stride;
  int32_t positions, dim, interleaved;
  const int32_t* at;
} fa_rotary;

/* The rotation of new tokens, and their way into the cache, in one pass. q [T, Hq, d]
 * (NULL: none, with q_out NULL) and k [T, Hkv, d] are rotated and rounded once to the
 * type, into q_out and k_out (k_out may be NULL; either may be its input, and must not
 * overlap it otherwise); the rotated keys and v [T, Hkv, d] go into the pages as
 * fa_cache_append (scales NULL) or fa_cache_append_8bit (from the rotated keys in fp32)
 * writes them: token i of sequence b to position start[b] + i. cache NULL: only
 * the rotation; v, scales, start are not looked at then, rotary->at is needed, and
 * cu may be NULL (every row is a token).
 * A token whose position lies outside the angles is left out altogether and records
 * FA_ERR_DEVICE_CHECK; one whose position or page in the cache lies outside is still
 * rotated. Rows behind cu[B] are left as they are. */
FA_API int fa_rotary_append(const fa_rows* q, const fa_rows* k, const fa_rows* v, const fa_rows* q_out,
                            const fa_rows* k_out, const fa_pages* cache, const fa_scales* scales,
                            const fa_rotary* rotary, const int32_t* start, const int32_t* cu, int B, int T, int Hq,
                            int Hkv, int d, int dtype, fa_stream_t stream);

/* The scales of a pool in 8 bits: plane x's lie plane_stride elements after plane 0's,
 * each [n_pages, Hkv, blocks] fp32, contiguous. */
typedef struct {
  float* data;
  int64_t plane_stride;
  int32_t blocks; /* page_size / block */
} fa_pool_scales;

/* fa_cache_update and fa_cache_compact of a pool whose elements have 8 bits
 * (plane_stride a multiple of 16): pages are copied and moved with their scales. A
 * page of which some tokens are copied takes the scales of the blocks that hold them. */
FA_API int fa_cache_update_8bit(const fa_pool* pool, const fa_pool_scales* scales, const int32_t* src,
                                const int32_t* new_lens, int32_t* info, void* workspace, size_t workspace_bytes,
                                fa_stream_t stream);
FA_API int fa_cache_compact_8bit(const fa_pool* pool, const fa_pool_scales* scales, int32_t* info, void* workspace,
                                 size_t workspace_bytes, fa_stream_t stream);

/* Static text for an fa_status value. */
FA_API const char* fa_status_string(int status);

/* Synchronises `stream`, then returns and clears the current device's status
 * word: FA_OK if no kernel recorded an error, else FA_ERR_TIMEOUT if some wait
 * ran out, else FA_ERR_DEVICE_CHECK. A failure of the CUDA
 * calls this makes returns FA_ERR_CUDA (fa_last_error_detail names it); a
 * device ordinal of 64 or more returns FA_ERR_UNSUPPORTED. The word's device
 * address is looked up once per device and context; after cudaDeviceReset the
 * next call looks it up again. */
FA_API int fa_get_last_device_status(fa_stream_t stream);

/* As fa_get_last_device_status; if detail is non-NULL it also receives 4 ints
 * describing the first recorded error of that code: code, site (which wait or check),
 * blockIdx.x, blockIdx.y (all 0 when none was recorded). */
FA_API int fa_get_last_device_status_detail(fa_stream_t stream, int* detail);

/* For the calling host thread: text naming the CUDA call that made the last
 * FA_ERR_CUDA return and its error (or the reason for a size rejection by
 * fa_backward_noalloc), or "" if none has. Static storage. */
FA_API const char* fa_last_error_detail(void);

/* Library version as major*10000 + minor*100 + patch. */
FA_API int fa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* IO_AWARE_EXACT_FA_H */
