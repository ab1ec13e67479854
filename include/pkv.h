/*
 * pkv.h -- C ABI of the paged KV-cache attention library (GB300, sm_103a).
 *
 * The operations are those of a nano-vllm style engine's attention layer:
 *   - the KV-cache store through a slot mapping, which nano-vllm performs with
 *     a Triton kernel (nano-vllm hub page, pomoai.com, "core tech 2:
 *     Attention + Triton kernel");
 *   - attention over the paged cache, with fixed 256-token blocks managed by a
 *     block manager (same page, "core tech 4: KV Cache block manager") and a
 *     per-sequence block table mapping logical to physical blocks (CSDN essay
 *     "from nanoVLLM to vLLM", Mountain 1: KV cache);
 *   - separate kernels for the compute-dense prefill phase and the
 *     memory-bound decode phase (same essay, Mountain 3 and the study route's
 *     attention/ module notes).
 * The result of both attention calls is that of standard attention,
 * softmax(q K^T * scale) V: FlashAttention-style tiling only reorders the
 * computation (same essay, Mountain 3).
 *
 * Conventions shared by every call
 * --------------------------------
 *  - bf16 tensors are passed as pointers to their 16-bit patterns.
 *  - Every pointer argument except `dev_status` and `stream` is a DEVICE
 *    pointer owned by the caller; no call allocates memory or keeps a
 *    reference after it returns.  The library caches small per-device tables
 *    (the SM count) and, loaded on a GPU, holds one fixed 16 MiB device array
 *    (the scratch of pkv_paged_decode_attn_noalloc).
 *  - Layouts (all row-major, contiguous):
 *      q             [T_q, Hq, D]
 *      k, v          [T_new, Hkv, D]   (token stride configurable in kv_store)
 *      k_cache       [num_blocks, block_size, Hkv, D]; one slot = Hkv*D values
 *      v_cache       same as k_cache
 *      out           [T_q, Hq, D]
 *      block_tables  int32 [num_seqs, max_blocks_per_seq], unused entries -1
 *      slot_mapping  int32 [T_new]; slot = block * block_size + offset; -1 = skip
 *      context_lens  int32 [num_seqs]; keys visible, INCLUDING the tokens just
 *                    stored
 *      cu_seqlens_q  int32 [num_seqs+1], prefix sums of new-token counts
 *      cu_seqlens_k  int32 [num_seqs+1], prefix sums of (cached + new) counts
 *      key_weights   fp32 [num_blocks, Hkv, block_size]: for each slot and kv
 *                    head, the attention weight its key has received so far
 *  - GQA: query head h reads kv head h / (Hq / Hkv).
 *  - Pointers to bf16 data must be 16-byte aligned.
 *  - Every call is asynchronous on `stream` (a cudaStream_t; NULL = the
 *    legacy default stream).  Host-side argument checks run before any
 *    launch: a failed check returns a status and launches nothing.
 *  - Data-dependent faults (a slot or block id out of range, an empty or
 *    oversize context) are caught by bounds checks on the device: the kernel
 *    skips the access, ORs a PKV_DEV_* bit into *dev_status (when dev_status is
 *    not NULL; it is a device int32) and finishes.  Nothing traps or spins
 *    without a limit; a wait that exceeds its limit sets PKV_DEV_TIMEOUT.
 */
#ifndef PKV_H_
#define PKV_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum pkv_status {
  PKV_OK = 0,
  PKV_ERR_INVALID_ARG = 1, /* null pointer, bad size, misaligned pointer */
  PKV_ERR_UNSUPPORTED = 2, /* head_dim, group size or block_size not built */
  PKV_ERR_WORKSPACE = 3,   /* workspace missing or too small */
  PKV_ERR_CUDA = 4,        /* a CUDA runtime/driver call or launch failed */
  PKV_ERR_OUT_OF_BLOCKS = 5 /* block manager: not enough free blocks (nothing changed) */
} pkv_status;

/* Bits OR-ed into *dev_status by the kernels. */
#define PKV_DEV_BAD_SLOT 0x1    /* slot_mapping entry outside [-1, NB*BS) */
#define PKV_DEV_BAD_BLOCK 0x2   /* block_tables entry outside [0, NB) */
#define PKV_DEV_BAD_CONTEXT 0x4 /* context length <= 0 or > max_blocks*BS */
#define PKV_DEV_TIMEOUT 0x8     /* a bounded wait ran out */
#define PKV_DEV_WORKSPACE 0x10  /* decode: more blocks than max_total_blocks */
#define PKV_DEV_BAD_SEQLEN 0x20 /* prefill: bad cu_seqlens (n > len_k, n > max_seqlen_q) */
#define PKV_DEV_NO_BLOCKS 0x40  /* plan_step: too few free blocks, sequences were refused */

/* Human-readable name of a pkv_status value (static string). */
const char *pkv_status_string(int status);

/* ABI revision of this header; bumped on any signature change. */
int pkv_abi_version(void);

/*
 * kv_store -- write this step's new K and V rows into the paged cache.
 *
 * For every token t in [0, num_tokens) with s = slot_mapping[t] >= 0:
 *   k_cache slot s (Hkv*D values) <- k row t,  v_cache slot s <- v row t.
 * A bit copy: no arithmetic touches the values.  Slots equal to -1 are
 * skipped (padding); any other slot outside [0, num_blocks*block_size) sets
 * PKV_DEV_BAD_SLOT and is skipped.  Slots >= 0 must be unique.
 *
 * k_token_stride / v_token_stride: elements between consecutive tokens of k
 * and v (0 = Hkv*D, i.e. contiguous); must keep rows 16-byte aligned.
 * Requires (Hkv*D) % 8 == 0.
 */
pkv_status pkv_kv_store(const uint16_t *k, const uint16_t *v, uint16_t *k_cache,
                        uint16_t *v_cache, const int32_t *slot_mapping, int64_t num_tokens,
                        int num_kv_heads, int head_dim, int64_t k_token_stride,
                        int64_t v_token_stride, int64_t num_blocks, int block_size,
                        int32_t *dev_status, void *stream);

/*
 * Bytes of device workspace paged_decode_attn needs: a 256-byte work counter,
 * then the split-K scratch.  max_total_blocks is an upper bound the caller
 * guarantees on sum_s ceil(context_lens[s]/block_size) (num_seqs *
 * max_blocks_per_seq always works).  Returns 0 for invalid sizes
 * and for sizes whose workspace would not fit a size_t.
 */
size_t pkv_decode_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                 int64_t max_total_blocks);

/*
 * paged_decode_attn -- one query token per sequence against its paged K/V.
 *
 * out[s, h, :] = softmax_p(scale * <q[s,h,:], K_s[p, h/g, :]>) V_s[p, h/g, :]
 * over p in [0, context_lens[s]), where K_s[p] is the cache slot
 * block_tables[s][p / block_size] * block_size + p % block_size and
 * g = Hq / Hkv.  bf16 in, fp32 accumulation, bf16 out (round to nearest even).
 *
 * Split-K flash-decoding: each (sequence, kv head, block) is one work item
 * (two consecutive blocks per item when the batch has very many of them)
 * whose partial (max, sum, unnormalised output) goes to the workspace; the
 * persistent CTAs take items from a counter in the workspace as they become
 * free.  A second kernel, launched as a programmatic dependent of the first,
 * merges the partials of every sequence that spans more than one item.  Two
 * kernel launches per call (one when max_blocks_per_seq == 1).
 *
 * workspace: device buffer of at least pkv_decode_workspace_size(...) bytes,
 * 256-byte aligned, zero-filled once before its first use.  Its first 256
 * bytes hold the work counter, which every call leaves at zero (also a call
 * whose waits ran out); the rest needs no initialisation (each call writes
 * every entry before reading it).  Calls that overlap on the device must not
 * share a workspace.
 *
 * scale: any finite value (zero averages the context's values; a NaN or
 * infinite scale returns PKV_ERR_INVALID_ARG and launches nothing).
 *
 * Supported: head_dim in {64, 128}; Hq/Hkv in {1, 2, 4, 8}; block_size in
 * {64, 128, 256, 512}; num_seqs <= 16384, and the kernel's per-CTA shared
 * memory (which holds every sequence's block offset and length) must fit in
 * 227 KiB: only head_dim 128 with Hq/Hkv 8 and block_size 512 reaches that
 * limit first, at 16093 sequences.  A batch beyond either limit returns
 * PKV_ERR_UNSUPPORTED; sizes whose workspace cannot be addressed return
 * PKV_ERR_INVALID_ARG.  Both launch nothing.
 */
pkv_status pkv_paged_decode_attn(uint16_t *out, const uint16_t *q, const uint16_t *k_cache,
                                 const uint16_t *v_cache, const int32_t *block_tables,
                                 const int32_t *context_lens, int num_seqs, int num_q_heads,
                                 int num_kv_heads, int head_dim, int block_size,
                                 int max_blocks_per_seq, int64_t num_blocks,
                                 int64_t max_total_blocks, float scale, void *workspace,
                                 size_t workspace_bytes, int32_t *dev_status, void *stream);

/*
 * paged_decode_store_attn -- kv_store of this step's tokens fused with
 * paged_decode_attn, in the same launches as paged_decode_attn alone.
 *
 * A decode step stores one new token per sequence and then attends over the
 * whole context including it (nano-vllm hub page, "core tech 2": the layer
 * writes K/V through the slot mapping, then runs attention; CSDN essay
 * "from nanoVLLM to vLLM", Mountain 3).  Here new_k / new_v [num_seqs, Hkv, D]
 * (contiguous) hold, in row s, the token at position context_lens[s] - 1 of
 * sequence s, and slot_mapping[s] is its slot (-1: attend to it but do not
 * store it).  The result and the cache afterwards are bit-identical to
 * pkv_kv_store followed by pkv_paged_decode_attn: the work item that holds
 * the newest token takes that token's row from new_k / new_v and, after using
 * it, writes it to the cache; no other work item of the call reads that slot.
 *
 * Arguments, workspace and errors as for paged_decode_attn and kv_store
 * (slots out of range set PKV_DEV_BAD_SLOT and are not written).
 */
pkv_status pkv_paged_decode_store_attn(uint16_t *out, const uint16_t *q, const uint16_t *new_k,
                                       const uint16_t *new_v, const int32_t *slot_mapping,
                                       uint16_t *k_cache, uint16_t *v_cache,
                                       const int32_t *block_tables, const int32_t *context_lens,
                                       int num_seqs, int num_q_heads, int num_kv_heads,
                                       int head_dim, int block_size, int max_blocks_per_seq,
                                       int64_t num_blocks, int64_t max_total_blocks, float scale,
                                       void *workspace, size_t workspace_bytes,
                                       int32_t *dev_status, void *stream);

/*
 * paged_decode_attn_noalloc -- paged_decode_attn without a caller workspace.
 *
 * The pages have no counterpart to this call; it exists for callers of this
 * library that cannot allocate device memory for a workspace: code running
 * under a host framework whose allocator owns all device memory and offers no
 * hook, a plugin that may not allocate inside its host process, or a serving
 * loop that must keep cudaMalloc/cudaFree (which synchronise the device) off
 * its latency path.
 *
 * The split-K scratch lives in a fixed 16 MiB array in the library's own
 * device memory, which every GPU that loads the library holds until the
 * process exits.  A call whose workspace need,
 * pkv_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
 * max_total_blocks), exceeds 16 MiB returns PKV_ERR_WORKSPACE and launches
 * nothing.  The call itself allocates nothing.
 *
 * The first call on each device looks up the array's device address
 * (cudaGetSymbolAddress) with that device current; make that first call
 * before any stream capture.  Each call then runs the same kernels as
 * pkv_paged_decode_attn on that array.  The array is zero when the library
 * loads and keeps the previous call's contents: its work counter (the first
 * 256 bytes) is left at zero by every call, and the rest is written before it
 * is read.  All calls on a device share the one array, so
 * calls that overlap on the GPU (other streams, other host threads) race and
 * corrupt each other's results: serialise them.
 *
 * Arguments, layouts, results and errors are those of pkv_paged_decode_attn.
 */
pkv_status pkv_paged_decode_attn_noalloc(uint16_t *out, const uint16_t *q,
                                         const uint16_t *k_cache, const uint16_t *v_cache,
                                         const int32_t *block_tables,
                                         const int32_t *context_lens, int num_seqs,
                                         int num_q_heads, int num_kv_heads, int head_dim,
                                         int block_size, int max_blocks_per_seq,
                                         int64_t num_blocks, int64_t max_total_blocks,
                                         float scale, int32_t *dev_status, void *stream);

/*
 * test_decode_fault -- TEST-ONLY fault injection for the decode kernels'
 * bounded waits (the pages have no counterpart; it exists so that tests can
 * make a wait run out without faulting or hanging the GPU).
 *
 * Sets, for the current device, the wall-clock limit of every wait in the
 * decode kernels (default 1 s) and a tile number that every decode CTA's
 * producer then skips instead of loading (-1: none, the default).  A decode
 * call made while a tile is withheld waits out the limit, flags
 * PKV_DEV_TIMEOUT in *dev_status, leaves its output undefined and returns;
 * the device stays usable.  Restore with pkv_test_decode_fault(1000000000, -1).
 * Synchronous (it copies to device memory).  Returns PKV_ERR_INVALID_ARG for
 * wait_limit_ns <= 0 or withhold_tile < -1.
 */
pkv_status pkv_test_decode_fault(int64_t wait_limit_ns, int withhold_tile);

/*
 * paged_prefill_attn -- causal attention of packed variable-length prompts
 * over the paged cache, including an already-cached prefix.
 *
 * For sequence s: n = cu_seqlens_q[s+1] - cu_seqlens_q[s] new queries and
 * len_k = cu_seqlens_k[s+1] - cu_seqlens_k[s] keys, of which c = len_k - n
 * were cached before this step (their K/V, and the new tokens' K/V, must
 * already be in the cache: call kv_store first).  Query i sits at absolute
 * position c + i and attends to keys 0 .. c + i:
 *   out[cu_q[s]+i, h, :] = softmax_{p <= c+i}(scale * <q, K_s[p, h/g]>) V_s[p, h/g]
 * bf16 operands on the tcgen05 tensor cores, fp32 accumulation in tensor
 * memory, bf16 out.
 *
 * total_q = cu_seqlens_q[num_seqs]; max_seqlen_q bounds every n (a larger n
 * sets PKV_DEV_BAD_SEQLEN and its excess rows are not written).  A sequence
 * with n = 0 has no rows.  A sequence's rows do not depend on the other
 * sequences of the call or on their order (the kernel schedules the longest
 * contexts first; the result is the same bit for bit).
 *
 * workspace: device memory of at least pkv_prefill_workspace_size() bytes,
 * 256-byte aligned, zero-filled before its first use.  It holds the counter
 * from which the kernel's CTAs take their work; every call leaves it zeroed
 * again, so one zero-fill at allocation is enough.  Calls that may run at the
 * same time on the GPU (other streams, other host threads) need workspaces
 * of their own.  Missing, short or misaligned: PKV_ERR_WORKSPACE.
 *
 * scale: any finite value (a NaN or infinite scale returns
 * PKV_ERR_INVALID_ARG and launches nothing).
 *
 * Supported: head_dim in {64, 128}; Hq/Hkv in {1, 2, 4, 8};
 * block_size in {64, 128, 256, 512}.
 */
pkv_status pkv_paged_prefill_attn(uint16_t *out, const uint16_t *q, const uint16_t *k_cache,
                                  const uint16_t *v_cache, const int32_t *block_tables,
                                  const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                                  int num_seqs, int64_t total_q, int max_seqlen_q,
                                  int num_q_heads, int num_kv_heads, int head_dim,
                                  int block_size, int max_blocks_per_seq, int64_t num_blocks,
                                  float scale, void *workspace, size_t workspace_bytes,
                                  int32_t *dev_status, void *stream);

/* Bytes of device workspace pkv_paged_prefill_attn needs (any shape). */
size_t pkv_prefill_workspace_size(void);

/*
 * Key weights and eviction -- the pages' engine frees whole sequences when its
 * blocks run out (CSDN essay, Mountain 1: basic preemption, no swap); these
 * calls let a sequence go on in fewer blocks instead, by giving up the keys
 * that have received the least attention.  key_weights holds, beside every
 * key of the cache, the softmax weight it has received, summed over queries
 * and over the query heads of its kv head:
 *   pkv_paged_prefill_weights       adds the weights of a prompt chunk's last queries,
 *   pkv_paged_decode_weights_attn   attends one new token and adds its weights,
 *   pkv_kv_evict                    keeps the heaviest keys and the most recent.
 * A key's sum starts when its token arrives: the call that brings the token
 * sets the sum, later calls add to it, so key_weights needs no clearing when a
 * block changes hands.  Sums are fp32; a slot held by one sequence gets one
 * addition per call, so its sum does not depend on the order of anything.  A
 * block that several sequences of the batch share collects the weights of all
 * of them, by atomic additions whose order (hence last bit) can differ; a slot
 * that any of them brings is cleared before anything is added to it.  So the
 * owner of a prefix and those that find it cached may be in one call, in any
 * order.  A call that brings a token again (the last token of a prompt whose
 * blocks were all found, stored once more) starts its sum again; its row should
 * be the one that is there, since others of the call may read it before or
 * after a fused store.
 */

/*
 * Bytes of device workspace paged_decode_weights_attn needs (split-K partials
 * and the logits of max_total_blocks blocks).  Returns 0 for invalid sizes
 * and for sizes whose workspace would not fit a size_t.
 */
size_t pkv_decode_weights_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads,
                                         int head_dim, int block_size, int64_t max_total_blocks);

/*
 * paged_decode_weights_attn -- decode attention that collects key weights.
 *
 * out as for paged_decode_attn (with new_k, new_v and slot_mapping: as for
 * paged_decode_store_attn, storing the new tokens too; all three NULL: no
 * store), and with w[s,h,p] the softmax weight of query head h for position p,
 * a[s,j,p] = sum of w[s,h,p] over the heads h of kv head j's group:
 *   key_weights(slot of p, j) += a[s,j,p]  for p < context_lens[s] - 1
 *   key_weights(slot of p, j)  = a[s,j,p]  for p = context_lens[s] - 1
 * (the newest token is this call's own: its slot's old sum was another's).
 * fp32 logits and statistics; for the product with V alone the weights are
 * taken as the sum of two bf16 (off by 2^-17 of a weight; an infinite value may give
 * NaN, its weight's second part being zero or below).  The batch's tokens are cut into
 * runs of equal length, so the last bits of a sequence's results can change with the
 * other sequences' lengths; the same call gives the same bits.
 *
 * workspace: device memory of at least pkv_decode_weights_workspace_size(...)
 * bytes, 256-byte aligned; it needs no initialisation (a call reads what it has
 * written itself).  Calls that overlap on the device must not share a workspace.
 *
 * A sequence of context length <= 0 is flagged (PKV_DEV_BAD_CONTEXT) and its
 * row of out is left as it was; one that is longer than its table is flagged
 * and clamped, and all of its weights are added.  A block id out of range is
 * flagged, its weights are dropped and what else the sequence gets is undefined.
 * More tokens than max_total_blocks blocks hold: PKV_DEV_WORKSPACE, nothing is
 * written.
 *
 * scale: finite, and scale * log2(e) too (else PKV_ERR_INVALID_ARG).
 *
 * Two launches.  Supported: head_dim in {64, 128}; Hq/Hkv in {1, 2, 4, 8};
 * block_size in {64, 128, 256, 512}; num_seqs <= 16384; max_blocks_per_seq *
 * block_size at most 65535 * 1024; max_total_blocks * block_size at most
 * (2^31 - 1) * 2048 / head_dim.
 */
pkv_status pkv_paged_decode_weights_attn(
    uint16_t *out, float *key_weights, const uint16_t *q, const uint16_t *new_k,
    const uint16_t *new_v, const int32_t *slot_mapping, uint16_t *k_cache, uint16_t *v_cache,
    const int32_t *block_tables, const int32_t *context_lens, int num_seqs, int num_q_heads,
    int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq, int64_t num_blocks,
    int64_t max_total_blocks, float scale, void *workspace, size_t workspace_bytes,
    int32_t *dev_status, void *stream);

/* Bytes of device workspace paged_prefill_weights needs (0 for invalid sizes
 * and for sizes whose workspace would not fit a size_t). */
size_t pkv_prefill_weights_workspace_size(int num_seqs, int64_t total_q, int max_seqlen_q,
                                          int window, int num_q_heads, int num_kv_heads,
                                          int max_blocks_per_seq, int block_size);

/*
 * paged_prefill_weights -- the key weights of a prompt chunk's last queries.
 *
 * q, k_cache, block_tables and cu_seqlens as for paged_prefill_attn, beside
 * which it is called (the chunk's K must be in the cache).  For a sequence of
 * n new queries of which the last R = min(window, n) count, c cached tokens,
 * query i at position c + i attending to keys 0 .. c + i:
 *   a[j,p] = sum of softmax_p(scale * <q_i,h, K_s[p, j]>) over the counted
 *            queries i with c + i >= p and the heads h of kv head j's group
 *   key_weights(slot of p, j) += a[j,p]  for p < c
 *   key_weights(slot of p, j)  = a[j,p]  for p >= c   (the chunk's own keys)
 * window >= max_seqlen_q counts every query.  A sequence with n = 0 changes
 * nothing.  One whose lengths do not fit (n > max_seqlen_q, n > len_k, more
 * keys than its table holds) is flagged, PKV_DEV_BAD_SEQLEN, and left out; a
 * block id out of range is flagged, its keys' sums are left as they were, and
 * the sequence's others are undefined.
 *
 * workspace: device memory of at least pkv_prefill_weights_workspace_size(...)
 * bytes, 256-byte aligned, zero-filled once before its first use.  Calls that
 * overlap on the device must not share a workspace.  How the work is split
 * depends on the batch, and with it the last bits; the same call gives the same
 * bits (keys in shared blocks apart).  A row's denominator is kept as one fp32
 * logarithm, so a weight is off by 2^-24 of that logarithm too.
 *
 * A wait that runs out (PKV_DEV_TIMEOUT) while the rows' denominators are
 * computed leaves rows out: the sums are then short of some queries' weights.
 * One that runs out later leaves the sums of the call's sequences undefined.
 *
 * scale: finite, and scale * log2(e) too (else PKV_ERR_INVALID_ARG).
 *
 * Two launches.  Supported: head_dim in {64, 128}; Hq/Hkv in {1, 2, 4, 8};
 * block_size in {64, 128, 256, 512}; max_blocks_per_seq * block_size at most 2^20.
 */
pkv_status pkv_paged_prefill_weights(
    float *key_weights, const uint16_t *q, const uint16_t *k_cache, const int32_t *block_tables,
    const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int num_seqs, int64_t total_q,
    int max_seqlen_q, int window, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
    int max_blocks_per_seq, int64_t num_blocks, float scale, void *workspace,
    size_t workspace_bytes, int32_t *dev_status, void *stream);

/*
 * test_prompt_fault -- TEST-ONLY fault injection for the bounded waits of
 * paged_prefill_weights, as pkv_test_decode_fault is for decode's: sets, for
 * the current device, the wall-clock limit of every wait (default 1 s) and,
 * for the process, how many CTAs of a pass (1: denominators, 2: sums) load
 * their tiles; the others wait for theirs in vain (-1: all load, the default).
 * Restore with pkv_test_prompt_fault(1000000000, 1, -1).  Synchronous.  Returns
 * PKV_ERR_INVALID_ARG for wait_limit_ns <= 0, a pass that is neither, or
 * loading_ctas < -1.
 */
pkv_status pkv_test_prompt_fault(int64_t wait_limit_ns, int pass, int loading_ctas);

/*
 * kv_evict -- shorten sequences to `budget` tokens, in place.
 *
 * For every sequence s with L = context_lens[s] > budget, and every kv head j
 * by itself: of the positions before the last `recent`, the H = budget -
 * recent with the largest key_weights are kept (a NaN counts as -inf, -0 as
 * +0; of equal ones the lowest position), and the last `recent` are kept.
 * Kept positions below H stay where they are; those behind, in order, take
 * the places below H that are not kept, in order; the recent ones follow in
 * order at H .. budget - 1.  K, V and key_weights move together.  Places
 * from `budget` on, and blocks past the first ceil(budget / block_size), are
 * left as they were and are the caller's to reuse (pkv_bm_evict).
 *   kept      int32 [num_seqs, Hkv, budget]: the position, before the call,
 *             of the token now at each place (-1 past a shorter sequence's end)
 *   new_lens  int32 [num_seqs]: min(L, budget); must not overlap context_lens,
 *             nor k_cache v_cache (PKV_ERR_INVALID_ARG)
 * Sequences of at most `budget` tokens are not touched.  Decode does not
 * depend on the order of the keys, so attention goes on with new_lens as the
 * context length; the positions that the model encodes count on from the old
 * length.  No block may belong to two sequences of the call, nor to one
 * outside it that still needs its keys (a shared prefix): its rows move.
 *
 * A negative context length, or one longer than the table, is flagged
 * (PKV_DEV_BAD_CONTEXT), a block id out of range among the sequence's blocks
 * too (PKV_DEV_BAD_BLOCK): the sequence is left as it was, its kept is all -1
 * and its new_lens its old length.
 *
 * Two launches, no workspace.  Requires 0 <= recent <= budget, budget > 0;
 * head_dim in {64, 128}; block_size in {64, 128, 256, 512}; budget and
 * max_blocks_per_seq * block_size at most 2^20 (PKV_ERR_UNSUPPORTED).
 */
pkv_status pkv_kv_evict(uint16_t *k_cache, uint16_t *v_cache, float *key_weights,
                        const int32_t *block_tables, const int32_t *context_lens, int num_seqs,
                        int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq,
                        int64_t num_blocks, int budget, int recent, int32_t *kept,
                        int32_t *new_lens, int32_t *dev_status, void *stream);

/*
 * plan_step -- block tables, slots and positions of a step, on the device.
 *
 * The device's counterpart of pkv_bm_append, pkv_bm_free, pkv_bm_block_table and
 * pkv_bm_slots, for a batch at a time: a captured loop of steps needs no host between
 * them.  What a row of the tables begins with may come from the block manager (a
 * shared prefix); the blocks behind come from a stack of free ones, free_blocks
 * [free_capacity] int32, of which the first *num_free are on it, the last one on top.
 *
 * For every sequence s that holds L = context_lens[s] tokens, new_lens[s] says:
 *   n > 0   n tokens arrive, at positions L .. L + n - 1.  They take n rows of the
 *           step, behind those of the sequences before s, and if they need blocks,
 *           need = ceil((L + n) / block_size) - ceil(L / block_size), these come off
 *           the top of the stack in order into block_tables[s]
 *   0       it pauses: no rows, nothing changes
 *   -1      it ends: its blocks go back onto the stack in order, but for the first
 *           borrowed_blocks[s] (NULL: none), which are somebody else's.  Its row of
 *           block_tables stays as it was
 * All sequences that end come first, in order of s, then those that need blocks: what
 * one gives back another one takes in the same step.
 * Written, for the step's num_rows rows of which cu_seqlens_q[num_seqs] are in use:
 *   slot_mapping[r], positions[r]   (-1 and 0 behind the last row in use)
 *   cu_seqlens_q, cu_seqlens_k      sums of n, and of the lengths after the step
 *   new_context_lens, *new_num_free (may be context_lens and num_free themselves, but
 *                                   not overlap them otherwise, PKV_ERR_INVALID_ARG;
 *                                   where they are others, a call can be repeated)
 * No other two of the arrays may overlap (not checked).
 *
 * A sequence whose blocks the stack does not hold is refused, PKV_DEV_NO_BLOCKS, and
 * with it all later ones that need any: those keep what they have, their rows have
 * slots of -1, and cu_seqlens_k counts no keys for them (so prefill leaves them out).
 * One that needs no block goes on.  Refused and flagged the same way are sequences
 * whose rows end behind num_rows (PKV_DEV_BAD_SEQLEN), and those with a negative
 * length or one that its table has no room for (PKV_DEV_BAD_CONTEXT; positions count
 * from 0 where L itself is bad).  new_lens < -1 counts as 0 and borrowed_blocks
 * outside [0, ceil(L / block_size)] as the nearer end, flagged BAD_SEQLEN and
 * BAD_CONTEXT.  A block id out of range gives slots of -1 (PKV_DEV_BAD_BLOCK); so is
 * flagged a *num_free outside [0, free_capacity], taken as the nearer end, and a stack
 * with no room for what comes back, which is then dropped.  No block may be held
 * twice, nor held and free, but in borrowed places.  Sums saturate at 2^31 - 1
 * (flagged BAD_SEQLEN).
 *
 * One launch for up to 256 sequences and 1024 rows, else two.  Supported: block_size in
 * {64, 128, 256, 512}; num_seqs <= 16384; max_blocks_per_seq * block_size at most 2^30;
 * num_blocks * block_size and free_capacity below 2^31, num_rows below 2^31 - 1.
 */
pkv_status pkv_plan_step(const int32_t *new_lens, const int32_t *context_lens,
                         const int32_t *borrowed_blocks, int32_t *block_tables,
                         int32_t *free_blocks, const int32_t *num_free,
                         int32_t *new_context_lens, int32_t *new_num_free, int32_t *slot_mapping,
                         int32_t *positions, int32_t *cu_seqlens_q, int32_t *cu_seqlens_k,
                         int num_seqs, int64_t num_rows, int max_blocks_per_seq, int block_size,
                         int64_t num_blocks, int64_t free_capacity, int32_t *dev_status,
                         void *stream);

/*
 * rope_turns -- frequencies as pkv_norm_rope_store reads them (host, no GPU work).
 *
 * turns[i] = the fraction of a turn that inv_freq[i] radians per position are, in units
 * of 2^-64 of a turn, rounded to nearest; inv_freq finite, at most 10^6 in magnitude
 * (PKV_ERR_INVALID_ARG, nothing is written).  Angles are as exact as inv_freq is: a
 * double's last bit is 2^-33 of a turn at position 2^20 where a pair turns at 1 radian
 * per position.  Any scaling for long contexts is one of inv_freq (and of amplitude).
 */
pkv_status pkv_rope_turns(const double *inv_freq, int num_pairs, uint64_t *turns);

/*
 * norm_rope_store -- norm of each query and key head, rotation by position, and
 * kv_store, in one pass over a step's projections.
 *
 * For each token t and each of the Hq heads x of q and Hkv heads of k:
 *   y  = x / sqrt(mean(x^2) + eps) * weight   (q_weight, k_weight [D] bf16; both NULL:
 *                                              y = x)
 *   y' = y with the pairs of its first rotary_dim values turned: pair i, (y[i],
 *        y[i + rotary_dim / 2]) or, interleaved, (y[2i], y[2i + 1]), by the angle
 *        positions[t] * turns[i] / 2^64 turns: (a, b) -> amplitude * (a cos - b sin,
 *        b cos + a sin)
 * y' of q goes to q_out [T, Hq, D], that of k to slot slot_mapping[t] of k_cache and, if
 * k_out is not NULL, to k_out [T, Hkv, D]; v goes to v_cache as it is, to the bit.
 * k_cache, v_cache and slot_mapping all NULL: nothing is stored, v is not read and
 * k_out is required.  All arithmetic in fp32, rounded once, to bf16 (a head whose squares
 * add up to 2^128 or more has an infinite norm and comes out as zeros).  positions may
 * be any int32 (negative ones turn backwards).
 *
 * q, k, v: as in kv_store, values between tokens given by their strides (0 =
 * contiguous), so that all three may be parts of one projection.  q_out may be q, and
 * k_out k, where those are contiguous; other overlaps of outputs and inputs return
 * PKV_ERR_INVALID_ARG (caches are not checked).  slot_mapping as for kv_store: -1
 * skips (q_out and k_out are written all the same), other slots out of range are
 * flagged (PKV_DEV_BAD_SLOT) and skipped, slots >= 0 must be unique.  A wait that runs
 * out (PKV_DEV_TIMEOUT; only calls of many tokens wait) leaves the call's rows of q_out
 * and k_out and its slots of the caches undefined, and nothing else touched.
 *
 * One launch.  Supported: head_dim in {64, 128}; rotary_dim a multiple of 16 from 0
 * (then turns and positions may be NULL) to head_dim; at most 65536 heads of a kind.
 * eps >= 0 and amplitude finite.
 */
pkv_status pkv_norm_rope_store(uint16_t *q_out, uint16_t *k_out, const uint16_t *q,
                               const uint16_t *k, const uint16_t *v, uint16_t *k_cache,
                               uint16_t *v_cache, const int32_t *slot_mapping,
                               const int32_t *positions, const uint64_t *turns,
                               const uint16_t *q_weight, const uint16_t *k_weight,
                               int64_t num_tokens, int num_q_heads, int num_kv_heads,
                               int head_dim, int64_t q_token_stride, int64_t k_token_stride,
                               int64_t v_token_stride, int rotary_dim, int interleaved, float eps,
                               float amplitude, int64_t num_blocks, int block_size,
                               int32_t *dev_status, void *stream);

/*
 * test_rope_fault -- TEST-ONLY, for norm_rope_store: sets, for the current device, the
 * wall-clock limit of every wait (default 1 s) and, for the process, how many CTAs of a
 * call of many tokens load them (the others wait for theirs in vain, PKV_DEV_TIMEOUT;
 * -1: all, the default).  Restore with pkv_test_rope_fault(1000000000, -1).
 * Synchronous.  Returns PKV_ERR_INVALID_ARG for wait_limit_ns <= 0 or loading_ctas < -1.
 */
pkv_status pkv_test_rope_fault(int64_t wait_limit_ns, int loading_ctas);

/*
 * Bytes of device workspace paged_decode_shared_attn needs: the plan of the batch and
 * the parts of its rows.  Returns 0 for invalid sizes, more than 8192 sequences among them.
 */
size_t pkv_decode_shared_workspace_size(int num_seqs, int num_groups, int num_q_heads,
                                        int num_kv_heads, int head_dim);

/*
 * paged_decode_shared_attn -- paged_decode_attn for a batch in which groups of
 * sequences begin with the same blocks (a system prompt, samples of one answer), whose
 * keys and values are then read once for a group.
 *
 * out, q, caches, block_tables and context_lens as for paged_decode_attn, and the same
 * result up to rounding.  Group g is the neighbouring sequences group_starts[g] ..
 * group_starts[g + 1] - 1 (group_starts int32 [num_groups + 1], from 0 to num_seqs);
 * the first shared_blocks[g] (int32 [num_groups]) entries of their rows of block_tables
 * are the same in all of them (any of the rows may be read).  A group uses no more of
 * them than its shortest context fills; a group of one, or one with shared_blocks of 0,
 * is attended like any other sequence, and so is every one where all contexts together
 * are so short that reading them whole is faster.  pkv_bm_prefix_groups finds groups.
 * fp32 logits and statistics; for the product with V alone the weights are taken as the
 * sum of two bf16 (off by 2^-16 of a weight).  How the work is split depends on the
 * batch, and with it the last bits; the same call gives the same bits.
 *
 * A sequence of context length <= 0 is flagged (PKV_DEV_BAD_CONTEXT) and its row of out
 * is left as it was; one that is longer than its table is flagged and clamped.
 * shared_blocks outside [0, max_blocks_per_seq] is flagged the same way and taken as the
 * nearer end.  group_starts that do not begin at 0, end at num_seqs or ever go back are
 * flagged (PKV_DEV_BAD_SEQLEN); every sequence is then attended by itself.  A block id
 * out of range is flagged and what its sequences get is undefined.  A wait that runs out
 * (PKV_DEV_TIMEOUT) leaves the rows of out undefined.
 *
 * workspace: device memory of at least pkv_decode_shared_workspace_size(...) bytes,
 * 256-byte aligned; it needs no initialisation.  Calls that overlap on the device must
 * not share a workspace.
 *
 * scale: finite, and scale * log2(e) too (else PKV_ERR_INVALID_ARG).
 *
 * out may be q.  Three launches, chosen by sizes and not by the lengths, which the host
 * does not know: two where num_seqs <= 384 and the tables have room for at most 16 MiB of
 * K and V (num_seqs * max_blocks_per_seq blocks), one where they have room for at most
 * 1024 tokens a sequence (512 for Hq/Hkv of 8) and num_seqs * num_kv_heads is at most two
 * per SM.  So tables trimmed to the batch make a call of few short contexts faster.
 * Supported: head_dim in {64, 128}; Hq/Hkv in {1, 2, 4, 8}; block_size in {64, 128, 256,
 * 512}; num_seqs <= 8192, 1 <= num_groups <= num_seqs (else PKV_ERR_INVALID_ARG); at most
 * 4096 kv heads; max_blocks_per_seq * block_size at most 2^20.
 */
pkv_status pkv_paged_decode_shared_attn(
    uint16_t *out, const uint16_t *q, const uint16_t *k_cache, const uint16_t *v_cache,
    const int32_t *block_tables, const int32_t *context_lens, const int32_t *group_starts,
    const int32_t *shared_blocks, int num_seqs, int num_groups, int num_q_heads,
    int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq, int64_t num_blocks,
    float scale, void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream);

/*
 * test_shared_fault -- TEST-ONLY, for paged_decode_shared_attn: sets, for the current
 * device, the wall-clock limit of every wait (default 1 s) and, for the process, how
 * many CTAs load the prefixes that they work on (the others wait for theirs in vain,
 * PKV_DEV_TIMEOUT; -1: all, the default), and whether prefixes are shared however
 * little there is to read (0: where it pays, the default).  Restore with
 * pkv_test_shared_fault(1000000000, -1, 0).  Synchronous.  Returns PKV_ERR_INVALID_ARG
 * for wait_limit_ns <= 0 or loading_ctas < -1.
 */
pkv_status pkv_test_shared_fault(int64_t wait_limit_ns, int loading_ctas, int share_always);

/*
 * w4a16_dequant -- W4A16-G128 weight dequantisation (s1nh.org post on
 * upgrading nano-vllm to big-vLLM, section on quantisation: every int32 of
 * weight_packed holds eight 4-bit values; int32 -> u4 unpack -> s4
 * reconstruct -> float x weight_scale, one scale per 128 weights).
 *
 *   out[n, j] = bf16( (u4(packed[n, j / 8], j % 8) - 8) * scales[n, j / 128] )
 *
 * where u4(w, i) = (w >> 4i) & 15 (the lowest nibble is the first value).
 * packed [n_rows, k/8] int32, scales [n_rows, k/128] bf16, out [n_rows, k]
 * bf16, all row-major and contiguous, device memory owned by the caller.
 * The product is exact in fp32 and rounded once (nearest even) to bf16.
 *
 * k must be a multiple of 128 and group_size 128 (PKV_ERR_INVALID_ARG /
 * PKV_ERR_UNSUPPORTED otherwise); out and packed 16-byte aligned, scales
 * 2-byte aligned.  n_rows == 0 or k == 0: nothing to do.
 */
pkv_status pkv_w4a16_dequant(uint16_t *out, const int32_t *packed, const uint16_t *scales,
                             int64_t n_rows, int64_t k, int group_size, void *stream);

/*
 * Block manager -- host-side allocator of the cache's blocks (no GPU work).
 *
 * The cache is a pool of fixed-size blocks handed out and released by
 * reference counting (nano-vllm hub page, "core tech 4: KV Cache block
 * manager"); a sequence takes a new block when its length reaches a multiple
 * of the block size plus one (CSDN essay "from nanoVLLM to vLLM", Mountain
 * 1).  Prefix sharing: every full block gets a content key, a 64-bit FNV-1a
 * hash chained over the key of the block before it and the block's token
 * ids; a new sequence whose prompt begins with full blocks whose keys (and
 * tokens) match reuses those blocks, reference count + 1, and only the rest
 * of the prompt needs kv_store and its own prefill rows.  Freed blocks keep
 * their content and key, and stay reusable, until they are handed out again
 * (oldest freed first; a sequence's tail is freed before its prefix).
 *
 * The outputs feed the kernels directly: pkv_bm_block_table gives a row of
 * block_tables (padded with -1), pkv_bm_slots the slot_mapping of a token
 * range, and pkv_bm_allocate the cached length c (cu_seqlens_k - cu_seqlens_q).
 * Not thread-safe: one manager per host thread.
 */
typedef struct pkv_block_manager pkv_block_manager;

/* num_blocks > 0 blocks of block_size tokens; NULL on bad arguments or no memory. */
pkv_block_manager *pkv_bm_create(int num_blocks, int block_size);
void pkv_bm_destroy(pkv_block_manager *m);
int pkv_bm_num_free_blocks(const pkv_block_manager *m);

/* Admit sequence seq_id (not yet present) with its num_tokens > 0 prompt
 * tokens: reuses the cached leading full blocks, takes fresh ones for the
 * rest (all or nothing: PKV_ERR_OUT_OF_BLOCKS leaves the manager unchanged).
 * *num_cached_tokens = tokens whose K/V are already in reused blocks, at most
 * num_tokens - 1 (the last prompt token is always computed). */
pkv_status pkv_bm_allocate(pkv_block_manager *m, int64_t seq_id, const int32_t *tokens,
                           int num_tokens, int *num_cached_tokens);
/* Append one generated token (a fresh block when it starts a new one). */
pkv_status pkv_bm_append(pkv_block_manager *m, int64_t seq_id, int32_t token);
/* Release the sequence's blocks (reference count - 1 each). */
pkv_status pkv_bm_free(pkv_block_manager *m, int64_t seq_id);

/* The sequence has been cut to its first keep_tokens > 0 places, by pkv_kv_evict
 * on its block table as it was before this call: releases the blocks past
 * them.  The rest lose their content keys, and the sequence's later blocks get
 * none: what they hold is no longer the prompt's tokens in order.  Nothing
 * changes for a sequence of at most keep_tokens tokens.  PKV_ERR_UNSUPPORTED,
 * with nothing changed, when one of the first ceil(keep_tokens / block_size)
 * blocks is shared with another sequence: evicting would move the other's
 * keys, so ask before launching pkv_kv_evict.  Released blocks can be handed
 * out at once; work that writes them must follow the eviction on its stream. */
pkv_status pkv_bm_evict(pkv_block_manager *m, int64_t seq_id, int keep_tokens);

/* Tokens held by the sequence, or -1 if unknown. */
int pkv_bm_num_tokens(const pkv_block_manager *m, int64_t seq_id);
/* Writes max_blocks entries of the sequence's block table (-1 past its
 * blocks) when out != NULL; returns its block count, -1 if unknown. */
int pkv_bm_block_table(const pkv_block_manager *m, int64_t seq_id, int32_t *out,
                       int max_blocks);
/* slots[i] = block_table[p / bs] * bs + p % bs for p = first .. first+count-1. */
pkv_status pkv_bm_slots(const pkv_block_manager *m, int64_t seq_id, int first, int count,
                        int32_t *slots);
/* An order of sequences, and groups of neighbours in it, for
 * pkv_paged_decode_shared_attn: group g is the seq_ids[order[i]] for i = group_starts[g]
 * .. group_starts[g + 1] - 1, which begin with the same shared_blocks[g] blocks.  Groups
 * are chosen so that the blocks that need not be read again, sum of (members - 1) *
 * shared_blocks, are many: where some sequences share more among themselves than with
 * the rest, they become a group of their own if that saves more.  Sequences that share
 * nothing are groups of one with shared_blocks 0.  order and shared_blocks have room
 * for num_seqs values, group_starts for num_seqs + 1; *num_groups are written.  An
 * unknown sequence, or one that is listed twice: PKV_ERR_INVALID_ARG; no host memory:
 * PKV_ERR_WORKSPACE. */
pkv_status pkv_bm_prefix_groups(const pkv_block_manager *m, const int64_t *seq_ids, int num_seqs,
                                int32_t *order, int32_t *group_starts, int32_t *shared_blocks,
                                int *num_groups);
/* Reference count of a block (0 = free), -1 on a bad index. */
int pkv_bm_ref_count(const pkv_block_manager *m, int block);

#ifdef __cplusplus
}
#endif

#endif /* PKV_H_ */
