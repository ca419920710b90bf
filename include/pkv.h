/*
 * pkv.h — C ABI of libpkv: attention over a paged KV cache for one
 * continuous-batching step, on one GB300 (sm_103a).
 *
 * What the operations are (the source pages name them, they print no API):
 *  - "Efficient management of attention key and value memory with
 *    PagedAttention" (Welcome to vLLM, feature list): K/V of every sequence
 *    live in fixed-size physical blocks reached through a per-sequence block
 *    table; "per-step KV bookkeeping handed to the kernels" (Litellama,
 *    Architecture tree, executor/attention_metadata.py).
 *  - "flash attention decode (online softmax, paged KV, GQA)" and
 *    "Split-KV paged attention for long context" (rvLLM: High-performance
 *    LLM inference in Rust, Kernel Compiler Stack / Tier 2: Hand-written CUDA
 *    kernels; FA3 v3 Attention Kernel).
 *  - partial attention "merged by log-sum-exp" (rapid_llm README, feature
 *    table, row "Decode context parallelism"), done here over KV partitions
 *    of one GPU.
 *  - "RoPE + KV cache write -- fused, no intermediate alloc" (rvLLM, Kernel
 *    Compiler Stack, decode step at c=128): rope_reshape_and_cache below; its
 *    cache-write half alone is reshape_and_cache.
 *  - "FP8 KV Cache" (Litellama, Features; rvLLM, Optional Features):
 *    E4M3 codes with one fp32 scale per KV head for K and one for V.
 *  - "Chunked Prefill ... 512-token chunks" (Litellama, Features): causal
 *    attention of a chunk of new query tokens over the same paged cache.
 *
 * Conventions shared by every entry point
 *  - All pointers are DEVICE pointers unless stated; the caller owns every
 *    buffer. The library allocates no device memory and keeps no per-call
 *    state. Its library-wide state: per device, the device error word, the
 *    scratch array of paged_attn_decode_noalloc (PKV_NOALLOC_SCRATCH_BYTES,
 *    a file-scope device array held by every GPU that loads the library),
 *    the cached SM count and the one-time kernel attribute and grid-size
 *    settings; process-wide, the driver's tensor-map encoder entry point.
 *  - `stream` is a cudaStream_t passed as an opaque pointer (NULL = the
 *    legacy default stream). Work is only enqueued; nothing synchronises,
 *    except pkv_get_device_error.
 *  - Argument checks are synchronous: a bad argument returns a status and
 *    nothing is launched. A launch failure returns PKV_ERR_CUDA.
 *  - Data-dependent checks run on the device (block ids outside
 *    [0, num_blocks), slots outside the pool, seq_lens above the stated
 *    maximum). A failing check skips the access, sets a bit in the device
 *    error word and never traps; pkv_get_device_error reads the word.
 *  - Tensors are dense and row-major. Every base pointer must be 16-byte
 *    aligned.
 *  - Layouts (B = num_seqs, Hq = num_q_heads, Hkv = num_kv_heads,
 *    G = Hq / Hkv, D = head_dim, BS = block_size):
 *      q            [B, Hq, D]                       q dtype
 *      out          [B, Hq, D]                       q dtype
 *      k_cache      [num_blocks, Hkv, BS, D]          kv dtype (same for v)
 *      block_tables int32 [B, max_blocks_per_seq]
 *      seq_lens     int32 [B]  context length INCLUDING the new token, whose
 *                              K/V reshape_and_cache has already written
 *    Logical token j of sequence b lives in physical block
 *    block_tables[b][j / BS] at offset j % BS. Query head h reads KV head
 *    h / G. Within a block each KV head's BS x D run is contiguous; the
 *    kernels read it as BS / 16 consecutive pages of 16 tokens, or gather a
 *    16-token page row by row when BS < 16 (BS = 1 is token-level paging).
 *  - Cache slots past a sequence's context (the rest of its last block) may
 *    hold anything, NaN included: they are read with weight 0 and their
 *    values are zeroed before they meet that weight.
 *  - E4M3 caches run f16 tensor-core MMAs on the codes widened to f16
 *    (exact). A bf16 q is scaled by a power of two 2^-e, rounded to f16, and
 *    the scores are multiplied back by 2^e: e is chosen per sequence and KV
 *    head in decode (per query row in prefill) so that the largest |q|
 *    element lands in [2^14, 2^15). Any finite bf16 q works (no overflow to
 *    inf). Elements within 2^-28 of the largest of their group convert
 *    exactly; smaller ones fall into f16's subnormal range and move by at
 *    most 2^-39 of the largest.
 *  - Supported: D in {64, 128, 256}; BS a power of two from 1 to 64 (decode
 *    and the cache writes; prefill, and decode at D = 256, need BS >= 16);
 *    G <= 16 (G <= 8 at D = 256); q dtype F16 or BF16; KV
 *    dtype equal to the q dtype, or FP8_E4M3 with per-KV-head fp32 scales
 *    (dequantised value = code * scale).
 */
#ifndef PKV_H
#define PKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PKV_OK = 0,
  PKV_ERR_INVALID_ARG = 1,   /* null pointer, bad size, misaligned pointer */
  PKV_ERR_UNSUPPORTED = 2,   /* valid but not built: D, BS, G or dtype pair */
  PKV_ERR_WORKSPACE = 3,     /* workspace missing or smaller than required */
  PKV_ERR_CUDA = 4,          /* a CUDA runtime call or a launch failed */
  PKV_ERR_DEVICE_CHECK = 5   /* a device-side check failed (see below) */
} pkv_status;

typedef enum {
  PKV_F16 = 0,
  PKV_BF16 = 1,
  PKV_FP8_E4M3 = 2,
  PKV_FP8_E4M3_BLOCK = 3     /* E4M3 codes, one E8M0 scale per (block, KV head);
                                rope_append_block_scaled, the _ext calls, paged_attn_tree
                                and kv_keep_path only */
} pkv_dtype;

/* Bits of the device error word. */
#define PKV_DEVERR_BLOCK_ID   0x1u  /* block table entry outside [0, num_blocks) */
#define PKV_DEVERR_SLOT       0x2u  /* slot >= num_blocks * block_size */
#define PKV_DEVERR_SEQ_LEN    0x4u  /* seq_len < 0 or above the stated maximum */
#define PKV_DEVERR_TIMEOUT    0x8u  /* a bounded wait on an async copy gave up */
#define PKV_DEVERR_QLEN       0x10u /* prefill: chunk longer than its context, or outside q's rows */
#define PKV_DEVERR_POSITION   0x20u /* rotary: position outside [0, max_position) */
#define PKV_DEVERR_COUNTER    0x40u /* decode: workspace counters were not zero */
#define PKV_DEVERR_PATH       0x80u /* kept path not rising or outside its tree, or no such parent row */
#define PKV_DEVERR_POOL       0x100u /* no unused block left, or one given back that was not in use */

/*
 * paged_attn_decode_workspace_size
 *   Bytes of device workspace paged_attn_decode needs for these sizes: the
 *   per-(sequence, KV head) partition counters and the fp32 partial outputs
 *   and log-sum-exps of the split-KV partitions. partition_tokens: as passed
 *   to paged_attn_decode (0 = automatic; the automatic size depends on the
 *   current device's SM count, so query on the device that will run the
 *   call). Returns 0 for invalid sizes.
 */
size_t paged_attn_decode_workspace_size(int num_seqs, int num_q_heads,
                                        int num_kv_heads, int head_dim,
                                        int max_seq_len, int partition_tokens);

/*
 * paged_attn_decode — one query token per sequence against its paged K/V.
 *   For each sequence b and query head h (KV head g = h / G):
 *     s_j   = scale * k_scale[g] * <q[b,h,:], Kcode_j>          j < seq_lens[b]
 *     out   = v_scale[g] * sum_j softmax(s)_j * Vcode_j          (q dtype, RNE)
 *     lse   = log(sum_j exp(s_j))                                (natural log)
 *   (k_scale = v_scale = 1 unless kv_dtype is FP8_E4M3.)
 *   Each context is cut into partitions (of `partition_tokens` tokens, a
 *   multiple of 16 up to 8192, or 0 = automatic sizes); each partition is
 *   reduced with an online softmax and the partitions of a sequence are
 *   merged by log-sum-exp in the same kernel launch. With 0, a batch whose
 *   (sequence, KV head) pairs fit one per SM may be planned as one partition
 *   per context (on head_dim <= 128 with blocks of 16 tokens or more): the
 *   same attention, summed in another order than a split plan.
 *   seq_lens[b] == 0 gives out = 0 and lse = -inf.
 *   max_seq_len: upper bound on every seq_lens[b] (sizes the plan); a larger
 *   seq_len sets PKV_DEVERR_SEQ_LEN and is clamped.
 *   k_scales, v_scales: fp32 [Hkv], required for FP8 KV, ignored otherwise.
 *   out_lse: optional fp32 [B, Hq] (NULL to skip).
 *   workspace: 256-byte aligned device buffer of at least
 *   paged_attn_decode_workspace_size() bytes, always required. Zero-fill it
 *   once before its first use: each call sets the per-(sequence, KV head)
 *   partition counters it used back to zero (CUDA-graph replays included),
 *   so a call enqueues nothing but its kernel. A call that ends with a
 *   device error may leave counters set; zero the workspace again before
 *   reusing it (PKV_DEVERR_COUNTER reports counters found non-zero). Two
 *   calls that share a workspace must not overlap on the GPU, and are calls of
 *   the same num_seqs and num_kv_heads (others' partial results lie where
 *   these counters do; zero it in between, or give each its own).
 *   The kernel is launched as a programmatic dependent of the kernel ahead
 *   of it on `stream`: it may become resident while that kernel runs, and
 *   reads no input before that kernel has finished.
 */
pkv_status paged_attn_decode(void* out, const void* q, pkv_dtype q_dtype,
                             const void* k_cache, const void* v_cache,
                             pkv_dtype kv_dtype, const int32_t* block_tables,
                             const int32_t* seq_lens, int num_seqs,
                             int num_q_heads, int num_kv_heads, int head_dim,
                             int block_size, int max_blocks_per_seq,
                             int num_blocks, int max_seq_len, float scale,
                             const float* k_scales, const float* v_scales,
                             int partition_tokens, float* out_lse,
                             void* workspace, size_t workspace_bytes,
                             void* stream);

/*
 * paged_attn_decode_step — one decode step of attention: the cache write of
 * every sequence's new token, then decode attention, in one call ("RoPE + KV
 * cache write" followed by "Flash Attention Decode", rvLLM: High-performance
 * LLM inference in Rust, Kernel Compiler Stack, decode step).
 *   key, value: [num_seqs, Hkv, D] in the q dtype, the new token of each
 *   sequence; slot_mapping: int64 [num_seqs], its slot. The step's contract:
 *   row b is sequence b's token at position seq_lens[b] - 1 (slot_mapping[b]
 *   is that position's slot, or < 0 to write nothing). Everything else is as
 *   reshape_and_cache followed by paged_attn_decode on `stream`, with the same
 *   results. Because the library itself writes the cache just ahead of the
 *   attention kernel, and only those rows, the attention kernel reads its
 *   inputs and loads every page but the newest token's before the cache write
 *   has finished (the separate calls must wait for it first).
 *   All arguments are checked before anything is enqueued.
 */
pkv_status paged_attn_decode_step(const void* key, const void* value,
                                  const int64_t* slot_mapping, void* out, const void* q,
                                  pkv_dtype q_dtype, void* k_cache, void* v_cache,
                                  pkv_dtype kv_dtype, const int32_t* block_tables,
                                  const int32_t* seq_lens, int num_seqs, int num_q_heads,
                                  int num_kv_heads, int head_dim, int block_size,
                                  int max_blocks_per_seq, int num_blocks, int max_seq_len,
                                  float scale, const float* k_scales, const float* v_scales,
                                  int partition_tokens, float* out_lse, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* Size of the scratch array paged_attn_decode_noalloc uses (32 MiB). */
#define PKV_NOALLOC_SCRATCH_BYTES (32u << 20)

/*
 * paged_attn_decode_noalloc — paged_attn_decode without a caller workspace.
 *   The source pages have no counterpart to this call; it exists for callers
 *   that cannot allocate device memory at the point where they run
 *   attention: an engine whose memory planner has already handed the whole
 *   device to weights and the KV pool, a latency-critical loop that cannot
 *   afford cudaMalloc/cudaFree (they can synchronise the device), or a plain
 *   C host with no allocator of its own.
 *   Same arguments, results and errors as paged_attn_decode, minus the
 *   workspace: the split-KV scratch is one device array of
 *   PKV_NOALLOC_SCRATCH_BYTES inside the library, held by every GPU that
 *   loads the library until the process exits. Sizes whose
 *   paged_attn_decode_workspace_size() exceeds PKV_NOALLOC_SCRATCH_BYTES are
 *   rejected with PKV_ERR_WORKSPACE before anything is launched.
 *   Nothing here allocates. The first call on a device looks up the array's
 *   device address (cudaGetSymbolAddress); make that first call before any
 *   stream capture. The array starts zero-filled and each call leaves the
 *   counters it used at zero. Every call on a device shares the one array,
 *   so calls that overlap on the GPU (on different streams, or from
 *   different threads) race: serialise them. After a race, or a call that
 *   reported a device error, clear the array with
 *   paged_attn_decode_noalloc_reset before the next call.
 */
pkv_status paged_attn_decode_noalloc(void* out, const void* q, pkv_dtype q_dtype,
                                     const void* k_cache, const void* v_cache,
                                     pkv_dtype kv_dtype,
                                     const int32_t* block_tables,
                                     const int32_t* seq_lens, int num_seqs,
                                     int num_q_heads, int num_kv_heads,
                                     int head_dim, int block_size,
                                     int max_blocks_per_seq, int num_blocks,
                                     int max_seq_len, float scale,
                                     const float* k_scales,
                                     const float* v_scales,
                                     int partition_tokens, float* out_lse,
                                     void* stream);

/*
 * paged_attn_decode_noalloc_reset — the way back to a clean scratch array for
 * paged_attn_decode_noalloc. The source pages have no counterpart to this
 * call either. Its callers cannot clear the library's array themselves, yet
 * its partition counters must be zero when a call starts; a call that ended
 * with a device error (PKV_DEVERR_TIMEOUT, for instance), or two calls that
 * overlapped on the GPU, can leave some set, and every later call on that
 * device is then flagged with PKV_DEVERR_COUNTER or merges stale partials.
 * This enqueues on `stream` one cudaMemsetAsync that zero-fills the whole
 * array of the current device (PKV_NOALLOC_SCRATCH_BYTES; it allocates
 * nothing). Call it, on the stream the decode calls use, after such an error
 * and before the next paged_attn_decode_noalloc; it must not overlap a
 * noalloc call on the GPU. Like the decode call, its first use on a device
 * looks up the array's address, so make that first call outside any stream
 * capture. PKV_ERR_CUDA if the lookup or the memset fails.
 */
pkv_status paged_attn_decode_noalloc_reset(void* stream);

/*
 * paged_attn_prefill_chunk — causal attention of a chunk of new query
 * tokens of each sequence over that sequence's paged cache.
 *   Sequence n owns query rows cu_q_lens[n] .. cu_q_lens[n+1]-1 of q/out
 *   ([total_q_tokens, Hq, D]); its chunk length L_n = cu_q_lens[n+1] -
 *   cu_q_lens[n] and seq_lens[n] is its whole context INCLUDING the chunk
 *   (whose K/V reshape_and_cache has already written), so P_n = seq_lens[n]
 *   - L_n tokens precede it. Query row i of the chunk sits at absolute
 *   position P_n + i and attends keys 0 .. P_n + i (causal, aligned to the
 *   bottom right). Same scores, scales and output dtype as decode.
 *   max_q_len: upper bound on every L_n (sizes the grid).
 *   out_lse: optional fp32 [total_q_tokens, Hq].
 *   A chunk with L_n > seq_lens[n], or whose rows do not lie within the
 *   total_q_tokens rows of q and out, sets PKV_DEVERR_QLEN and is skipped.
 *   Launch: one CTA per tile of query rows; when those would occupy at most
 *   half of the SMs, a cluster of two CTAs per tile, each over half of the
 *   tile's keys, merged by log-sum-exp on chip (tensor-core kernel: 16-bit
 *   caches at D 64/128/256, E4M3 caches at D 64/128). With an E4M3 cache a
 *   bf16 q goes to f16 MMAs as described at the top of this file.
 */
pkv_status paged_attn_prefill_chunk(void* out, const void* q,
                                    pkv_dtype q_dtype, const void* k_cache,
                                    const void* v_cache, pkv_dtype kv_dtype,
                                    const int32_t* block_tables,
                                    const int32_t* seq_lens,
                                    const int32_t* cu_q_lens, int num_seqs,
                                    int total_q_tokens, int max_q_len,
                                    int num_q_heads, int num_kv_heads,
                                    int head_dim, int block_size,
                                    int max_blocks_per_seq, int num_blocks,
                                    float scale, const float* k_scales,
                                    const float* v_scales, float* out_lse,
                                    void* stream);

/*
 * paged_attn_varlen — attention for a whole continuous-batching step in one
 * call: decode sequences and prefill chunks over the same paged cache
 * ("Continuous batching" and "Chunked Prefill", Litellama, Features).
 *   Sequences [0, num_decode_seqs) are decode sequences, one query row each:
 *   q rows 0 .. num_decode_seqs-1. Sequences [num_decode_seqs, num_seqs) are
 *   prefill chunks: query_start_loc int32 [num_seqs + 1] holds the first q row
 *   of every sequence (query_start_loc[i] = i for the decode sequences) and
 *   query_start_loc[num_seqs] = total_q_tokens.
 *   q, out: [total_q_tokens, Hq, D]; out_lse (optional): fp32
 *   [total_q_tokens, Hq]. block_tables [num_seqs, max_blocks_per_seq] and
 *   seq_lens [num_seqs] as for decode and prefill (seq_lens include the new
 *   tokens, already cached by reshape_and_cache).
 *   Decode rows are computed by paged_attn_decode's kernel (max_decode_seq_len
 *   bounds their seq_lens and sizes the split; the workspace is
 *   paged_attn_decode_workspace_size(num_decode_seqs, Hq, Hkv, D,
 *   max_decode_seq_len, partition_tokens) bytes). With an explicit
 *   partition_tokens they equal a separate paged_attn_decode call bit for
 *   bit; with partition_tokens = 0 and chunks in the call, the automatic
 *   partitions are sized for one resident decode CTA per SM (the prefill
 *   grid holds SMs meanwhile), so they may round differently from a
 *   separate call. Chunk rows are the causal attention of
 *   paged_attn_prefill_chunk (max_q_len bounds every chunk); a chunk call of
 *   its own may use other tile shapes and sum in another order.
 *   Everything is enqueued on `stream`: the prefill kernel, then the decode
 *   kernel launched as a programmatic dependent of the prefill kernel, so
 *   decode CTAs start on the room the prefill grid leaves instead of
 *   waiting for it to finish (the workspace's split-KV counters reset
 *   themselves, as for paged_attn_decode). Block sizes: >= 16 when there
 *   are chunks.
 */
pkv_status paged_attn_varlen(void* out, const void* q, pkv_dtype q_dtype,
                             const void* k_cache, const void* v_cache,
                             pkv_dtype kv_dtype, const int32_t* block_tables,
                             const int32_t* seq_lens,
                             const int32_t* query_start_loc, int num_seqs,
                             int num_decode_seqs, int total_q_tokens,
                             int max_q_len, int max_decode_seq_len,
                             int num_q_heads, int num_kv_heads, int head_dim,
                             int block_size, int max_blocks_per_seq,
                             int num_blocks, float scale,
                             const float* k_scales, const float* v_scales,
                             int partition_tokens, float* out_lse,
                             void* workspace, size_t workspace_bytes,
                             void* stream);

/*
 * reshape_and_cache — write the K/V rows of new tokens into their slots.
 *   key, value: [num_tokens, Hkv, D] in src_dtype (F16 or BF16).
 *   slot_mapping: int64 [num_tokens]; slot s names block s / BS, offset
 *   s % BS; s < 0 means "write nothing" (padding tokens).
 *   For every token t and KV head h, the D values land in
 *   k_cache[s / BS][h][s % BS][:] (same for v_cache):
 *     kv_dtype == src_dtype : bit copy
 *     kv_dtype == FP8_E4M3  : code = E4M3(x / k_scales[h]) with the division
 *                             done as one correctly rounded fp32 operation
 *                             and the conversion rounding to nearest even,
 *                             saturating at +-448 (NaN stays NaN).
 *   A slot >= num_blocks * BS sets PKV_DEVERR_SLOT and is skipped.
 */
pkv_status reshape_and_cache(const void* key, const void* value,
                             pkv_dtype src_dtype, void* k_cache, void* v_cache,
                             pkv_dtype kv_dtype, const int64_t* slot_mapping,
                             int num_tokens, int num_kv_heads, int head_dim,
                             int block_size, int num_blocks,
                             const float* k_scales, const float* v_scales,
                             void* stream);

/*
 * rope_reshape_and_cache — the rotary position embedding of the new tokens'
 * queries and keys, fused with the cache write of their keys and values
 * (rvLLM, Kernel Compiler Stack, "RoPE + KV cache write -- fused, no
 * intermediate alloc"). The rotation is the rotary embedding of RoFormer:
 * each pair of dims of a head is turned by the angle of the token's position.
 *   query:  [num_tokens, Hq, D] src_dtype, rotated IN PLACE.
 *   key, value: [num_tokens, Hkv, D] src_dtype, read only; the rotated key
 *           is not stored anywhere but in the cache.
 *   positions: int64 [num_tokens], the token's position in its sequence.
 *   cos_sin_cache: fp32 [max_position, rot_dim]; row p holds rot_dim/2
 *           cosines, then rot_dim/2 sines (the model's rotary table).
 *   rot_dim: rotated dims per head, a multiple of 16 in [16, D]; dims from
 *           rot_dim on pass through unchanged.
 *   neox_style: nonzero = pair i is dims (i, i + rot_dim/2) (rotate-half);
 *           zero = pair i is dims (2i, 2i+1) (interleaved).
 *   For pair (x1, x2) and (c, s) = row positions[t], entries i, rot_dim/2+i:
 *     y1 = x1 c - x2 s,  y2 = x2 c + x1 s
 *   with both products exact in double, one rounding of the sum to double
 *   and one round-to-nearest-even to src_dtype. The key's rotated row, in
 *   src_dtype, and the value row are then written to slot_mapping[t] exactly
 *   as reshape_and_cache writes them (bit copy, or the E4M3 encode with
 *   k_scales / v_scales). Slot < 0: the query is still rotated, nothing is
 *   written. A position outside [0, max_position) sets PKV_DEVERR_POSITION:
 *   that token's query is left as it was and nothing is written; a slot
 *   >= num_blocks * BS sets PKV_DEVERR_SLOT and writes nothing.
 */
pkv_status rope_reshape_and_cache(void* query, const void* key, const void* value,
                                  pkv_dtype src_dtype, void* k_cache, void* v_cache,
                                  pkv_dtype kv_dtype, const int64_t* slot_mapping,
                                  const int64_t* positions, const float* cos_sin_cache,
                                  int max_position, int rot_dim, int neox_style,
                                  int num_tokens, int num_q_heads, int num_kv_heads,
                                  int head_dim, int block_size, int num_blocks,
                                  const float* k_scales, const float* v_scales,
                                  void* stream);

/*
 * rope_append_block_scaled — appends new tokens to a paged cache that is held
 * in E4M3 with one power-of-two scale per block of tokens and KV head
 * (PKV_FP8_E4M3_BLOCK), the rotary embedding of their queries and keys applied
 * on the way.
 *   k_cache, v_cache: E4M3 codes [num_blocks, Hkv, BS, D]; k_scales, v_scales:
 *           uint8 [num_blocks, Hkv], E8M0: a code stands for
 *           code * 2^(scale - 127) (255 is NaN).
 *   Sequence n appends rows cu_q_lens[n] .. cu_q_lens[n+1]-1 of key and value
 *           ([total_q_tokens, Hkv, D] src_dtype): its L_n tokens at positions
 *           P_n .. seq_lens[n]-1, P_n = seq_lens[n] - L_n (seq_lens includes
 *           them); token at position j goes to block block_tables[n][j / BS],
 *           offset j % BS. cu_q_lens does not decrease. L_n = 0 appends
 *           nothing; rows outside every sequence are left alone.
 *   The scale of a block and KV head, for K and for V:
 *     need = the smallest e with amax <= 448 * 2^e, e >= -60, amax the largest
 *            finite magnitude among the elements this call writes there;
 *     a block whose offset 0 the call writes starts anew with scale need;
 *     any other keeps its stored scale if that is at least need, and otherwise
 *     takes need: then every slot of it that the call does not write is
 *     re-encoded, code = E4M3(code * 2^(old - need)), exact unless the code
 *     becomes subnormal.
 *     The call's elements: code = E4M3(x * 2^-e), to nearest even, saturating
 *     at +-448 (infinities saturate, NaN stays NaN; both leave amax alone).
 *   cos_sin_cache: as in rope_reshape_and_cache, fp32 [max_position, rot_dim],
 *           the row of a token being its position; or NULL for no rotation
 *           (max_position, rot_dim, neox_style and the queries are then
 *           ignored). A rotated element is the fp32 value nearest to the exact
 *           y1 or y2, rounded to src_dtype; keys are rotated first. (Not through
 *           double as in rope_reshape_and_cache: about one element in 2^17, next
 *           to a midpoint of src_dtype, may differ by a step between the calls.)
 *   query, query_out: [total_q_tokens, Hq, D] src_dtype, the rotated queries;
 *           query_out may be query itself (in place), or both NULL.
 *   A stored scale of 255 (NaN) counts as 254, the codes beside it as they are.
 *   A block that the call writes belongs to one sequence: copy a shared,
 *   partly filled block before appending to it. (Two sequences, or two entries
 *   of one's table row, through which one block is written leave its contents
 *   undefined, nothing else.)
 *   A sequence with L_n > seq_lens[n], a context past its row of block_tables
 *   or rows outside the total_q_tokens sets PKV_DEVERR_QLEN, one with
 *   seq_lens[n] > max_position sets PKV_DEVERR_POSITION, and is skipped whole
 *   (its queries too); a block id outside [0, num_blocks) sets
 *   PKV_DEVERR_BLOCK_ID and the tokens of that block are skipped.
 *   D in {64, 128, 256}; BS 16, 32 or 64.
 */
pkv_status rope_append_block_scaled(const void* key, const void* value, pkv_dtype src_dtype,
                                    void* k_cache, void* v_cache, uint8_t* k_scales,
                                    uint8_t* v_scales, const int32_t* block_tables,
                                    const int32_t* seq_lens, const int32_t* cu_q_lens,
                                    int num_seqs, int total_q_tokens, void* query_out,
                                    const void* query, const float* cos_sin_cache,
                                    int max_position, int rot_dim, int neox_style,
                                    int num_q_heads, int num_kv_heads, int head_dim,
                                    int block_size, int max_blocks_per_seq, int num_blocks,
                                    void* stream);

/*
 * paged_attn_decode_ext_workspace_size — bytes of workspace that
 *   paged_attn_decode_ext needs (window as passed to it); 0 for invalid sizes.
 *   Query on the device that will run the call. More sequences, a larger
 *   max_seq_len or a larger window (none being the largest) never need less,
 *   the heads, head_dim and partition_tokens being the same: a workspace made
 *   for the largest call serves the smaller ones. Zero-fill the workspace once
 *   before its first use, and again after a call that ended with a device
 *   error; apart from that calls of paged_attn_decode_ext of any sizes may use
 *   it in turn, captured in graphs or not. (The other entry points with a
 *   workspace expect their counters at zero, which calls of other sizes
 *   overwrite: give them one of their own.)
 */
size_t paged_attn_decode_ext_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads,
                                            int head_dim, int max_seq_len, int window,
                                            int partition_tokens);

/*
 * paged_attn_decode_ext — paged_attn_decode over a cache with block scales,
 * or with modified scores, or both. For each sequence b, query head h (KV
 * head g) and context position j:
 *     x_j = scale * <q[b,h,:], K_j>
 *     softcap > 0:   x_j = softcap * tanh(x_j / softcap)
 *     alibi_slopes:  x_j = x_j - alibi_slopes[h] * (pos - j),  pos = seq_lens[b] - 1
 *     window > 0:    only j with pos - j < window are seen
 *     out = sum_j softmax(x)_j V_j,   lse = log sum_j exp(x_j)
 *   kv_dtype PKV_FP8_E4M3_BLOCK: k_scales, v_scales are uint8
 *   [num_blocks, Hkv] (see rope_append_block_scaled); PKV_FP8_E4M3: fp32 [Hkv];
 *   otherwise ignored. softcap = 0, window = 0 and alibi_slopes = NULL (fp32
 *   [Hq]) leave a step out. Blocks wholly outside a sequence's window are not
 *   read, and their block table entries may hold anything.
 *   scale is positive and finite, softcap finite. seq_lens[b] == 0 gives
 *   out = 0, lse = -inf. A NaN score (from q, K or a K scale of 255) makes the
 *   row's out and lse NaN, a V scale of 255 its out. (With a bf16 q over an E4M3
 *   cache a KV head's queries are scaled together: a NaN or infinity in one
 *   leaves the results of the others without meaning.) BS 16, 32 or 64; everything else as
 *   paged_attn_decode (a workspace of paged_attn_decode_ext_workspace_size()
 *   bytes, partition_tokens, errors, programmatic launch), but for contexts cut
 *   into more than 2^23 partitions, which are PKV_ERR_UNSUPPORTED.
 */
pkv_status paged_attn_decode_ext(void* out, const void* q, pkv_dtype q_dtype,
                                 const void* k_cache, const void* v_cache, pkv_dtype kv_dtype,
                                 const int32_t* block_tables, const int32_t* seq_lens,
                                 int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                 int block_size, int max_blocks_per_seq, int num_blocks,
                                 int max_seq_len, float scale, const void* k_scales,
                                 const void* v_scales, float softcap, int window,
                                 const float* alibi_slopes, int partition_tokens,
                                 float* out_lse, void* workspace, size_t workspace_bytes,
                                 void* stream);

/*
 * paged_attn_prefill_chunk_ext — paged_attn_prefill_chunk over a cache with
 * block scales, or with modified scores, or both: the steps of
 * paged_attn_decode_ext for every row of a chunk, with pos its position.
 *   prefix_lens: optional int32 [num_seqs]: positions j < prefix_lens[n] are
 *   seen by every row of sequence n, later ones included (a prefix that
 *   attends both ways); values past seq_lens[n] mean the whole context, below
 *   0 none. A row sees j < seq_lens[n] with j <= pos or j < prefix_lens[n],
 *   and, with a window, pos - j < window; the distance of the bias is
 *   |pos - j|. Blocks outside every row's window are not read. A NaN or an
 *   infinity in V may also reach rows that do not see its key, of the tokens
 *   that share a query tile (128 / G tokens) with one that does, as in
 *   paged_attn_prefill_chunk.
 *   A chunk with L_n > max_q_len sets PKV_DEVERR_QLEN and is skipped, with
 *   max_q_len = 0 every chunk that has rows (out = NULL is fine then, and the
 *   call does nothing).
 *   Everything else as paged_attn_prefill_chunk and paged_attn_decode_ext.
 */
pkv_status paged_attn_prefill_chunk_ext(void* out, const void* q, pkv_dtype q_dtype,
                                        const void* k_cache, const void* v_cache,
                                        pkv_dtype kv_dtype, const int32_t* block_tables,
                                        const int32_t* seq_lens, const int32_t* cu_q_lens,
                                        int num_seqs, int total_q_tokens, int max_q_len,
                                        int num_q_heads, int num_kv_heads, int head_dim,
                                        int block_size, int max_blocks_per_seq, int num_blocks,
                                        float scale, const void* k_scales, const void* v_scales,
                                        float softcap, int window, const float* alibi_slopes,
                                        const int32_t* prefix_lens, float* out_lse,
                                        void* stream);

/*
 * paged_attn_tree_workspace_size — bytes of workspace that paged_attn_tree needs: of
 *   the head_dim alone, whatever the sequences and their lengths. 0 for invalid sizes.
 *   Query on the device that will run the call.
 */
size_t paged_attn_tree_workspace_size(int num_q_heads, int num_kv_heads, int head_dim);

/*
 * paged_attn_tree — attention of a tree of drafted tokens of each sequence over its
 * paged cache, as a check of drafted tokens (speculative decoding) runs it.
 *   Sequence n owns query rows cu_q_lens[n] .. cu_q_lens[n+1]-1 of q and out
 *   ([total_q_tokens, Hq, D]): the L_n nodes of its tree, whose keys and values the
 *   caller has written behind the P_n = seq_lens[n] - L_n tokens before them, node m at
 *   position P_n + m (seq_lens includes the tree). With its row's 32 * mask_words bits
 *   of tree_masks [total_q_tokens, mask_words], node m in bit m % 32 of word m / 32,
 *   node i sees
 *     every position j < P_n, and position P_n + m of every m < L_n whose bit is set
 *   (its own bit too, if it is to see itself); without tree_masks (NULL) every m <= i,
 *   a chain. Any set of bits will do, an empty one too. Scores, scales and output as
 *   paged_attn_decode; kv_dtype PKV_FP8_E4M3_BLOCK as paged_attn_decode_ext (k_scales,
 *   v_scales uint8 [num_blocks, Hkv]). Positions play no part: rotate queries and keys
 *   by the nodes' depths first.
 *   A row that sees nothing gives out = 0 and lse = -inf. L_n = 0 is fine; rows outside
 *   every sequence are left alone. out is not q, nor overlaps it. out_lse: optional fp32
 *   [total_q_tokens, Hq]. No cap, window, bias or prefix: those are the _ext calls'.
 *   What a row does not see does not reach it, whatever it is. A NaN or an infinity in an
 *   element of V comes out in that element of the rows that see its key (an infinity from
 *   before the tree perhaps as NaN). A score of NaN or +infinity (from q, K or a K scale of
 *   255) makes the row's out and lse NaN, a V scale of 255 on a block that the row sees its out.
 *   workspace: 256-byte aligned, paged_attn_tree_workspace_size() bytes, with any
 *   contents; two calls that share one must not overlap on the GPU, in no other way do
 *   they depend on each other.
 *   A sequence with L_n < 0 or > seq_lens[n], with rows outside the total_q_tokens, with a
 *   context past its row of block_tables or with more nodes than mask bits sets
 *   PKV_DEVERR_QLEN and is skipped.
 *   D, BS (16, 32, 64), G and dtypes as paged_attn_decode_ext; scale positive and finite.
 *   Two kernels, each launched as a programmatic dependent of the one ahead of it.
 */
pkv_status paged_attn_tree(void* out, const void* q, pkv_dtype q_dtype, const void* k_cache,
                           const void* v_cache, pkv_dtype kv_dtype, const int32_t* block_tables,
                           const int32_t* seq_lens, const int32_t* cu_q_lens,
                           const uint32_t* tree_masks, int mask_words, int num_seqs,
                           int total_q_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                           int block_size, int max_blocks_per_seq, int num_blocks, float scale,
                           const void* k_scales, const void* v_scales, float* out_lse,
                           void* workspace, size_t workspace_bytes, void* stream);

/*
 * kv_keep_path — after a check of drafted trees: the tokens of the path that is kept move
 * to the front of the tree's places, in the K and V caches of every layer, so that the
 * sequence goes on as if it had never had another branch.
 *   k_caches, v_caches: HOST arrays of num_layers device pointers, each cache
 *           [num_blocks, Hkv, BS, D] and listed once (num_layers = 0: new_seq_lens alone).
 *           k_scales, v_scales: with PKV_FP8_E4M3_BLOCK, HOST arrays of num_layers pointers
 *           to uint8 [num_blocks, Hkv]; otherwise ignored (a scale per head moves with no
 *           token). The block tables are the layers' own common ones. Pointers are read
 *           before the call returns.
 *   Trees as for paged_attn_tree: sequence n has L_n = cu_q_lens[n+1] - cu_q_lens[n] nodes
 *           at positions P_n .. seq_lens[n] - 1.
 *   paths: int32 [num_seqs, max_path], path_lens: int32 [num_seqs]: of sequence n the
 *           nodes paths[n][0 .. path_lens[n]-1], strictly rising, each < L_n. The token at
 *           position P_n + paths[n][i] moves to position P_n + i. A path of 0 moves nothing.
 *   new_seq_lens: optional int32 [num_seqs]: P_n + path_lens[n]. A buffer of its own: not
 *           seq_lens, cu_q_lens, paths or path_lens.
 *   Positions behind the path keep what they had or what moved from there. Block scales: a
 *   block that gets tokens of the path gets them as rope_append_block_scaled would append
 *   their values (unrotated), its scale and the slots beside them too; the elements are
 *   code * 2^(scale - 127), E4M3 again with the new scale, exact unless they become
 *   subnormal. (A source scale of 255 makes NaN codes. A block whose offset 0 the path
 *   does not reach and in which no token moves is left as it is.)
 *   A path that does not rise, leaves its tree or is longer than max_path, or a tree
 *   that does not fit its context or the table's row, sets PKV_DEVERR_PATH: nothing of
 *   that sequence moves and new_seq_lens[n] = seq_lens[n]. A token whose source or
 *   destination block id is outside the pool sets PKV_DEVERR_BLOCK_ID and is skipped: its
 *   slot counts as one that no token reaches, a block of such slots alone stays as it is.
 *   Blocks from P_n on belong to one sequence. BS 1 .. 64 (block scales 16, 32, 64);
 *   D in {64, 128, 256}. One kernel for every 64 layers.
 */
pkv_status kv_keep_path(void* const* k_caches, void* const* v_caches, pkv_dtype kv_dtype,
                        void* const* k_scales, void* const* v_scales, int num_layers,
                        const int32_t* block_tables, const int32_t* seq_lens,
                        const int32_t* cu_q_lens, const int32_t* paths, const int32_t* path_lens,
                        int max_path, int32_t* new_seq_lens, int num_seqs, int num_kv_heads,
                        int head_dim, int block_size, int max_blocks_per_seq, int num_blocks,
                        void* stream);

/*
 * kv_copy_blocks — copies whole blocks: for every cache c and pair i, block
 * pairs[i][1] of caches[c] = block pairs[i][0].
 *   caches: HOST array of num_caches device pointers, block_bytes: HOST array of the bytes
 *   of a block in each (a K or V cache: Hkv * BS * D elements; block scales are one more
 *   cache, of Hkv bytes). 16-byte aligned where block_bytes is a multiple of 16. Pointers
 *   and sizes are read before the call returns. pairs: int32 [num_pairs, 2] (device).
 *   A pair with a negative entry, or of a block with itself, copies nothing; an entry >=
 *   num_blocks sets PKV_DEVERR_BLOCK_ID and the pair is skipped. A block that is the
 *   destination of two pairs, or the source of one and the destination of another, is
 *   left with undefined contents (nothing else is). One kernel for every 128 caches.
 */
pkv_status kv_copy_blocks(void* const* caches, const size_t* block_bytes, int num_caches,
                          const int32_t* pairs, int num_pairs, int num_blocks, void* stream);

/*
 * kv_fork_blocks — a table whose rows descend from another's: a step of a beam search,
 * samples of one prompt (several rows of one parent), sequences that end (none).
 *   block_tables int32 [num_rows, max_blocks_per_seq], seq_lens int32 [num_rows]: row r holds
 *   ceil(seq_lens[r] / BS) entries. ref_counts int32 [num_blocks]: how many entries name
 *   each block; 0: unused.
 *   parents int32 [num_rows]: new row r becomes row p = parents[r] of block_tables, or
 *   empty (p < 0): new_lens[r] = seq_lens[p] (0), its full blocks are shared; a partly
 *   filled last block is shared by the first new row of that parent, and each other one
 *   gets an unused block for it, the copy to make being
 *     copies[r] = (the parent's block, the new block), else (-1, -1)
 *   (int32 [num_rows, 2], as kv_copy_blocks takes it). Entries behind are -1.
 *   ref_counts: one more for each new entry, one less for each entry of block_tables, so
 *   that blocks no new row names become unused; new blocks are the lowest that are then
 *   unused, in the order of the rows. new_tables and new_lens are other buffers than
 *   block_tables, seq_lens and parents, which stay as they are.
 *   No block left: the entry and copies[r] are -1, PKV_DEVERR_POOL. Entries that are -1
 *   stay so; one >= num_blocks sets PKV_DEVERR_BLOCK_ID and is not counted. Where a parent's
 *   partly filled block is such an entry there is nothing to copy: the rows that would get
 *   a block of their own have -1 there, and copies[r] = (-1, -1). A length below
 *   0 or above the row's width counts as 0 (PKV_DEVERR_SEQ_LEN), a parent >= num_rows as
 *   none (PKV_DEVERR_PATH). A count that would fall below 0 stays (PKV_DEVERR_POOL).
 *   A partly filled last block of block_tables belongs to its row alone: the first new row
 *   of a parent goes on writing into it, whatever its count. (A fork leaves its rows so;
 *   see kv_resize_blocks for a row that is cut.)
 *   copies: 16-byte aligned. num_rows <= 16384; BS a power of two from 1 to 64. The table
 *   and counts of a pool belong to one call at a time.
 */
pkv_status kv_fork_blocks(int32_t* new_tables, int32_t* new_lens, const int32_t* block_tables,
                          const int32_t* seq_lens, const int32_t* parents, int32_t* ref_counts,
                          int32_t* copies, int num_rows, int max_blocks_per_seq, int block_size,
                          int num_blocks, void* stream);

/*
 * kv_resize_blocks — block tables take blocks for longer contexts and give back those of
 * shorter ones, in place.
 *   Row r holds ceil(seq_lens[r] / BS) entries and is to hold ceil(new_lens[r] / BS). An
 *   entry too many becomes -1 and its block's count falls by one (a block is unused at
 *   0); then each entry that is missing gets an unused block, the lowest ones in the
 *   order of the rows and of the entries in a row, whose count becomes 1. new_lens[r] = 0
 *   frees a row. Other entries are left alone; so are seq_lens and new_lens.
 *   No block left: the entry is -1, PKV_DEVERR_POOL. A row with a length below 0 or above
 *   its width is left as it is (PKV_DEVERR_SEQ_LEN). Entries, counts and sizes otherwise
 *   as for kv_fork_blocks.
 *   A row that is cut to end inside a block keeps that block, also where other rows share
 *   it (a count above 1): it may be read so, but what the row appended next would overwrite
 *   the others' tokens. For a block of its own cut the row to the block's beginning, then
 *   resize it to the length, and copy: pairs (the entry before, the entry after) for
 *   kv_copy_blocks.
 */
pkv_status kv_resize_blocks(int32_t* block_tables, const int32_t* seq_lens,
                            const int32_t* new_lens, int32_t* ref_counts, int num_rows,
                            int max_blocks_per_seq, int block_size, int num_blocks,
                            void* stream);

/*
 * pkv_get_device_error — synchronises `stream`, then reads and clears the
 * device error word of the current device. Returns PKV_OK when no check
 * failed since the last read, else PKV_ERR_DEVICE_CHECK with the PKV_DEVERR_*
 * bits in *bits (bits may be NULL). PKV_ERR_CUDA if the sync fails.
 */
pkv_status pkv_get_device_error(void* stream, unsigned int* bits);

/* Static, human-readable name of a status. */
const char* pkv_status_string(pkv_status status);

/*
 * pkv_selftest_bounded_wait — checks the failure path every kernel's waits
 * share: enqueues on `stream` one CTA whose thread waits on a shared-memory
 * mbarrier that nothing ever arrives at, with the library's bounded wait
 * limited to `polls` polls (1 .. 2^20). The wait gives up, sets
 * PKV_DEVERR_TIMEOUT in the device error word and the kernel returns; the
 * context stays usable. PKV_ERR_INVALID_ARG for polls outside the range.
 */
pkv_status pkv_selftest_bounded_wait(unsigned int polls, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_H */
