// launch_ext.h — host-side parameter blocks and launchers of the
// block-scaled append and of the attentions over block scales or with
// modified scores (not part of the public ABI).
#pragma once
#include "launch.h"
#include "launch_prefill.h"

namespace pkv {

struct AppendBlockParams {
  const void* key;
  const void* value;
  void* k_cache;
  void* v_cache;
  uint8_t* k_scales;
  uint8_t* v_scales;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* cu_q_lens;
  void* query_out;              // null: no queries
  const void* query;
  const float* cos_sin;         // null: no rotation
  unsigned int* err;
  int64_t max_position;         // longest context that the rotary table covers
  int rot, neox, num_seqs, rows, Hq, Hkv, max_blocks, num_blocks;
  int d_log2;                   // log2(head_dim)
  int bs_log2;                  // log2(block_size), 4 to 6
  int window;                   // rows per cache-write CTA (at most 32)
  unsigned int kv_ctas;         // cache-write CTAs, the first of the grid
  int slices_log2;              // log2 of the warps per row of queries
};

// Launches nothing for rows = 0; validates nothing (the entry point does).
pkv_status launch_append_block(const AppendBlockParams& p, pkv_dtype src_dtype,
                               cudaStream_t stream);

// Decode over block scales and/or with modified scores. `base`: the plan, the
// workspace and the tensors as for paged_attn_decode (its k_scales / v_scales
// hold per-head scales; wpart, full_first and early are not used).
struct DecodeExtParams {
  DecodeParams base;
  const uint8_t* k_block_scales;    // E8M0 [num_blocks, Hkv], or null: no block scales
  const uint8_t* v_block_scales;
  const float* slopes;              // ALiBi slopes [Hq], or null
  float cap_log2;                   // softcap * log2(e), 0 = off
  float two_over_cap;               // 2 / softcap
  int window;                       // keys seen, counting the newest; 0 = all
};

// block_scaled: E4M3 pages with block scales (kv_dtype is then PKV_FP8_E4M3).
pkv_status launch_decode_ext(const DecodeExtParams& p, int head_dim, pkv_dtype q_dtype,
                             pkv_dtype kv_dtype, bool block_scaled, const CUtensorMap& tmK,
                             const CUtensorMap& tmV, cudaStream_t stream);
pkv_status launch_decode_ext_wide(const DecodeExtParams& p, int head_dim, pkv_dtype q_dtype,
                                  pkv_dtype kv_dtype, bool block_scaled, const CUtensorMap& tmK,
                                  const CUtensorMap& tmV, cudaStream_t stream);

// Prefill over block scales and/or with modified scores. `base` as for
// paged_attn_prefill_chunk.
struct PrefillExtParams {
  PrefillParams base;
  const uint8_t* k_block_scales;    // E8M0 [num_blocks, Hkv], or null: no block scales
  const uint8_t* v_block_scales;
  const float* slopes;              // ALiBi slopes [Hq], or null
  const int32_t* prefix_lens;       // [num_seqs], or null
  float cap_log2;                   // softcap * log2(e), 0 = off
  float two_over_cap;               // 2 / softcap
  int window;                       // keys a row sees, counting its own; 0 = all
};

// Over block scales (E4M3, head_dim 64, 128 or 256), with modified scores or not.
// tmQ as for launch_prefill_tc.
pkv_status launch_prefill_block(const PrefillExtParams& p, int head_dim, pkv_dtype q_dtype,
                                const CUtensorMap& tmQ, const CUtensorMap& tmK,
                                const CUtensorMap& tmV, cudaStream_t stream);
// Over the other caches, with modified scores (or none).
pkv_status launch_prefill_mod(const PrefillExtParams& p, int head_dim, pkv_dtype q_dtype,
                              pkv_dtype kv_dtype, const CUtensorMap& tmQ,
                              const CUtensorMap& tmK, const CUtensorMap& tmV,
                              cudaStream_t stream);

}  // namespace pkv
