// api_tree.cu — the extern "C" entry points for drafted trees of tokens and the pages they
// need: synchronous argument checks and the launches.
#include <cuda_runtime.h>
#include <algorithm>
#include <cstdint>

#pragma GCC visibility push(default)
#include "../../include/pkv.h"
#pragma GCC visibility pop
#include "host.h"
#include "launch_pages.h"
#include "launch_tree.h"

using namespace pkv;

namespace {

constexpr float kLog2eHost = 1.4426950408889634f;

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

extern "C" {

size_t paged_attn_tree_workspace_size(int num_q_heads, int num_kv_heads, int head_dim) {
  if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
      (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return 0;
  return tree_workspace_bytes(sm_count(), head_dim);
}

pkv_status paged_attn_tree(void* out, const void* q, pkv_dtype q_dtype, const void* k_cache,
                           const void* v_cache, pkv_dtype kv_dtype, const int32_t* block_tables,
                           const int32_t* seq_lens, const int32_t* cu_q_lens,
                           const uint32_t* tree_masks, int mask_words, int num_seqs,
                           int total_q_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                           int block_size, int max_blocks_per_seq, int num_blocks, float scale,
                           const void* k_scales, const void* v_scales, float* out_lse,
                           void* workspace, size_t workspace_bytes, void* stream) {
  if (total_q_tokens < 0 || (tree_masks != nullptr && mask_words <= 0)) return PKV_ERR_INVALID_ARG;
  pkv_status st = check_attn(q_dtype, kv_dtype, num_seqs, num_q_heads, num_kv_heads, head_dim,
                             block_size, max_blocks_per_seq, num_blocks, scale, 0.f, 0);
  if (st != PKV_OK || num_seqs == 0 || total_q_tokens == 0) return st;
  if (!block_tables || !seq_lens || !cu_q_lens) return PKV_ERR_INVALID_ARG;
  st = check_tensors(out, q, k_cache, v_cache, kv_dtype, k_scales, v_scales);
  if (st != PKV_OK) return st;
  if (out == q) return PKV_ERR_INVALID_ARG;   // one CTA would write rows that another has to read
  const int ctas = sm_count();
  if (ctas <= 0) return PKV_ERR_CUDA;
  if (workspace == nullptr || workspace_bytes < tree_workspace_bytes(ctas, head_dim) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return PKV_ERR_WORKSPACE;
  const bool block_scaled = kv_dtype == PKV_FP8_E4M3_BLOCK;
  unsigned int* err = err_word();
  if (err == nullptr) return PKV_ERR_CUDA;
  TreeParams p{};
  p.out = out;
  p.q = q;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.cu_q_lens = cu_q_lens;
  p.masks = tree_masks;
  p.mask_words = tree_masks != nullptr ? mask_words : 0;
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  if (kv_dtype == PKV_FP8_E4M3) p.v_head_scales = static_cast<const float*>(v_scales);
  p.out_lse = out_lse;
  p.err = err;
  p.part_o = static_cast<float*>(workspace);
  p.part_lse = p.part_o + (size_t)ctas * kTreeParts * tree_part_floats(head_dim);
  p.splits = reinterpret_cast<TreeSplit*>(p.part_lse + (size_t)ctas * kTreeParts * kTreeRows);
  p.odd = reinterpret_cast<TreeOdd*>(p.splits + ctas + 1);
  p.kv_dtype = kv_dtype;
  p.num_seqs = num_seqs;
  p.Hq = num_q_heads;
  p.Hkv = num_kv_heads;
  p.G = num_q_heads / num_kv_heads;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.q_rows = total_q_tokens;
  p.q_tile = kTreeRows / p.G;
  p.ppb_shift = page_shift(block_size);
  p.ctas = ctas;
  p.qk_scale_log2 = scale * kLog2eHost;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  st = block_scaled                ? launch_tree_e4m3_block(p, head_dim, q_dtype, s)
       : kv_dtype == PKV_FP8_E4M3 ? launch_tree_e4m3_head(p, head_dim, q_dtype, s)
                                   : launch_tree_16bit(p, head_dim, q_dtype, s);
  return st == PKV_OK ? launch_tree_merge(p, head_dim, q_dtype, s) : st;
}

pkv_status kv_copy_blocks(void* const* caches, const size_t* block_bytes, int num_caches,
                          const int32_t* pairs, int num_pairs, int num_blocks, void* stream) {
  if (num_caches < 0 || num_pairs < 0 || num_blocks <= 0) return PKV_ERR_INVALID_ARG;
  if (num_caches == 0 || num_pairs == 0) return PKV_OK;
  if (!caches || !block_bytes || !pairs || !aligned4(pairs)) return PKV_ERR_INVALID_ARG;
  for (int c = 0; c < num_caches; ++c)
    if (!caches[c] || block_bytes[c] == 0 || block_bytes[c] > ((size_t)1 << 32) ||
        (block_bytes[c] % 16 == 0 && !aligned16(caches[c])))
      return PKV_ERR_INVALID_ARG;
  unsigned int* err = err_word();
  const int sms = sm_count();
  if (err == nullptr || sms <= 0) return PKV_ERR_CUDA;
  for (int c0 = 0; c0 < num_caches; c0 += kCachesPerLaunch) {
    CopyBlocksParams p;
    p.num_caches = std::min(kCachesPerLaunch, num_caches - c0);
    for (int c = 0; c < p.num_caches; ++c) {
      p.cache[c] = static_cast<uint8_t*>(caches[c0 + c]);
      p.bytes[c] = (int64_t)block_bytes[c0 + c];
    }
    p.pairs = pairs;
    p.num_pairs = num_pairs;
    p.num_blocks = num_blocks;
    p.err = err;
    const pkv_status st = launch_copy_blocks(p, sms, reinterpret_cast<cudaStream_t>(stream));
    if (st != PKV_OK) return st;
  }
  return PKV_OK;
}

pkv_status kv_keep_path(void* const* k_caches, void* const* v_caches, pkv_dtype kv_dtype,
                        void* const* k_scales, void* const* v_scales, int num_layers,
                        const int32_t* block_tables, const int32_t* seq_lens,
                        const int32_t* cu_q_lens, const int32_t* paths, const int32_t* path_lens,
                        int max_path, int32_t* new_seq_lens, int num_seqs, int num_kv_heads,
                        int head_dim, int block_size, int max_blocks_per_seq, int num_blocks,
                        void* stream) {
  if (num_layers < 0 || num_seqs < 0 || max_path < 0 || num_kv_heads <= 0 ||
      max_blocks_per_seq <= 0 || num_blocks <= 0)
    return PKV_ERR_INVALID_ARG;
  const bool block_scaled = kv_dtype == PKV_FP8_E4M3_BLOCK;
  if (kv_dtype != PKV_F16 && kv_dtype != PKV_BF16 && kv_dtype != PKV_FP8_E4M3 && !block_scaled)
    return PKV_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return PKV_ERR_UNSUPPORTED;
  if (block_log2(block_size) < 0 || (block_scaled && block_log2(block_size) < 4))
    return PKV_ERR_UNSUPPORTED;
  if (num_seqs > 65535 || num_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
  if (!page_rows_fit(num_blocks, num_kv_heads, block_size, max_blocks_per_seq))
    return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0 || (num_layers == 0 && new_seq_lens == nullptr)) return PKV_OK;
  if (!block_tables || !seq_lens || !cu_q_lens || !path_lens || (max_path > 0 && !paths) ||
      (new_seq_lens != nullptr && (new_seq_lens == seq_lens || new_seq_lens == cu_q_lens ||
                                   new_seq_lens == paths || new_seq_lens == path_lens)))
    return PKV_ERR_INVALID_ARG;             // (one CTA would write what another has to read)
  if (num_layers > 0 && (!k_caches || !v_caches || (block_scaled && (!k_scales || !v_scales))))
    return PKV_ERR_INVALID_ARG;
  for (int c = 0; c < num_layers; ++c) {
    if (!k_caches[c] || !v_caches[c] || !aligned16(k_caches[c]) || !aligned16(v_caches[c]))
      return PKV_ERR_INVALID_ARG;
    if (block_scaled && (!k_scales[c] || !v_scales[c])) return PKV_ERR_INVALID_ARG;
  }
  unsigned int* err = err_word();
  if (err == nullptr) return PKV_ERR_CUDA;
  constexpr int kLayers = kCachesPerLaunch / 2;
  for (int c0 = 0; c0 == 0 || c0 < num_layers; c0 += kLayers) {
    const int layers = std::min(kLayers, num_layers - c0);
    KeepPathParams p{};
    for (int c = 0; c < layers; ++c) {
      p.cache[c] = static_cast<uint8_t*>(k_caches[c0 + c]);
      p.cache[layers + c] = static_cast<uint8_t*>(v_caches[c0 + c]);
      if (!block_scaled) continue;
      p.scales[c] = static_cast<uint8_t*>(k_scales[c0 + c]);
      p.scales[layers + c] = static_cast<uint8_t*>(v_scales[c0 + c]);
    }
    p.num_caches = 2 * layers;
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.cu_q_lens = cu_q_lens;
    p.paths = paths;
    p.path_lens = path_lens;
    p.new_seq_lens = c0 == 0 ? new_seq_lens : nullptr;
    p.err = err;
    p.num_seqs = num_seqs;
    p.Hkv = num_kv_heads;
    p.max_path = max_path;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.row_bytes = head_dim * (kv_dtype == PKV_F16 || kv_dtype == PKV_BF16 ? 2 : 1);
    p.bs_log2 = block_log2(block_size);
    const pkv_status st =
        launch_keep_path(p, block_scaled, reinterpret_cast<cudaStream_t>(stream));
    if (st != PKV_OK) return st;
  }
  return PKV_OK;
}

pkv_status kv_fork_blocks(int32_t* new_tables, int32_t* new_lens, const int32_t* block_tables,
                          const int32_t* seq_lens, const int32_t* parents, int32_t* ref_counts,
                          int32_t* copies, int num_rows, int max_blocks_per_seq, int block_size,
                          int num_blocks, void* stream) {
  if (num_rows < 0 || max_blocks_per_seq <= 0 || num_blocks <= 0) return PKV_ERR_INVALID_ARG;
  if (block_log2(block_size) < 0 || num_rows > kMaxPoolRows) return PKV_ERR_UNSUPPORTED;
  if ((int64_t)max_blocks_per_seq * block_size >= ((int64_t)1 << 30) ||
      num_blocks > (1 << 30))
    return PKV_ERR_INVALID_ARG;
  if (num_rows == 0) return PKV_OK;
  if (!new_tables || !new_lens || !block_tables || !seq_lens || !parents || !ref_counts ||
      !copies || new_tables == block_tables || new_lens == seq_lens || new_lens == parents ||
      !aligned16(copies))
    return PKV_ERR_INVALID_ARG;
  unsigned int* err = err_word();
  if (err == nullptr) return PKV_ERR_CUDA;
  ForkParams p{};
  p.new_tables = new_tables;
  p.new_lens = new_lens;
  p.tables = block_tables;
  p.lens = seq_lens;
  p.parents = parents;
  p.refs = ref_counts;
  p.copies = copies;
  p.err = err;
  p.rows = num_rows;
  p.width = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.bs_log2 = block_log2(block_size);
  return launch_fork(p, reinterpret_cast<cudaStream_t>(stream));
}

pkv_status kv_resize_blocks(int32_t* block_tables, const int32_t* seq_lens,
                            const int32_t* new_lens, int32_t* ref_counts, int num_rows,
                            int max_blocks_per_seq, int block_size, int num_blocks,
                            void* stream) {
  if (num_rows < 0 || max_blocks_per_seq <= 0 || num_blocks <= 0) return PKV_ERR_INVALID_ARG;
  if (block_log2(block_size) < 0 || num_rows > kMaxPoolRows) return PKV_ERR_UNSUPPORTED;
  if ((int64_t)max_blocks_per_seq * block_size >= ((int64_t)1 << 30) ||
      (int64_t)max_blocks_per_seq * num_rows >= ((int64_t)1 << 31) || num_blocks > (1 << 30))
    return PKV_ERR_INVALID_ARG;
  if (num_rows == 0) return PKV_OK;
  if (!block_tables || !seq_lens || !new_lens || !ref_counts) return PKV_ERR_INVALID_ARG;
  unsigned int* err = err_word();
  if (err == nullptr) return PKV_ERR_CUDA;
  ResizeParams p{};
  p.tables = block_tables;
  p.lens = seq_lens;
  p.new_lens = new_lens;
  p.refs = ref_counts;
  p.err = err;
  p.rows = num_rows;
  p.width = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.bs_log2 = block_log2(block_size);
  return launch_resize(p, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
