// api_ext.cu — the extern "C" entry points of the block-scaled append and of
// the attentions over block scales or with modified scores: synchronous
// argument checks, planning, and the launches.
#include <cuda.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cmath>
#include <cstdint>

#pragma GCC visibility push(default)
#include "../../include/pkv.h"
#pragma GCC visibility pop
#include "host.h"
#include "launch_ext.h"
#include "plan_ext.h"

using namespace pkv;

namespace {

constexpr float kLog2eHost = 1.4426950408889634f;

// Keys a decode plan has to cover: with a window, its keys and those before them
// on the first one's 16-token page; never more than a table's row holds
// (page_rows_fit), so that the plan's sums stay in 32 bits.
int plan_span(int max_seq_len, int window) {
  const int64_t span = std::min(max_seq_len, 1 << 30);
  return (int)(window > 0 ? std::min<int64_t>(span, (int64_t)window + 15) : span);
}

bool valid_ext_dtypes(pkv_dtype q, pkv_dtype kv) {
  return valid_dtypes(q, kv == PKV_FP8_E4M3_BLOCK ? PKV_FP8_E4M3 : kv);
}

// The checks that decode and prefill share.
pkv_status check_attn(pkv_dtype q_dtype, pkv_dtype kv_dtype, int num_seqs, int num_q_heads,
                      int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq,
                      int num_blocks, float scale, float softcap, int window) {
  if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || max_blocks_per_seq <= 0 ||
      num_blocks <= 0 || window < 0)
    return PKV_ERR_INVALID_ARG;
  if (num_q_heads % num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
  // the softmax takes its maximum before the scale: a positive one keeps the order
  if (!(scale > 0.f) || !std::isfinite(scale)) return PKV_ERR_INVALID_ARG;
  if (!(softcap >= 0.f) || !std::isfinite(softcap * kLog2eHost) ||
      (softcap > 0.f && !std::isfinite(2.f / softcap)))
    return PKV_ERR_INVALID_ARG;
  if (!valid_ext_dtypes(q_dtype, kv_dtype)) return PKV_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return PKV_ERR_UNSUPPORTED;
  if (block_log2(block_size) < 4) return PKV_ERR_UNSUPPORTED;
  if (!page_rows_fit(num_blocks, num_kv_heads, block_size, max_blocks_per_seq))
    return PKV_ERR_INVALID_ARG;
  const int G = num_q_heads / num_kv_heads;
  if (G > 16 || (head_dim > 128 && G > 8)) return PKV_ERR_UNSUPPORTED;
  if (num_seqs > 65535 || num_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
  return PKV_OK;
}

pkv_status check_tensors(const void* out, const void* q, const void* k_cache, const void* v_cache,
                         pkv_dtype kv_dtype, const void* k_scales, const void* v_scales) {
  if (!out || !q || !k_cache || !v_cache) return PKV_ERR_INVALID_ARG;
  const bool scaled = kv_dtype == PKV_FP8_E4M3 || kv_dtype == PKV_FP8_E4M3_BLOCK;
  if (scaled && (!k_scales || !v_scales)) return PKV_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
    return PKV_ERR_INVALID_ARG;
  return PKV_OK;
}

}  // namespace

extern "C" {

size_t paged_attn_decode_ext_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads,
                                            int head_dim, int max_seq_len, int window,
                                            int partition_tokens) {
  if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      max_seq_len < 0 || window < 0 || partition_tokens < 0 || partition_tokens % 16 != 0 ||
      partition_tokens > kMaxPartitionTokens)
    return 0;
  // E4M3 caches have the most resident CTAs, hence the most partitions: enough for any
  return decode_ext_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim,
                          plan_span(max_seq_len, window), partition_tokens, true, sm_count());
}

pkv_status paged_attn_decode_ext(void* out, const void* q, pkv_dtype q_dtype, const void* k_cache,
                                 const void* v_cache, pkv_dtype kv_dtype,
                                 const int32_t* block_tables, const int32_t* seq_lens,
                                 int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                 int block_size, int max_blocks_per_seq, int num_blocks,
                                 int max_seq_len, float scale, const void* k_scales,
                                 const void* v_scales, float softcap, int window,
                                 const float* alibi_slopes, int partition_tokens, float* out_lse,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  if (max_seq_len < 0 || partition_tokens < 0 || partition_tokens % 16 != 0 ||
      partition_tokens > kMaxPartitionTokens)
    return PKV_ERR_INVALID_ARG;
  pkv_status st = check_attn(q_dtype, kv_dtype, num_seqs, num_q_heads, num_kv_heads, head_dim,
                             block_size, max_blocks_per_seq, num_blocks, scale, softcap, window);
  if (st != PKV_OK || num_seqs == 0) return st;
  if (!block_tables || !seq_lens) return PKV_ERR_INVALID_ARG;
  st = check_tensors(out, q, k_cache, v_cache, kv_dtype, k_scales, v_scales);
  if (st != PKV_OK) return st;

  const int sms = sm_count();
  const int span = plan_span(max_seq_len, window);
  const bool block_scaled = kv_dtype == PKV_FP8_E4M3_BLOCK;
  const pkv_dtype page_dtype = block_scaled ? PKV_FP8_E4M3 : kv_dtype;
  const DecodePlan pl = plan_decode_ext(num_seqs, num_q_heads, num_kv_heads, head_dim, span,
                                        partition_tokens, page_dtype == PKV_FP8_E4M3, sms);
  if (pl.max_parts > kMaxDecodeExtParts) return PKV_ERR_UNSUPPORTED;
  const size_t need = decode_ext_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, span,
                                       partition_tokens, page_dtype == PKV_FP8_E4M3, sms);
  if (workspace == nullptr || workspace_bytes < need ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return PKV_ERR_WORKSPACE;
  const int shift = page_shift(block_size), bs_log2 = block_log2(block_size);
  CUtensorMap tmK, tmV;
  if (!make_kv_tmap(&tmK, k_cache, page_dtype, head_dim, num_kv_heads, num_blocks, shift) ||
      !make_kv_tmap(&tmV, v_cache, page_dtype, head_dim, num_kv_heads, num_blocks, shift))
    return PKV_ERR_CUDA;
  unsigned int* err = err_word();
  if (err == nullptr) return PKV_ERR_CUDA;
  char* ws = static_cast<char*>(workspace);
  DecodeExtParams ep{};
  DecodeParams& p = ep.base;
  p.out = out;
  p.q = q;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  if (block_scaled) {
    ep.k_block_scales = static_cast<const uint8_t*>(k_scales);
    ep.v_block_scales = static_cast<const uint8_t*>(v_scales);
  } else {
    p.k_scales = static_cast<const float*>(k_scales);
    p.v_scales = static_cast<const float*>(v_scales);
  }
  p.out_lse = out_lse;
  p.done = reinterpret_cast<unsigned long long*>(ws + pl.off_done);
  p.ws_o = reinterpret_cast<float*>(ws + pl.off_o);
  p.ws_lse = reinterpret_cast<float*>(ws + pl.off_lse);
  p.err = err;
  p.B = num_seqs;
  p.Hq = num_q_heads;
  p.Hkv = num_kv_heads;
  p.G = num_q_heads / num_kv_heads;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.max_seq_len = max_seq_len;
  p.ppb_shift = shift;
  p.bs_log2 = bs_log2;
  p.part = pl.part;
  p.max_parts = pl.max_parts;
  p.wide = wide_decode((int64_t)num_seqs * num_kv_heads, sms, span, partition_tokens, bs_log2,
                       head_dim, kDecodeWorkers) ? 1 : 0;
  if (p.wide) p.part = std::max(16, (span + 15) / 16 * 16);   // one partition
  p.grid_parts = std::max(1, (span + p.part - 1) / p.part);
  p.qk_scale_log2 = scale * kLog2eHost;
  ep.slopes = alibi_slopes;
  ep.cap_log2 = softcap * kLog2eHost;
  ep.two_over_cap = softcap > 0.f ? 2.f / softcap : 0.f;
  ep.window = window;
  return launch_decode_ext(ep, head_dim, q_dtype, page_dtype, block_scaled, tmK, tmV,
                           reinterpret_cast<cudaStream_t>(stream));
}

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
                                        void* stream) {
  if (total_q_tokens < 0 || max_q_len < 0) return PKV_ERR_INVALID_ARG;
  pkv_status st = check_attn(q_dtype, kv_dtype, num_seqs, num_q_heads, num_kv_heads, head_dim,
                             block_size, max_blocks_per_seq, num_blocks, scale, softcap, window);
  if (st != PKV_OK || num_seqs == 0 || total_q_tokens == 0) return st;
  if (max_q_len == 0 && out == nullptr) return PKV_OK;   // no chunk, and nowhere to put one
  if (!block_tables || !seq_lens || !cu_q_lens) return PKV_ERR_INVALID_ARG;
  st = check_tensors(out, q, k_cache, v_cache, kv_dtype, k_scales, v_scales);
  if (st != PKV_OK) return st;
  const bool block_scaled = kv_dtype == PKV_FP8_E4M3_BLOCK;
  const pkv_dtype page_dtype = block_scaled ? PKV_FP8_E4M3 : kv_dtype;
  const int shift = page_shift(block_size);
  CUtensorMap tmQ{}, tmK, tmV;
  if (!make_kv_tmap(&tmK, k_cache, page_dtype, head_dim, num_kv_heads, num_blocks, shift) ||
      !make_kv_tmap(&tmV, v_cache, page_dtype, head_dim, num_kv_heads, num_blocks, shift))
    return PKV_ERR_CUDA;
  const int G = num_q_heads / num_kv_heads;
  if (page_dtype != PKV_FP8_E4M3 &&
      !make_q_tmap(&tmQ, q, head_dim, num_q_heads, G, kPrefillTcRows / G, total_q_tokens))
    return PKV_ERR_CUDA;
  unsigned int* err = err_word();
  if (err == nullptr) return PKV_ERR_CUDA;
  PrefillExtParams ep{};
  PrefillParams& p = ep.base;
  p.out = out;
  p.q = q;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.cu_q_lens = cu_q_lens;
  if (block_scaled) {
    ep.k_block_scales = static_cast<const uint8_t*>(k_scales);
    ep.v_block_scales = static_cast<const uint8_t*>(v_scales);
  } else {
    p.k_scales = static_cast<const float*>(k_scales);
    p.v_scales = static_cast<const float*>(v_scales);
  }
  p.out_lse = out_lse;
  p.err = err;
  p.num_seqs = num_seqs;
  p.Hq = num_q_heads;
  p.Hkv = num_kv_heads;
  p.G = G;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  // no chunk is longer than the rows there are (with 0 every chunk that has a row is
  // flagged)
  p.max_q_len = std::min(max_q_len, total_q_tokens);
  p.q_rows = total_q_tokens;
  p.ppb_shift = shift;
  p.qk_scale_log2 = scale * kLog2eHost;
  ep.slopes = alibi_slopes;
  ep.prefix_lens = prefix_lens;
  ep.cap_log2 = softcap * kLog2eHost;
  ep.two_over_cap = softcap > 0.f ? 2.f / softcap : 0.f;
  ep.window = window;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return block_scaled ? launch_prefill_block(ep, head_dim, q_dtype, tmQ, tmK, tmV, s)
                      : launch_prefill_mod(ep, head_dim, q_dtype, kv_dtype, tmQ, tmK, tmV, s);
}

pkv_status rope_append_block_scaled(const void* key, const void* value, pkv_dtype src_dtype,
                                    void* k_cache, void* v_cache, uint8_t* k_scales,
                                    uint8_t* v_scales, const int32_t* block_tables,
                                    const int32_t* seq_lens, const int32_t* cu_q_lens,
                                    int num_seqs, int total_q_tokens, void* query_out,
                                    const void* query, const float* cos_sin_cache,
                                    int max_position, int rot_dim, int neox_style,
                                    int num_q_heads, int num_kv_heads, int head_dim,
                                    int block_size, int max_blocks_per_seq, int num_blocks,
                                    void* stream) {
  if (num_seqs < 0 || total_q_tokens < 0 || num_kv_heads <= 0 || max_blocks_per_seq <= 0 ||
      num_blocks <= 0)
    return PKV_ERR_INVALID_ARG;
  if (src_dtype != PKV_F16 && src_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return PKV_ERR_UNSUPPORTED;
  if (block_log2(block_size) < 4) return PKV_ERR_UNSUPPORTED;
  if (!page_rows_fit(num_blocks, num_kv_heads, block_size, max_blocks_per_seq))
    return PKV_ERR_INVALID_ARG;
  const bool rotate = cos_sin_cache != nullptr;
  if (rotate) {
    if (max_position <= 0 || rot_dim < 16 || rot_dim > head_dim || rot_dim % 16 != 0)
      return PKV_ERR_INVALID_ARG;
    if ((query == nullptr) != (query_out == nullptr)) return PKV_ERR_INVALID_ARG;
    if (query != nullptr && num_q_heads <= 0) return PKV_ERR_INVALID_ARG;
    if (!aligned16(cos_sin_cache) || !aligned16(query) || !aligned16(query_out))
      return PKV_ERR_INVALID_ARG;
  }
  if (num_seqs == 0 || total_q_tokens == 0) return PKV_OK;
  if (!key || !value || !k_cache || !v_cache || !k_scales || !v_scales || !block_tables ||
      !seq_lens || !cu_q_lens)
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(key) || !aligned16(value) || !aligned16(k_cache) || !aligned16(v_cache))
    return PKV_ERR_INVALID_ARG;
  unsigned int* err = err_word();
  if (err == nullptr) return PKV_ERR_CUDA;
  AppendBlockParams p{};
  p.key = key;
  p.value = value;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.cu_q_lens = cu_q_lens;
  p.query_out = rotate ? query_out : nullptr;
  p.query = query;
  p.cos_sin = cos_sin_cache;
  p.err = err;
  p.max_position = max_position;
  p.rot = rot_dim;
  p.neox = neox_style != 0;
  p.num_seqs = num_seqs;
  p.rows = total_q_tokens;
  p.Hq = num_q_heads;
  p.Hkv = num_kv_heads;
  p.d_log2 = head_dim == 64 ? 6 : head_dim == 128 ? 7 : 8;
  p.max_blocks = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.bs_log2 = block_log2(block_size);
  return launch_append_block(p, src_dtype, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
