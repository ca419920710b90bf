// plan_ext.h — the split-KV plan of paged_attn_decode_ext (host code). The
// workspace layout is plan.h's; partitions are sized by another rule, which also
// covers the calls that leave most of the GPU idle.
#pragma once
#include <algorithm>
#include <cmath>
#include "plan.h"

namespace pkv {

// Partitions of a context: a count of them is told from two floats by being smaller
// than the bits of any normal one.
constexpr int kMaxDecodeExtParts = 1 << 23;

// CTAs of kDecodeWarps warps an SM holds by the shared memory of their rings (3 stages of
// E4M3 pages or 2 of 16-bit ones per warp, K and V), 8 at most. Registers hold fewer at
// head_dim 64 (7 of E4M3 pages; with more than 8 heads to a KV head 4) and, with more
// than 8, at 128 (2 of 4): such a call may take a second wave, which costs time alone.
inline int decode_ext_ctas_per_sm(int head_dim, bool e4m3) {
  const int page = 16 * head_dim * (e4m3 ? 1 : 2);
  const int smem = 4096 + kDecodeWarps * (e4m3 ? 3 : 2) * 2 * page;
  return std::max(1, std::min(8, 227 * 1024 / smem));
}

// Tokens of a partition of `span` keys for a call alone on the GPU (below).
inline int best_part(int span) { return std::max(64, (int)std::sqrt(16.0 * std::max(0, span))); }

// Automatic partitions (partition_tokens = 0) of `span` keys:
//  - A call alone on the GPU takes about a + b * part + c * parts: a CTA reads a
//    token in b = 0.01 us (head_dim 128, E4M3), the merging CTA a partition in c =
//    0.1 to 0.16 us, so parts of sqrt(16 span) tokens cost least (one sequence, 8
//    KV heads: 700 keys 11.4 us in parts of 512, 7.4 in parts of 112; 4,000 keys
//    11.8 in 512, 9.1 in 256; 32,000 keys 23.6 in 512, 22.6 in 1,024);
//  - but no more parts than keep every CTA resident at once, while one wave can
//    hold the call: a second wave that is mostly empty costs as much as the first
//    (16 sequences of 4,000: 4 parts 30.6 us, 6 parts 37.8; 64 of 700: one part
//    21.7, two 30.4);
//  - and no part above 2,048 tokens, so that long uneven contexts share the GPU
//    (4 sequences of 32 K to 128 K: 133 us in 2,048, 158 in 4,096).
inline DecodePlan plan_decode_ext(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                  int span, int partition_tokens, bool e4m3, int sms) {
  int part = partition_tokens;
  if (part <= 0) {
    if (sms <= 0) sms = 148;
    const int64_t units = std::max<int64_t>(1, (int64_t)num_seqs * num_kv_heads);
    const int64_t resident = (int64_t)sms * decode_ext_ctas_per_sm(head_dim, e4m3);
    const int best = best_part(span);
    const int64_t parts =
        std::min<int64_t>(std::max(1, (span + best - 1) / best), std::max<int64_t>(1, resident / units));
    part = (int)std::min<int64_t>(2048, ((span + parts - 1) / parts + 15) / 16 * 16);
    part = std::max(16, part);
  }
  // (an explicit size: the same layout)
  return plan_decode(num_seqs, num_q_heads, num_kv_heads, head_dim, span, part, sms);
}

// Bytes that paged_attn_decode_ext asks for: enough for its plan and for those of every
// call with as many sequences and keys or fewer, so that a workspace made for the
// largest batch serves the smaller ones, whose contexts are split into more parts.
inline size_t decode_ext_bytes(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                               int span, int partition_tokens, bool e4m3, int sms) {
  int64_t parts;                                   // of all sequences, a KV head
  if (partition_tokens > 0) {
    parts = num_seqs * std::max<int64_t>(1, ((int64_t)span + partition_tokens - 1) / partition_tokens);
  } else {
    if (sms <= 0) sms = 148;
    const int64_t resident = (int64_t)sms * decode_ext_ctas_per_sm(head_dim, e4m3);
    // the most parts of up to `span` keys: of these, or of the longest with the next
    // smaller best part
    const int64_t k = best_part(span), below = (k * k - 1) / 16;
    int64_t most = std::max<int64_t>(1, ((int64_t)span + k - 1) / k);
    if (k > 64) most = std::max(most, (below + k - 2) / (k - 1));
    parts = std::max(std::min(num_seqs * most, std::max<int64_t>(num_seqs, resident / num_kv_heads)),
                     num_seqs * (((int64_t)span + 2047) / 2048));
  }
  const size_t rows = (size_t)parts * num_q_heads;
  return align256((size_t)num_seqs * num_kv_heads * 8) + align256(rows * head_dim * sizeof(float)) +
         align256(rows * sizeof(float));
}

}  // namespace pkv
