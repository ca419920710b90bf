// tree_work.cuh — how the key tiles of a call are cut into ranges and walked through, and which
// nodes of a tree a node sees: what the tree attention (tree_kernel.cuh) and its merge
// (tree_merge.cu) share.
#pragma once
#include "common.cuh"
#include "launch_tree.h"

namespace pkv {

template <int KEYS>
__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, int q0, int q1, int ctx,
                                            bool* bad = nullptr) {
  TreeSeq s{q0, q1 - q0, ctx, 0, 0};
  const bool refused = s.L < 0 || s.L > ctx || q0 < 0 || q0 > p.q_rows - s.L ||
                       ctx > ((p.max_blocks * kBS) << p.ppb_shift) ||
                       (p.masks != nullptr && s.L > 32 * (int64_t)p.mask_words);
  if (bad != nullptr) *bad = refused;
  if (refused || s.L == 0) return s;
  s.kt = (ctx + KEYS - 1) / KEYS;
  s.rt = (s.L + p.q_tile - 1) / p.q_tile;
  return s;
}

// A CTA's range of key tiles as its warps walk through it, segment by segment.
template <int KEYS, bool OUT_OF_LINE>
struct TreeWork {
  const TreeParams* p;
  int left;                           // key tiles of the range behind this segment
  TreeSeq s;                          // this segment's sequence
  int n, h, r;                        // sequence, KV head, row tile
  int t0, cnt;                        // key tiles [t0, t0 + cnt) of the item; cnt = 0: done
  int nq0, nq1, nctx;                 // as they stand in memory: sequence n + 1

  __device__ __forceinline__ void peek() {
    nq0 = nq1 = nctx = 0;
    if (n + 1 < p->num_seqs) {
      nq0 = p->cu_q_lens[n + 1];
      nq1 = p->cu_q_lens[n + 2];
      nctx = p->seq_lens[n + 1];
    }
  }
  __device__ __forceinline__ void take() {
    cnt = min(s.kt - t0, left);
    left -= cnt;
  }
  // The range of `total` key tiles that begins with key tile `start.t0` of an item.
  __device__ __forceinline__ TreeWork(const TreeParams& params, const TreeStart& start, int total)
      : p(&params), left(total), s(start.s), n(start.n), h(start.h), r(start.r), t0(start.t0),
        cnt(0) {
    if (total <= 0) return;
    peek();
    take();
  }
  __device__ __forceinline__ void step() {
    if (left <= 0) {
      cnt = 0;
      return;
    }
    t0 = 0;
    if (++r == s.rt) {
      r = 0;
      if (++h == p->Hkv) {
        h = 0;
        do {
          s = tree_seq<KEYS>(*p, nq0, nq1, nctx);
          ++n;
          peek();
        } while (s.rt == 0 && n < p->num_seqs);
      }
    }
    take();
  }
  __device__ __noinline__ static TreeWork stepped(TreeWork w) {
    w.step();
    return w;
  }
  // The next segment. Six places take it, in 3 KB of code each: with an E4M3 cache, whose
  // producers have more code than a copy, out of line (365 us on four contexts of 80,000 of 8
  // bits, so 361, and 93 on eight of 16,384 with block scales, so 91; but 128 of 1,024 with a scale
  // per head 128, so 132. A small tree over 16 bits 12.4 us, so 12.7, and 128 of 1,024 121, so 124).
  __device__ __forceinline__ void next() {
    if constexpr (OUT_OF_LINE) *this = stepped(*this);
    else step();
  }
  // Keys of the sequence before its tree, this item's first node and its nodes.
  __device__ __forceinline__ int before() const { return s.ctx - s.L; }
  __device__ __forceinline__ int node0() const { return r * p->q_tile; }
  __device__ __forceinline__ int nodes() const { return min(p->q_tile, s.L - node0()); }
};

// Which of the 64 keys from place m0 of a tree on a node sees (m0 may be negative: keys
// before the tree, which every row sees). node: its row of q; i: its place in the tree.
__device__ __forceinline__ uint64_t tree_sees(const TreeParams& p, int node, int i, int m0, int L) {
  if (m0 <= -64) return ~(uint64_t)0;
  if (p.masks == nullptr) {
    const int last = i - m0;          // the last one seen
    return last < 0 ? 0u : last >= 63 ? ~(uint64_t)0 : ((uint64_t)2 << last) - 1;
  }
  const uint32_t* row = p.masks + (int64_t)node * p.mask_words;
  auto word = [&](int k) { return k >= 0 && k < p.mask_words ? row[k] : 0u; };
  const int k = m0 >> 5, s = m0 & 31;
  const uint32_t a = word(k), b = word(k + 1), c = word(k + 2);
  uint64_t w = ((uint64_t)__funnelshift_r(b, c, s) << 32) | __funnelshift_r(a, b, s);
  const int end = L - m0;             // nodes behind the last
  if (end < 64) w &= end <= 0 ? 0u : ((uint64_t)1 << end) - 1;
  return m0 < 0 ? w | (((uint64_t)1 << -m0) - 1) : w;
}

}  // namespace pkv
