// launch_tree.h — host-side parameter block and launchers of the attention of a
// tree of drafted tokens (not part of the public ABI).
#pragma once
#include <algorithm>
#include "launch.h"

namespace pkv {

constexpr int kTreeRows = 128;        // (node, head) rows of a tile, the M of its MMAs
constexpr int kTreeParts = 3;         // partial results of a CTA
constexpr int tree_keys(int head_dim) { return head_dim <= 128 ? 128 : 64; }   // of a tile

// What a sequence asks for.
struct TreeSeq {
  int q0, L, ctx;                     // first row, nodes, tokens with them
  int kt, rt;                         // key tiles, row tiles; 0 where there is nothing to do
};

// Where a CTA's range begins: a key tile of an item.
struct TreeStart {
  TreeSeq s;
  int n, h, r, t0;
  int64_t ahead;                      // key tiles of all items before it
};

// What a CTA leaves for the merge: where its range of key tiles begins inside an
// item (a row tile of one sequence and KV head), that item and the CTAs that share it.
struct TreeSplit {
  int first, last;                    // CTAs; last = 0: nothing to merge here
  int row;                            // first row of q and out
  int nodes;                          // nodes of the row tile
  int head;                           // KV head
  int seq, node0;                     // its sequence, and of that the tile's first node
  int pad;
};

// And where V of a tree in its range held what is no number: its range. The attention takes
// such elements for 0; the merge adds them to the outputs of the rows that see them.
struct TreeOdd {
  int tiles;                          // 0: nothing of the kind
  TreeStart begin;
};

struct TreeParams {
  void* out;
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* cu_q_lens;
  const uint32_t* masks;              // [q_rows, mask_words], or null: a chain
  const void* k_scales;               // fp32 [Hkv], or E8M0 [num_blocks, Hkv]
  const void* v_scales;
  const float* v_head_scales;         // fp32 [Hkv] with a scale per head, else null
  float* out_lse;
  unsigned int* err;
  // Of CTA c: partial results 3 c (of an item that an earlier CTA began) and 3 c + 1 (of
  // one that goes on in the next), each the rows' normalised O, [D / 4][128] float4, and
  // their log2 sums [128], of every copy of a row; 3 c + 2: where the copies of a whole
  // item are added up. Then the CTAs' TreeSplit and TreeOdd.
  float* part_o;
  float* part_lse;
  TreeSplit* splits;
  TreeOdd* odd;
  pkv_dtype kv_dtype;
  int num_seqs, Hq, Hkv, G, max_blocks, num_blocks, q_rows, mask_words;
  int q_tile;                         // nodes of a row tile
  int ppb_shift;                      // log2(block_size / 16)
  int ctas;                           // CTAs that share the work
  float qk_scale_log2;
};

// Workspace: ctas * (three partial results, a TreeSplit, a TreeOdd), and a TreeSplit that is empty;
// 0 without a device.
constexpr size_t tree_part_floats(int head_dim) { return (size_t)kTreeRows * head_dim; }
constexpr size_t tree_workspace_bytes(int ctas, int head_dim) {
  return ctas == 0 ? 0
                   : (size_t)ctas * (kTreeParts * (tree_part_floats(head_dim) + kTreeRows) *
                                         sizeof(float) +
                                     sizeof(TreeSplit) + sizeof(TreeOdd)) +
                         sizeof(TreeSplit);
}

// Validate nothing (the entry point does); PKV_ERR_CUDA on a launch failure. A call is two
// kernels: the attention, and the merge of the items that several CTAs share.
pkv_status launch_tree_16bit(const TreeParams& p, int head_dim, pkv_dtype q_dtype,
                             cudaStream_t stream);
pkv_status launch_tree_e4m3_head(const TreeParams& p, int head_dim, pkv_dtype q_dtype,
                                 cudaStream_t stream);
pkv_status launch_tree_e4m3_block(const TreeParams& p, int head_dim, pkv_dtype q_dtype,
                                  cudaStream_t stream);
pkv_status launch_tree_merge(const TreeParams& p, int head_dim, pkv_dtype q_dtype,
                             cudaStream_t stream);

}  // namespace pkv
