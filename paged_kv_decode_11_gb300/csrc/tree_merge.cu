// tree_merge.cu — the merge of the items whose keys several CTAs of the tree attention
// (tree_kernel.cuh) share.
//
// Of an item's CTAs each left, per row and copy of it, O_i (normalised) and the log2 sum l_i
// of its keys: out = sum_i O_i 2^(l_i - l), l = log2 sum_i 2^l_i. An item cut at k places has k
// columns of this kernel's blocks, one for each place, and their warps take its (32 rows, 4
// columns) units in turn, so that a cut costs the same wherever it falls; a lane is a row, and
// every load of a warp is 512 consecutive bytes. What bounds it is the latency of its loads:
// BATCH parts' are under way together. Eight, with three CTAs an SM (32 sequences on 4 KV heads
// of 1,280 tokens, with the attention, 51 us, where 16 take 56; 128 on 8 heads of 1,024 121 and
// 124); 16 where there are so few sequences and heads that an item is cut into four parts and more
// (one of 900 tokens on 8 heads 12.4 us, where 8 take 12.8; of 8,000 22.2 and 23.1. The rule
// counts no row tiles: the host knows no tree's size).
//   Elements of V in a tree that are no numbers, which the attention took for 0, are added here to
// the outputs of the rows that see their keys, for every item: a weight of 0 in the attention's
// product would not keep them from the other rows. (There it cost the E4M3 kernels 2 to 4%, in
// code that is hardly ever run; here nothing, but for two loads that nothing waits for. With such
// an element 128 trees of 16 on 1,024 tokens take 142 to 167 us where they take 121.)
#include <cuda_runtime.h>
#include "kv_store.cuh"
#include "tree_work.cuh"

namespace pkv {

constexpr int kMergeWarps = 8, kMergeBlocks = 4;        // warps of a block, blocks of a cut

// The nodes of an item whose V holds what is no number, which the attention took for 0: to the
// outputs of the rows that see them, after they are written. The warp takes units `unit`, `unit` +
// step, .. of (32 rows, 4 columns), a lane to a row, and looks at 32 nodes at a time. Rare.
template <int D, bool QBF16>
__device__ __noinline__ void tree_add_odd(const TreeParams& p, int n, int head, int node0,
                                          int nodes, int unit, int step) {
  const int lane = threadIdx.x & 31, q0 = p.cu_q_lens[n], ctx = p.seq_lens[n];
  const int L = p.cu_q_lens[n + 1] - q0, rows = nodes * p.G, row_blocks = (rows + 31) / 32;
  for (int u = unit; u < row_blocks * (D / 4); u += step) {
    const int c = u / row_blocks * 4, row = 32 * (u % row_blocks) + lane;
    const bool mine = row < rows;
    const int node = node0 + min(row, rows - 1) / p.G;
    float add[4] = {};
    for (int m0 = 0; m0 < L; m0 += 32) {
      float x[4] = {};                                  // of the lane's node, what is no number
      if (m0 + lane < L) {
        const int pos = ctx - L + m0 + lane, page = pos / kBS;
        int id = p.block_tables[(int64_t)n * p.max_blocks + (page >> p.ppb_shift)];
        if (id < 0 || id >= p.num_blocks) id = 0;       // (as the page loads read it)
        const int z = ((id * p.Hkv + head) << p.ppb_shift) + (page & ((1 << p.ppb_shift) - 1));
        const int64_t at = ((int64_t)z * kBS + pos % kBS) * D + c;
        for (int k = 0; k < 4; ++k) {
          if (p.kv_dtype == PKV_F16 || p.kv_dtype == PKV_BF16) {
            const uint16_t v = static_cast<const uint16_t*>(p.v_cache)[at + k];
            x[k] = p.kv_dtype == PKV_BF16 ? widen16<true>(v) : widen16<false>(v);
          } else if ((static_cast<const uint8_t*>(p.v_cache)[at + k] & 0x7Fu) == 0x7Fu) {
            x[k] = __int_as_float(0x7FFFFFFF);
          }
          if (fabsf(x[k]) < INFINITY) x[k] = 0.f;
        }
      }
      const bool some = x[0] != 0.f || x[1] != 0.f || x[2] != 0.f || x[3] != 0.f;
      const uint32_t sees = (uint32_t)tree_sees(p, q0 + node, node, m0, L);
      for (uint32_t odd = __ballot_sync(0xFFFFFFFFu, some); odd != 0u; odd &= odd - 1) {
        const int m = __ffs(odd) - 1;
        for (int k = 0; k < 4; ++k) {
          const float v = __shfl_sync(0xFFFFFFFFu, x[k], m);
          if ((sees >> m) & 1u) add[k] += v;
        }
      }
    }
    if (!mine) continue;
    uint16_t* to = static_cast<uint16_t*>(p.out) +
                   ((int64_t)(q0 + node) * p.Hq + head * p.G + row % p.G) * D + c;
    for (int k = 0; k < 4; ++k)
      if (add[k] != 0.f) to[k] = (uint16_t)pack2<QBF16>(widen16<QBF16>(to[k]) + add[k], 0.f);
  }
}

// The same of the items that a CTA of the attention had by itself.
template <int D, bool QBF16>
__device__ __noinline__ void tree_add_odd_own(const TreeParams& p, int cta, int tiles, int warp) {
  for (TreeWork<tree_keys(D), true> w(p, p.odd[cta].begin, tiles); w.cnt > 0; w.next())
    if (w.cnt == w.s.kt)
      tree_add_odd<D, QBF16>(p, w.n, w.h, w.node0(), w.nodes(), warp, kMergeWarps * kMergeBlocks);
}

template <int D, bool QBF16, int BATCH>
__global__ void __launch_bounds__(32 * kMergeWarps, BATCH == 8 ? 3 : 2) tree_merge_kernel(
    const __grid_constant__ TreeParams p) {
  // what comes next on the stream may become resident; it waits for this grid
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();                                       // the attention is done
  const int cta = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
  const int own = p.odd[cta].tiles;
  const TreeSplit d = p.splits[cta + 1];                // (behind the last: an empty one)
  if (d.last == 0) {
    if (own != 0) tree_add_odd_own<D, QBF16>(p, cta, own, warp);
    return;
  }
  const int cuts = d.last - d.first, rows = d.nodes * p.G;
  const int row_blocks = (rows + 31) / 32, units = row_blocks * (D / 4);
  // every CTA's copies of a row (tree_kernel.cuh): RP rows apart
  const int reps_log2 = rows <= 32 ? 2 : rows <= 64 ? 1 : 0, RP = kTreeRows >> reps_log2;
  const int parts = (cuts + 1) << reps_log2;
  const float vs = p.v_head_scales != nullptr ? p.v_head_scales[d.head] : 1.f;
  // (used behind the units, so that nothing waits for it before)
  int odd = d.first + lane <= d.last ? p.odd[d.first + lane].tiles : 0;
  for (int u = cta - d.first + cuts * warp; u < units;
       u += cuts * kMergeWarps * kMergeBlocks) {
    const int cg = u / row_blocks, row = 32 * (u % row_blocks) + lane;
    if (row >= rows) continue;
    const float* lp = p.part_lse + row;
    const float4* op = reinterpret_cast<const float4*>(p.part_o) + cg * kTreeRows + row;
    float top = -INFINITY, sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < parts; i0 += BATCH) {
      float l[BATCH];
      float4 x[BATCH];
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        l[k] = -INFINITY;
        const int i = i0 + k, c = i >> reps_log2;
        if (i >= parts) continue;
        // (the first CTA's part is the one that goes on, the others' the one that went before)
        const int64_t slot = kTreeParts * (d.first + c) + (c == 0 ? 1 : 0);
        const int copy = (i & ((1 << reps_log2) - 1)) * RP;
        l[k] = lp[slot * kTreeRows + copy];
        x[k] = op[slot * (int64_t)(tree_part_floats(D) / 4) + copy];
      }
      float now = top;
#pragma unroll
      for (int k = 0; k < BATCH; ++k) now = fmaxf(now, l[k]);
      if (top != -INFINITY) {                           // (else the sums are 0, or NaN)
        const float w = exp2f(top - now);
        sum *= w;
        o = make_float4(o.x * w, o.y * w, o.z * w, o.w * w);
      }
      top = now;
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        if (l[k] == -INFINITY) continue;                // no key seen there
        const float w = exp2f(l[k] - top);              // (NaN where l is)
        sum += w;
        o = make_float4(fmaf(x[k].x, w, o.x), fmaf(x[k].y, w, o.y), fmaf(x[k].z, w, o.z),
                        fmaf(x[k].w, w, o.w));
      }
    }
    const bool some = !(sum == 0.f);
    const float f = some ? vs / sum : 0.f;
    const int node = row / p.G, head = d.head * p.G + row % p.G;
    const int64_t at = (int64_t)(d.row + node) * p.Hq + head;
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at * D + 4 * cg) =
        make_uint2(pack2<QBF16>(o.x * f, o.y * f), pack2<QBF16>(o.z * f, o.w * f));
    if (cg == 0 && p.out_lse != nullptr)
      p.out_lse[at] = some ? (top + log2f(sum)) * kLn2 : -INFINITY;
  }
  for (int c = d.first + lane + 32; c <= d.last; c += 32) odd |= p.odd[c].tiles;
  __syncwarp();
  if (__any_sync(0xFFFFFFFFu, odd != 0))
    tree_add_odd<D, QBF16>(p, d.seq, d.head, d.node0, d.nodes, cta - d.first + cuts * warp,
                           cuts * kMergeWarps * kMergeBlocks);
  if (own != 0) tree_add_odd_own<D, QBF16>(p, cta, own, warp);
}

template <int D, bool QBF16, int BATCH>
static pkv_status launch(const TreeParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(p.ctas, kMergeBlocks);
  cfg.blockDim = dim3(32 * kMergeWarps);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_merge_kernel<D, QBF16, BATCH>, p) == cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

template <int D, bool QBF16>
static pkv_status launch(const TreeParams& p, cudaStream_t stream) {
  return (int64_t)p.num_seqs * p.Hkv * 4 <= p.ctas ? launch<D, QBF16, 16>(p, stream)
                                                   : launch<D, QBF16, 8>(p, stream);
}

pkv_status launch_tree_merge(const TreeParams& p, int head_dim, pkv_dtype q_dtype,
                             cudaStream_t stream) {
  const bool bf = q_dtype == PKV_BF16;
  if (head_dim == 256) return bf ? launch<256, true>(p, stream) : launch<256, false>(p, stream);
  if (head_dim == 128) return bf ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
  return bf ? launch<64, true>(p, stream) : launch<64, false>(p, stream);
}

}  // namespace pkv
