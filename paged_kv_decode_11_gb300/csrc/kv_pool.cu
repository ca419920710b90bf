// kv_pool.cu — kv_fork_blocks and kv_resize_blocks: block tables and reference counts on
// the device, so that a step that forks, grows or trims its sequences needs no host.
//
// The pool's state is a count per block, the table entries that name it; a block is unused
// at 0. New blocks are the lowest unused ones, in the order of the places that ask (row,
// then entry), which makes the result a function of the inputs alone. Both are one launch
// of one thread-block cluster: entries are shared and given back (atomic adds, whose order
// does not matter), a cluster barrier, then every CTA looks over its part of the counts, 16
// a thread in flight, and the CTAs' totals go through each other's shared memory. A place's
// rank finds its row by bisection of the rows' running sums, held in shared memory.
// What bounds it is latency: of a resize two or three dependent trips to L2 (lengths, counts, for
// rows that shrink entries) and two cluster barriers; of a fork six (lengths and parents, last
// entries, tables, tables again, counts, the copies' sources) and three. Blocks of 16: one row by
// 64 tokens 4.1 us, 256 rows by up to 600 tokens with 131,072 counts 12.7; a prompt of 900 into
// four rows 8.5, 256 rows of up to 8,192 tokens with 98,304 counts 19.9.
#include <cuda_runtime.h>
#include <atomic>
#include "launch_pages.h"
#include "ptx.cuh"

namespace pkv {

constexpr int kPoolCtas = 8;
constexpr int kPoolThreads = 1024;
constexpr int kPoolWarps = kPoolThreads / 32;
constexpr int kPoolEach = 16;                           // counts a thread looks at per round

__device__ __forceinline__ uint32_t pool_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Every thread of the cluster; what they wrote before it is visible after it.
__device__ __forceinline__ void pool_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" :::
                   "memory");
}
__device__ __forceinline__ void pool_store(const int* here, uint32_t rank, int v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(here)), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// Running sums of count(row) over the rows into sums[0 .. rows]; every thread of the CTA.
template <class F>
__device__ __forceinline__ void pool_sums(int* sums, int rows, F count) {
  __shared__ int s_warp[kPoolWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int each = (rows + kPoolThreads - 1) / kPoolThreads;
  const int r0 = min(tid * each, rows), r1 = min(r0 + each, rows);
  int mine = 0;
  for (int r = r0; r < r1; ++r) mine += count(r);
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) s_warp[warp] = upto;
  __syncthreads();
  int at = upto - mine;
  for (int w = 0; w < warp; ++w) at += s_warp[w];
  for (int r = r0; r < r1; ++r) {
    sums[r] = at;
    at += count(r);
  }
  if (r1 == rows && r0 < r1) sums[rows] = at;
  if (rows == 0 && tid == 0) sums[0] = 0;
  __syncthreads();
}

// The row that place `rank` (< sums[rows]) belongs to: sums[row] <= rank < sums[row + 1].
__device__ __forceinline__ int pool_row(const int* sums, int rows, int rank) {
  int lo = 0, hi = rows;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (sums[mid] <= rank) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Gives `wanted` places the lowest unused blocks: give(rank, id) for each, ranks in the
// order of the ids. Returns how many there were (at most a round's more than wanted). Each of a
// thread's counts lies in another stripe of ids, the cluster's threads side by side in it, so
// that the few lowest blocks, which are the ones that are given, fall to many warps. Counts that
// the cluster wrote before a barrier are read past L1.
template <class F>
__device__ __forceinline__ int pool_take(int32_t* refs, int num_blocks, int wanted, F give) {
  __shared__ int s_ahead[kPoolEach][kPoolWarps];          // unused of the stripe in lower warps
  __shared__ int s_all[2][kPoolEach][kPoolCtas], s_base[kPoolEach + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = (int)pool_rank();
  constexpr int kStripe = kPoolCtas * kPoolThreads, kRound = kStripe * kPoolEach;
  int found = 0;
  for (int first = 0, round = 0; first < num_blocks && found < wanted; ++round) {
    const int base = first + cta * kPoolThreads + tid;
    int v[kPoolEach];
#pragma unroll
    for (int k = 0; k < kPoolEach; ++k) {
      const int id = base + k * kStripe;
      v[k] = id < num_blocks ? __ldcg(refs + id) : 1;
    }
    uint32_t unused[kPoolEach];
#pragma unroll
    for (int k = 0; k < kPoolEach; ++k) {
      unused[k] = __ballot_sync(0xFFFFFFFFu, v[k] == 0);
      if (lane == 0) s_ahead[k][warp] = __popc(unused[k]);
    }
    __syncthreads();
    if (warp < kPoolEach) {                               // a warp to a stripe
      const int mine = s_ahead[warp][lane];
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += x;
      }
      s_ahead[warp][lane] = upto - mine;
      const int total = __shfl_sync(0xFFFFFFFFu, upto, 31);
      if (lane < kPoolCtas) pool_store(&s_all[round & 1][warp][cta], lane, total);
    }
    pool_barrier();
    if (warp == 0) {
      // of each stripe, the rank of this CTA's first
      int lower = 0, all = 0;
      if (lane < kPoolEach)
        for (int c = 0; c < kPoolCtas; ++c) {
          const int x = s_all[round & 1][lane][c];
          if (c < cta) lower += x;
          all += x;
        }
      int upto = all;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += x;
      }
      if (lane < kPoolEach) s_base[lane] = found + upto - all + lower;
      if (lane == 31) s_base[kPoolEach] = found + upto;
    }
    __syncthreads();
    found = s_base[kPoolEach];
#pragma unroll
    for (int k = 0; k < kPoolEach; ++k) {
      const int at = s_base[k] + s_ahead[k][warp] + __popc(unused[k] & ((1u << lane) - 1u));
      if (v[k] == 0 && at < wanted) {
        const int id = base + k * kStripe;
        refs[id] = 1;
        give(at, id);
      }
    }
    if (num_blocks - first <= kRound) break;
    first += kRound;
    __syncthreads();                                      // before s_ahead and s_base are used again
  }
  return found;
}

// One table entry less for a block: false where it names no block in use.
__device__ __forceinline__ void pool_give_back(int32_t* refs, int num_blocks, int id,
                                               unsigned int* err) {
  if (id < 0) return;                                   // none was to be had
  if (id >= num_blocks) {
    atomicOr(err, PKV_DEVERR_BLOCK_ID);
  } else if (atomicSub(refs + id, 1) <= 0) {
    atomicAdd(refs + id, 1);
    atomicOr(err, PKV_DEVERR_POOL);
  }
}

// Blocks of a length; 0 for one that the table's width does not hold (flagged once).
__device__ __forceinline__ int pool_blocks(int len, int bs_log2, int width, unsigned int* err) {
  if (len < 0 || len > ((int64_t)width << bs_log2)) {
    if (err != nullptr) atomicOr(err, PKV_DEVERR_SEQ_LEN);
    return -1;
  }
  return (int)(((int64_t)len + (1 << bs_log2) - 1) >> bs_log2);
}

__global__ void __cluster_dims__(kPoolCtas, 1, 1) __launch_bounds__(kPoolThreads, 1)
    resize_kernel(const ResizeParams p) {
  extern __shared__ int s_sums[];                       // [rows + 1] places that ask
  int* s_place = s_sums + p.rows + 1;                   // [rows] table place of rank 0, were it the row's
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int warp = (int)pool_rank() * kPoolWarps + (threadIdx.x >> 5);
  // A row with a bad length is left as it is.
  auto blocks = [&](int r, int& have, int& want, unsigned int* err) {
    have = pool_blocks(p.lens[r], p.bs_log2, p.width, err);
    want = pool_blocks(p.new_lens[r], p.bs_log2, p.width, err);
    if (have < 0 || want < 0) have = want = 0;
  };
  pool_sums(s_sums, p.rows, [&](int r) {
    int have, want;
    blocks(r, have, want, nullptr);
    s_place[r] = r * p.width + have;
    return max(0, want - have);
  });
  const int wanted = s_sums[p.rows];
  for (int r = threadIdx.x; r < p.rows; r += kPoolThreads) s_place[r] -= s_sums[r];
  for (int r = warp; r < p.rows; r += kPoolCtas * kPoolWarps) {
    int have, want;
    blocks(r, have, want, p.err);
    int32_t* row = p.tables + (int64_t)r * p.width;
    for (int j = want + lane; j < have; j += 32) {
      pool_give_back(p.refs, p.num_blocks, row[j], p.err);
      row[j] = -1;
    }
  }
  if (wanted == 0) return;                              // (the same in every CTA)
  pool_barrier();
  auto give = [&](int at, int id) { p.tables[s_place[pool_row(s_sums, p.rows, at)] + at] = id; };
  const int found = pool_take(p.refs, p.num_blocks, wanted, give);
  if (found < wanted) {                                 // the places past the last block
    if (warp == 0 && lane == 0) atomicOr(p.err, PKV_DEVERR_POOL);
    const int t = (int)pool_rank() * kPoolThreads + threadIdx.x;
    for (int at = found + t; at < wanted; at += kPoolCtas * kPoolThreads) give(at, -1);
  }
}

constexpr int kAsks = 1 << 30;                          // (in a row's parent) it gets a block of its own
constexpr int kLacks = 1 << 30;                         // (in a row's length) its last, partly filled
                                                        // block is none of the pool's
constexpr int kForkBatch = 8;                           // a lane's entries whose loads are under way

__global__ void __cluster_dims__(kPoolCtas, 1, 1) __launch_bounds__(kPoolThreads, 1)
    fork_kernel(const ForkParams p) {
  extern __shared__ int s_rows[];
  int* s_sums = s_rows;                                 // [rows + 1] rows that ask for a block; before
  int* s_first = s_rows;                                // that a row's first descendant
  int* s_parent = s_rows + p.rows + 1;                  // [rows], -1: none
  int* s_len = s_parent + p.rows;                       // [rows] of the old table, kLacks with it
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int warp = (int)pool_rank() * kPoolWarps + (threadIdx.x >> 5);
  unsigned int* err = warp < kPoolWarps ? p.err : nullptr;   // (one CTA reports)
  const int part = (1 << p.bs_log2) - 1;
  for (int r = threadIdx.x; r < p.rows; r += kPoolThreads) {
    const int q = p.parents[r], len = p.lens[r];
    if (q >= p.rows && err != nullptr) atomicOr(err, PKV_DEVERR_PATH);
    s_parent[r] = q < p.rows ? max(q, -1) : -1;
    // a length that the width does not hold counts as 0
    const bool bad = pool_blocks(len, p.bs_log2, p.width, err) < 0;
    // a last block that is not there (the pool had run out) cannot be copied: its row's
    // descendants lack it too
    bool lacks = false;
    if (!bad && (len & part) != 0) {
      const int last = p.tables[(int64_t)r * p.width + (len >> p.bs_log2)];
      lacks = last < 0 || last >= p.num_blocks;
      if (last >= p.num_blocks && err != nullptr) atomicOr(err, PKV_DEVERR_BLOCK_ID);
    }
    s_len[r] = bad ? 0 : lacks ? len | kLacks : len;
    s_first[r] = p.rows;
  }
  __syncthreads();
  for (int r = threadIdx.x; r < p.rows; r += kPoolThreads)
    if (s_parent[r] >= 0) atomicMin(s_first + s_parent[r], r);
  __syncthreads();
  for (int r = threadIdx.x; r < p.rows; r += kPoolThreads) {
    const int q = s_parent[r];
    if (q >= 0 && (s_len[q] & part) != 0 && s_first[q] != r) s_parent[r] = q | kAsks;
  }
  __syncthreads();
  auto asks = [&](int r) { return s_parent[r] >= kAsks; };
  pool_sums(s_sums, p.rows, [&](int r) {
    return asks(r) && (s_len[s_parent[r] & ~kAsks] & kLacks) == 0 ? 1 : 0;
  });
  for (int r = warp; r < p.rows; r += kPoolCtas * kPoolWarps) {
    const int q = s_parent[r] < 0 ? -1 : s_parent[r] & ~kAsks;
    const int len = q >= 0 ? s_len[q] & ~kLacks : 0;
    const int mine = asks(r) ? len >> p.bs_log2 : (len + part) >> p.bs_log2;   // shared entries
    const int held = ((s_len[r] & ~kLacks) + part) >> p.bs_log2;
    const int32_t* old = p.tables + (int64_t)r * p.width;
    const int32_t* from = p.tables + (int64_t)max(q, 0) * p.width;
    int32_t* to = p.new_tables + (int64_t)r * p.width;
    for (int j0 = lane; j0 < p.width; j0 += 32 * kForkBatch) {
      int next[kForkBatch], was[kForkBatch];
#pragma unroll
      for (int k = 0; k < kForkBatch; ++k) {
        const int j = j0 + 32 * k;
        next[k] = j < mine ? from[j] : -1;
        was[k] = j < held ? old[j] : -1;
      }
#pragma unroll
      for (int k = 0; k < kForkBatch; ++k) {
        if (j0 + 32 * k >= p.width) continue;
        to[j0 + 32 * k] = next[k];
        if (next[k] >= p.num_blocks) atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
        // (an entry that stays the same block's: one more and one less)
        else if (next[k] >= 0 && next[k] != was[k]) atomicAdd(p.refs + next[k], 1);
      }
    }
    if (lane == 0) {
      p.new_lens[r] = len;
      *reinterpret_cast<int2*>(p.copies + 2 * r) = make_int2(-1, -1);
    }
  }
  pool_barrier();
  // given back only when every descendant has taken its share, so that no count in use
  // passes through 0
  for (int r = warp; r < p.rows; r += kPoolCtas * kPoolWarps) {
    const int held = ((s_len[r] & ~kLacks) + part) >> p.bs_log2;
    const int32_t* old = p.tables + (int64_t)r * p.width;
    const int32_t* to = p.new_tables + (int64_t)r * p.width;
    for (int j0 = lane; j0 < held; j0 += 32 * kForkBatch) {
      int was[kForkBatch], next[kForkBatch];
#pragma unroll
      for (int k = 0; k < kForkBatch; ++k) {
        const int j = j0 + 32 * k;
        was[k] = j < held ? old[j] : -1;
        next[k] = j < held ? to[j] : -1;
      }
#pragma unroll
      for (int k = 0; k < kForkBatch; ++k)
        if (was[k] != next[k]) pool_give_back(p.refs, p.num_blocks, was[k], p.err);
    }
  }
  const int wanted = s_sums[p.rows];
  if (wanted == 0) return;                              // (the same in every CTA)
  pool_barrier();
  auto give = [&](int at, int id) {
    const int r = pool_row(s_sums, p.rows, at), q = s_parent[r] & ~kAsks;
    const int j = s_len[q] >> p.bs_log2;
    p.new_tables[(int64_t)r * p.width + j] = id;
    *reinterpret_cast<int2*>(p.copies + 2 * r) = make_int2(p.tables[(int64_t)q * p.width + j], id);
  };
  const int found = pool_take(p.refs, p.num_blocks, wanted, give);
  if (found < wanted && warp == 0 && lane == 0) atomicOr(p.err, PKV_DEVERR_POOL);
}

template <class Params>
static pkv_status launch_pool(void (*kern)(Params), std::atomic<bool>* prepared, const Params& p,
                              size_t smem, cudaStream_t stream) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PKV_ERR_CUDA;
  if (!prepared[dev]) {                                 // per device; the call is idempotent
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (3 * kMaxPoolRows + 1) * 4) != cudaSuccess)
      return PKV_ERR_CUDA;
    prepared[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(kPoolCtas);
  cfg.blockDim = dim3(kPoolThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

pkv_status launch_fork(const ForkParams& p, cudaStream_t stream) {
  static std::atomic<bool> prepared[64];
  return launch_pool(fork_kernel, prepared, p, (3 * (size_t)p.rows + 1) * 4, stream);
}

pkv_status launch_resize(const ResizeParams& p, cudaStream_t stream) {
  static std::atomic<bool> prepared[64];
  return launch_pool(resize_kernel, prepared, p, (2 * (size_t)p.rows + 1) * 4, stream);
}

}  // namespace pkv
