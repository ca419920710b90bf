// kv_move.cu — kv_copy_blocks and kv_keep_path: cached tokens and blocks move within the
// caches of every layer, in one launch for up to 128 caches.
//
// Both only move bytes (a block-scaled path apart, whose codes may take another exponent),
// so that what bounds them is the memory's rate, and for a step's few tokens the latency of
// a launch and of the look-ups in front of the first load: lengths, path and table. 96 blocks of
// 32 KB in 64 caches take 61 us (6.6 TB/s, read and written), one block 4.0, a path of 13 in 64
// caches 4.5; 64 paths of up to 60 in 32 block-scaled caches 18.0.
#include <cuda_runtime.h>
#include <algorithm>
#include <climits>
#include "block_scale.cuh"
#include "launch_pages.h"

namespace pkv {

constexpr int kMoveThreads = 256;

template <class Params>
static pkv_status launch_dependent(void (*kern)(Params), const Params& p, dim3 grid, int threads,
                                   cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

// CTA (pair and piece, cache): a piece is U * 4 KB of a block, every load of a thread ahead
// of its stores.
template <int U>
__global__ void __launch_bounds__(kMoveThreads)
    copy_blocks_kernel(const __grid_constant__ CopyBlocksParams p) {
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();
  const int pair = blockIdx.x / p.pieces, piece = blockIdx.x % p.pieces, c = blockIdx.y;
  const int src = p.pairs[2 * pair], dst = p.pairs[2 * pair + 1];
  if (src < 0 || dst < 0 || src == dst) return;
  if (src >= p.num_blocks || dst >= p.num_blocks) {
    if (threadIdx.x == 0 && piece == 0 && c == 0) atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
    return;
  }
  const int64_t bytes = p.bytes[c];
  const uint8_t* from = p.cache[c] + src * bytes;
  uint8_t* to = p.cache[c] + dst * bytes;
  if (bytes % 16 == 0) {
    const int64_t words = bytes / 16;
    const int64_t w0 = (int64_t)piece * U * kMoveThreads + threadIdx.x;
    uint4 v[U];
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (w0 + k * kMoveThreads < words)
        v[k] = reinterpret_cast<const uint4*>(from)[w0 + k * kMoveThreads];
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (w0 + k * kMoveThreads < words) reinterpret_cast<uint4*>(to)[w0 + k * kMoveThreads] = v[k];
  } else {                                              // a few scales
    for (int64_t i = (int64_t)piece * kMoveThreads + threadIdx.x; i < bytes;
         i += (int64_t)p.pieces * kMoveThreads)
      to[i] = from[i];
  }
}

pkv_status launch_copy_blocks(CopyBlocksParams& p, int sms, cudaStream_t stream) {
  int64_t most = 1, all = 0;
  for (int c = 0; c < p.num_caches; ++c) {
    most = std::max(most, p.bytes[c]);
    all += p.bytes[c];
  }
  // pieces of 16 KB keep enough bytes on their way for the memory's rate; where they would
  // be fewer than four to an SM, 4 KB
  const bool small = all * p.num_pairs < (int64_t)sms * 4 * 16384;
  const int piece = kMoveThreads * 16 * (small ? 1 : 4);
  p.pieces = (int)((most + piece - 1) / piece);
  const int64_t ctas = (int64_t)p.pieces * p.num_pairs;
  if (ctas > 0x7FFFFFFF) return PKV_ERR_INVALID_ARG;
  const dim3 grid((unsigned)ctas, p.num_caches);
  return launch_dependent(small ? copy_blocks_kernel<1> : copy_blocks_kernel<4>, p, grid,
                          kMoveThreads, stream);
}

// Sequence n's tree and path, as the CTA's threads agree on it. False: nothing to do.
struct Path {
  int start, L, len, moved;           // tokens before the tree, nodes, kept, first that moves
};
__device__ __forceinline__ bool read_path(const KeepPathParams& p, int n, bool reports, Path& t) {
  const int q0 = p.cu_q_lens[n], ctx = p.seq_lens[n];
  t.L = p.cu_q_lens[n + 1] - q0;
  t.len = p.path_lens[n];
  t.start = ctx - t.L;
  const int32_t* path = p.paths + (int64_t)n * p.max_path;
  bool ok = t.L >= 0 && t.L <= ctx && t.len >= 0 && t.len <= t.L && t.len <= p.max_path &&
            ctx <= (int64_t)p.max_blocks << p.bs_log2;
  int same = 0;                       // path[i] == i: as the path rises, a run at its start
  if (ok)
    for (int i = threadIdx.x; i < t.len; i += blockDim.x) {
      const int a = path[i], before = i > 0 ? path[i - 1] : -1;
      ok = ok && a > before && a < t.L;
      same += a == i;
    }
  __shared__ int s_same;
  if (threadIdx.x == 0) s_same = 0;
  ok = __syncthreads_and(ok);
  if (same > 0) atomicAdd(&s_same, same);
  __syncthreads();
  t.moved = s_same;
  if (reports && threadIdx.x == 0) {
    if (!ok) atomicOr(p.err, PKV_DEVERR_PATH);
    if (p.new_seq_lens != nullptr) p.new_seq_lens[n] = ok ? t.start + t.len : ctx;
  }
  return ok;
}

// Caches that hold each value by itself: rows move as they are. CTA (256 16-byte columns of
// the (cache, KV head) rows, sequence). A thread owns a column and moves its path in order;
// as the path rises, path[i] >= i, no later source is an earlier destination, so that it may
// read eight of them ahead of its stores.
__global__ void __launch_bounds__(kMoveThreads)
    keep_path_kernel(const __grid_constant__ KeepPathParams p) {
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();
  __shared__ int s_from[kMoveThreads], s_to[kMoveThreads];     // rows of a cache, head 0; -1: none
  const int n = blockIdx.y;
  Path t;
  if (!read_path(p, n, blockIdx.x == 0, t)) return;
  const int cpr = p.row_bytes / 16;
  const int64_t i = (int64_t)blockIdx.x * kMoveThreads + threadIdx.x;
  const int unit = (int)(i / cpr), ch = (int)(i % cpr);
  const int c = unit / p.Hkv, h = unit % p.Hkv;
  const bool active = c < p.num_caches;
  uint8_t* cache = p.cache[active ? c : 0] + (((int64_t)h << p.bs_log2) * p.row_bytes) + 16 * ch;
  const int32_t* path = p.paths + (int64_t)n * p.max_path;
  const int32_t* table = p.block_tables + (int64_t)n * p.max_blocks;
  auto row_of = [&](int pos) {
    const int id = table[pos >> p.bs_log2];
    if (id < 0 || id >= p.num_blocks) {
      if (blockIdx.x == 0) atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
      return -1;
    }
    return (int)(((int64_t)id * p.Hkv << p.bs_log2) + (pos & ((1 << p.bs_log2) - 1)));
  };
  for (int k0 = t.moved; k0 < t.len; k0 += kMoveThreads) {
    const int cnt = min(kMoveThreads, t.len - k0);
    __syncthreads();
    if ((int)threadIdx.x < cnt) {
      const int k = k0 + threadIdx.x;
      const int from = row_of(t.start + path[k]), to = row_of(t.start + k);
      s_from[threadIdx.x] = to < 0 ? -1 : from;
      s_to[threadIdx.x] = to;
    }
    __syncthreads();
    if (!active) continue;
    for (int b = 0; b < cnt; b += 8) {
      uint4 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (b + k < cnt && s_from[b + k] >= 0)
          v[k] = *reinterpret_cast<const uint4*>(cache + (int64_t)s_from[b + k] * p.row_bytes);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (b + k < cnt && s_from[b + k] >= 0)
          *reinterpret_cast<uint4*>(cache + (int64_t)s_to[b + k] * p.row_bytes) = v[k];
    }
  }
}

// Sixteen codes times 2^d, to the nearest E4M3.
__device__ __forceinline__ uint4 rescale16(uint4 w, int d) {
  const float f = pow2_any(max(min(d, 127), -126));
  uint32_t in[4] = {w.x, w.y, w.z, w.w}, out[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t two[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint32_t h = e4m3x2_to_f16x2((in[k] >> (16 * s)) & 0xFFFFu);
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
      two[s] = f32x2_to_e4m3x2(v.x * f, v.y * f);
    }
    out[k] = two[0] | (two[1] << 16);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// Block scales. A warp has a (cache, KV head) pair of one sequence; the path's places are looked up
// once for a CTA's eight. (64 paths in 32 caches of 8 heads: 18.0 us. When one pair a warp took
// 17.5, two took 19.7, three 23.4, and eight chunks to a lane, 80 registers and so three CTAs an
// SM instead of five, 21.5.) A warp goes from destination block to destination block (none of the
// path's later sources lies in an earlier one): it reads the path's rows there, reduces their
// exponents, and writes them with the block's new one.
// A block's rows of more than 128 16-byte chunks are read twice, for the exponent and to be
// written, the rows in order, so that none is overwritten before it is read.
constexpr int kKeepWarps = 8, kKeepChunks = 4;          // chunks of a lane at a time
constexpr int kKeepPath = 256;                          // places looked up at a time

// What exponent sixteen codes with scale byte s need: kBlockMinExp where all are 0 or NaN.
__device__ __forceinline__ int chunk_exponent(uint4 v, int s) {
  if (s == 255) return kBlockMinExp;
  uint32_t top = 0u;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const uint32_t m = w[a] & 0x7F7F7F7Fu;              // magnitudes; 0x7F is NaN
    top = __vmaxu4(top, m & ~__vcmpeq4(m, 0x7F7F7F7Fu));
  }
  top = max(max(top & 0xFFu, (top >> 8) & 0xFFu), max((top >> 16) & 0xFFu, top >> 24));
  if (top == 0u) return kBlockMinExp;
  const uint32_t f16 = e4m3x2_to_f16x2(top);
  const uint32_t b = __float_as_uint(__half2float(__ushort_as_half((unsigned short)f16)));
  // amax = m 2^k: 448 2^e holds it from e = k - 8 on, k - 7 where m > 1.75
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e + s - kE8M0Bias;
}

__global__ void __launch_bounds__(32 * kKeepWarps, 5)
    keep_path_block_kernel(const __grid_constant__ KeepPathParams p) {
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();
  // of each place: its source's block (-1: none) and slot, and its destination's block
  __shared__ int s_src[kKeepPath], s_slot[kKeepPath], s_dst[kKeepPath];
  const int n = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Path t;
  if (!read_path(p, n, blockIdx.x == 0, t)) return;
  const int bs = 1 << p.bs_log2, cpr = p.row_bytes / 16;
  const int64_t block_bytes = ((int64_t)p.row_bytes * p.Hkv) << p.bs_log2;
  const int32_t* path = p.paths + (int64_t)n * p.max_path;
  const int32_t* table = p.block_tables + (int64_t)n * p.max_blocks;
  auto block_of = [&](int pos) {
    const int id = table[pos >> p.bs_log2];
    if (id >= 0 && id < p.num_blocks) return id;
    if (blockIdx.x == 0) atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
    return -1;
  };
  const int unit = blockIdx.x * kKeepWarps + warp, h = unit % p.Hkv;
  const bool active = unit < p.num_caches * p.Hkv;
  const int c = active ? unit / p.Hkv : 0;
  uint8_t* cache = p.cache[c] + (((int64_t)h * p.row_bytes) << p.bs_log2);
  uint8_t* scales = p.scales[c] + h;
  for (int k0 = 0; k0 < t.len;) {
    // places up to a destination block's end
    int k1 = min(t.len, k0 + kKeepPath);
    if (k1 < t.len) k1 -= (t.start + k1) & (bs - 1);
    __syncthreads();
    for (int i = k0 + threadIdx.x; i < k1; i += blockDim.x) {
      const int pos = t.start + path[i];
      s_src[i - k0] = block_of(pos);
      s_slot[i - k0] = pos & (bs - 1);
      s_dst[i - k0] = block_of(t.start + i);
    }
    __syncthreads();
    for (int i0 = active ? k0 : k1; i0 < k1;) {
      const int off = (t.start + i0) & (bs - 1);      // the first slot that is written
      const int cnt = min(bs - off, k1 - i0), chunks = cnt * cpr, first = i0;
      i0 += cnt;
      const int dst = s_dst[first - k0];
      if (dst < 0 || (off > 0 && i0 <= t.moved)) continue;   // (nothing moves, nothing changes)
      uint8_t* to = cache + dst * block_bytes;
      const int old = scales[(int64_t)dst * p.Hkv];
      uint4 v[kKeepChunks];
      int s[kKeepChunks];                             // its scale; -1: no such chunk or source
      auto read = [&](int q0) {
#pragma unroll
        for (int k = 0; k < kKeepChunks; ++k) {
          const int q = q0 + lane + 32 * k, i = first - k0 + q / cpr;
          s[k] = -1;
          if (q >= chunks || s_src[i] < 0) continue;
          s[k] = scales[(int64_t)s_src[i] * p.Hkv];
          v[k] = *reinterpret_cast<const uint4*>(cache + s_src[i] * block_bytes +
                                                 (int64_t)s_slot[i] * p.row_bytes + 16 * (q % cpr));
        }
      };
      int need = INT_MIN;
      for (int q0 = 0; q0 < chunks; q0 += 32 * kKeepChunks) {
        read(q0);
#pragma unroll
        for (int k = 0; k < kKeepChunks; ++k)
          if (s[k] >= 0) need = max(need, chunk_exponent(v[k], s[k]));
      }
      need = __reduce_max_sync(0xFFFFFFFFu, need);    // (every row, and scale, has been read)
      if (need == INT_MIN) continue;                  // every source's block is outside the pool
      need = max(need, kBlockMinExp);
      const int was = min(old, 254) - kE8M0Bias, now = off == 0 ? need : max(was, need);
      for (int q0 = 0; q0 < chunks; q0 += 32 * kKeepChunks) {
        if (chunks > 32 * kKeepChunks) {
          read(q0);
          __syncwarp();
        }
#pragma unroll
        for (int k = 0; k < kKeepChunks; ++k) {
          if (s[k] < 0) continue;
          const int q = q0 + lane + 32 * k, row = off + q / cpr;
          uint4 x = v[k];
          if (s[k] == 255) x = make_uint4(x.x | 0x7F7F7F7Fu, x.y | 0x7F7F7F7Fu, x.z | 0x7F7F7F7Fu,
                                          x.w | 0x7F7F7F7Fu);
          else if (s[k] - kE8M0Bias != now) x = rescale16(x, s[k] - kE8M0Bias - now);
          *reinterpret_cast<uint4*>(to + (int64_t)row * p.row_bytes + 16 * (q % cpr)) = x;
        }
        __syncwarp();
      }
      if (off > 0 && now != was) {
        // the slots that nothing reached, to the exponent that has grown
        for (int q = lane; q < bs * cpr; q += 32) {
          const int row = q / cpr, k = row - off;
          if (k >= 0 && k < cnt && s_src[first - k0 + k] >= 0) continue;
          uint4* at = reinterpret_cast<uint4*>(to + (int64_t)row * p.row_bytes + 16 * (q % cpr));
          *at = rescale16(*at, was - now);
        }
      }
      if (lane == 0) scales[(int64_t)dst * p.Hkv] = (uint8_t)(now + kE8M0Bias);
      __syncwarp();
    }
    k0 = k1;
  }
}

pkv_status launch_keep_path(const KeepPathParams& p, bool block_scaled, cudaStream_t stream) {
  // (no caches: one CTA a sequence, for the new lengths)
  if (block_scaled) {
    const int ctas = std::max(1, (p.num_caches * p.Hkv + kKeepWarps - 1) / kKeepWarps);
    return launch_dependent(keep_path_block_kernel, p, dim3(ctas, p.num_seqs), 32 * kKeepWarps, stream);
  }
  const int64_t columns = std::max<int64_t>(1, (int64_t)p.num_caches * p.Hkv * (p.row_bytes / 16));
  const dim3 grid((unsigned)((columns + kMoveThreads - 1) / kMoveThreads), p.num_seqs);
  return launch_dependent(keep_path_kernel, p, grid, kMoveThreads, stream);
}

}  // namespace pkv
