// append_block.cu — rope_append_block_scaled: new tokens' keys (rotated) and
// values into E4M3 blocks with one power-of-two scale per block and KV head,
// and the rotation of their queries, in one launch.
//
// Mathematics. For each block and head that the call writes, K and V apart:
//   amax = largest finite |x| of the elements written there by this call,
//   e    = smallest whole number >= -60 with amax <= 448 * 2^e,
//   a block written from offset 0 starts anew with e; another keeps its stored
//   exponent s if s >= e, else takes e and its other slots are re-encoded:
//   code <- E4M3(code * 2^(s - e)). New codes are E4M3(x * 2^-e').
//
// Work decomposition. Tokens of a sequence that fall into one block are
// consecutive rows (a run of at most BS), so a run, not a token, is the unit:
// its first row (the leader) starts a sequence's chunk or a block. A CTA takes
// `window` consecutive rows and one KV head and does the runs whose leaders
// lie among its rows; its first 64 threads do the keys, the other 64 the
// values. A group goes over the run twice, 16 elements per thread and step: for
// amax, then (the rows now in L1) to encode; the rotation is cheaper to repeat
// than to keep. No two CTAs touch one block and head, so nothing is atomic and
// the result does not depend on scheduling. The queries' CTAs follow in the same
// grid, 16 elements a thread.
//
// Bound: bytes (16-bit rows in, 8-bit codes out, queries in and out) when the call is
// long; for the tokens of a decode batch the chain of loads before the first
// store (sequence, block id, scale, row) is what takes the time.
#include "block_scale.cuh"
#include "rope.cuh"
#include "launch_ext.h"

namespace pkv {
namespace {

constexpr int kGroup = 64;                 // threads on the keys, and on the values, of a run
constexpr int kThreads = 2 * kGroup;

// The row's sequence n, its position and the rows of its chunk; n = -1 for rows
// that no sequence owns or whose sequence is not valid (flagged elsewhere).
struct RowPlace {
  int n, pos, q0, ctx;
};

__device__ __forceinline__ bool seq_valid(const AppendBlockParams& p, int q0, int q1, int ctx) {
  return q0 >= 0 && q1 >= q0 && q1 <= p.rows && ctx >= q1 - q0 &&
         ctx <= (p.max_blocks << p.bs_log2) &&
         (p.cos_sin == nullptr || ctx <= p.max_position);
}

__device__ __forceinline__ RowPlace place_of(const AppendBlockParams& p, int row) {
  RowPlace r{-1, 0, 0, 0};
  // a decode batch has row n in sequence n: one round trip to see it
  int n = row;
  const bool guess = row < p.num_seqs;
  int q0 = guess ? p.cu_q_lens[row] : -1, q1 = guess ? p.cu_q_lens[row + 1] : -1;
  if (!(q0 <= row && row < q1)) {
    // the last n with cu_q_lens[n] <= row
    int lo = 0, hi = p.num_seqs + 1;       // cu[lo] <= row (if any), cu[hi] > row
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.cu_q_lens[mid] <= row) lo = mid;
      else hi = mid;
    }
    n = lo;
    if (n >= p.num_seqs) return r;
    q0 = p.cu_q_lens[n];
    q1 = p.cu_q_lens[n + 1];
    if (row < q0 || row >= q1) return r;
  }
  const int ctx = p.seq_lens[n];
  if (!seq_valid(p, q0, q1, ctx)) return r;
  r.n = n;
  r.q0 = q0;
  r.ctx = ctx;
  r.pos = ctx - (q1 - row);
  return r;
}

// Largest finite magnitude (bits) of the 16-bit values of a word pair by pair.
template <bool BF16>
__device__ __forceinline__ uint32_t finite_max(uint32_t m, const uint4& v) {
  constexpr uint32_t INF = BF16 ? 0x7F80u : 0x7C00u;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = w[i] & 0x7FFFu, b = (w[i] >> 16) & 0x7FFFu;
    if (a < INF) m = max(m, a);
    if (b < INF) m = max(m, b);
  }
  return m;
}

// Eight 16-bit values times 2^-e -> eight E4M3 codes.
template <bool BF16>
__device__ __forceinline__ uint2 encode_pow2_x8(const uint4& in, float inv) {
  const uint32_t w[4] = {in.x, in.y, in.z, in.w};
  uint32_t out[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t lo = f32x2_to_e4m3x2(widen16<BF16>(w[2 * j] & 0xFFFFu) * inv,
                                        widen16<BF16>(w[2 * j] >> 16) * inv);
    const uint32_t hi = f32x2_to_e4m3x2(widen16<BF16>(w[2 * j + 1] & 0xFFFFu) * inv,
                                        widen16<BF16>(w[2 * j + 1] >> 16) * inv);
    out[j] = lo | (hi << 16);
  }
  return make_uint2(out[0], out[1]);
}

// Four E4M3 codes times f (a power of two, at most 1) -> four E4M3 codes.
__device__ __forceinline__ uint32_t rescale_e4m3x4(uint32_t w, float f) {
  uint32_t out = 0;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t h2 = e4m3x2_to_f16x2((w >> (16 * j)) & 0xFFFFu);
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    out |= (uint32_t)f32x2_to_e4m3x2(v.x * f, v.y * f) << (16 * j);
  }
  return out;
}

// The 16 elements of item j of a head row, rotated where the row is a key or a
// query and the item lies in the rotated part; o.a / o.b go to off_a / off_b.
template <bool BF16, bool NEOX>
__device__ __forceinline__ Pair8 take_item(const uint16_t* row, const float* cs, int rot, int j,
                                           int& off_a, int& off_b) {
  if (cs != nullptr && j < rot / 16) return rotate_item<BF16, NEOX>(row, cs, rot, j, off_a, off_b);
  off_a = 16 * j;
  off_b = 16 * j + 8;
  return Pair8{*reinterpret_cast<const uint4*>(row + off_a),
               *reinterpret_cast<const uint4*>(row + off_b)};
}

template <bool BF16, bool NEOX>
__global__ void __launch_bounds__(kThreads) append_block_kernel(const AppendBlockParams p) {
  // a decode launched behind this kernel may become resident now; it waits
  // for this grid to finish before it reads anything
  if (threadIdx.x == 0) griddep_launch_dependents();
  __shared__ uint32_t s_max[4];
  const int tid = threadIdx.x;
  const int items = p.D / 16;               // of a head row

  if (blockIdx.x < p.kv_ctas) {
    const int h = blockIdx.x % p.Hkv;
    const int r0 = (int)(blockIdx.x / p.Hkv) * p.window;
    const bool is_v = tid >= kGroup;
    const int t = tid & (kGroup - 1);
    const uint16_t* src = static_cast<const uint16_t*>(is_v ? p.value : p.key);
    uint8_t* cache = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache);
    uint8_t* scales = is_v ? p.v_scales : p.k_scales;
    const int bs = 1 << p.bs_log2;
    for (int row = r0; row < min(p.rows, r0 + p.window); ++row) {
      const RowPlace at = place_of(p, row);        // the same for every thread of the CTA
      if (at.n < 0) continue;
      const int off = at.pos & (bs - 1);
      if (row != at.q0 && off != 0) continue;      // not the first row of a run
      const int run = min(bs - off, at.ctx - at.pos);
      const int id = p.block_tables[(int64_t)at.n * p.max_blocks + (at.pos >> p.bs_log2)];
      if (id < 0 || id >= p.num_blocks) {
        if (tid == 0 && h == 0) atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
        continue;
      }
      const int64_t unit = (int64_t)id * p.Hkv + h;
      const int stored = off == 0 ? -kE8M0Bias : min((int)scales[unit], 254) - kE8M0Bias;
      const uint16_t* rows = src + ((int64_t)row * p.Hkv + h) * p.D;
      const int64_t stride = (int64_t)p.Hkv * p.D;
      const float* cs = is_v || p.cos_sin == nullptr ? nullptr : p.cos_sin + (int64_t)at.pos * p.rot;

      uint32_t m = 0u;
      for (int i = t; i < run * items; i += kGroup) {
        const int k = i / items, j = i - k * items;
        int oa, ob;
        const Pair8 x = take_item<BF16, NEOX>(rows + k * stride,
                                              cs == nullptr ? nullptr : cs + (int64_t)k * p.rot,
                                              p.rot, j, oa, ob);
        m = finite_max<BF16>(finite_max<BF16>(m, x.a), x.b);
      }
      m = __reduce_max_sync(0xffffffffu, m);
      if ((tid & 31) == 0) s_max[tid >> 5] = m;
      __syncthreads();
      m = max(s_max[is_v ? 2 : 0], s_max[is_v ? 3 : 1]);
      __syncthreads();                             // the next run reuses s_max
      const int need = block_exponent(widen16<BF16>(m));
      const int e = max(stored, need);

      uint8_t* block = cache + (unit << p.bs_log2) * p.D;
      if (off != 0 && e > stored) {
        // the slots before and behind the run, to the new scale
        const float f = pow2_any(max(stored - e, -126));
        const int cpr = p.D / 16;
        for (int i = t; i < (bs - run) * cpr; i += kGroup) {
          int k = i / cpr;
          if (k >= off) k += run;
          uint4* c = reinterpret_cast<uint4*>(block + (int64_t)k * p.D + 16 * (i % cpr));
          const uint4 w = *c;
          *c = make_uint4(rescale_e4m3x4(w.x, f), rescale_e4m3x4(w.y, f), rescale_e4m3x4(w.z, f),
                          rescale_e4m3x4(w.w, f));
        }
      }
      const float inv = pow2_any(-e);
      for (int i = t; i < run * items; i += kGroup) {
        const int k = i / items, j = i - k * items;
        int oa, ob;
        const Pair8 x = take_item<BF16, NEOX>(rows + k * stride,
                                              cs == nullptr ? nullptr : cs + (int64_t)k * p.rot,
                                              p.rot, j, oa, ob);
        uint8_t* dst = block + (int64_t)(off + k) * p.D;
        *reinterpret_cast<uint2*>(dst + oa) = encode_pow2_x8<BF16>(x.a, inv);
        *reinterpret_cast<uint2*>(dst + ob) = encode_pow2_x8<BF16>(x.b, inv);
      }
      if (t == 0) scales[unit] = (uint8_t)(e + kE8M0Bias);
    }
    return;
  }

  // ---- queries: one thread per 16 elements --------------------------------------------
  const int64_t base = (int64_t)(blockIdx.x - p.kv_ctas) * kThreads;
  if (base == 0) {
    // one CTA looks every sequence over and says what is wrong with it
    for (int n = tid; n < p.num_seqs; n += kThreads) {
      const int q0 = p.cu_q_lens[n], q1 = p.cu_q_lens[n + 1], ctx = p.seq_lens[n];
      if (!seq_valid(p, q0, q1, ctx) && q0 != q1) {
        const bool past = p.cos_sin != nullptr && ctx > p.max_position;
        atomicOr(p.err, past ? PKV_DEVERR_POSITION : PKV_DEVERR_QLEN);
      }
    }
  }
  if (p.query_out == nullptr) return;
  const int64_t i = base + tid;
  const int per_row = p.Hq * items;
  const int64_t row = i / per_row;
  if (row >= p.rows) return;
  const RowPlace at = place_of(p, (int)row);
  if (at.n < 0) return;
  const int rest = (int)(i - row * per_row);
  const int hq = rest / items, j = rest - hq * items;
  const int64_t o = (row * p.Hq + hq) * p.D;
  int oa, ob;
  const Pair8 x = take_item<BF16, NEOX>(static_cast<const uint16_t*>(p.query) + o,
                                        p.cos_sin + (int64_t)at.pos * p.rot, p.rot, j, oa, ob);
  uint16_t* dst = static_cast<uint16_t*>(p.query_out) + o;
  *reinterpret_cast<uint4*>(dst + oa) = x.a;
  *reinterpret_cast<uint4*>(dst + ob) = x.b;
}

}  // namespace

pkv_status launch_append_block(const AppendBlockParams& params, pkv_dtype src_dtype,
                               cudaStream_t stream) {
  AppendBlockParams p = params;
  if (p.rows == 0) return PKV_OK;
  // rows per cache-write CTA: one while that gives at most some thousand CTAs
  // (most rows of a decode batch lead a run), up to 16 when rows are many (then
  // most do not, and a CTA per row would be spent finding that out)
  p.window = 1;
  while (p.window < 16 && (int64_t)p.rows * p.Hkv > (int64_t)8192 * p.window) p.window *= 2;
  const int64_t kv = (((int64_t)p.rows + p.window - 1) / p.window) * p.Hkv;
  const int64_t q = p.query_out == nullptr
                        ? 1
                        : ((int64_t)p.rows * p.Hq * (p.D / 16) + kThreads - 1) / kThreads;
  if (kv + q > 0x7FFFFFFF) return PKV_ERR_INVALID_ARG;
  p.kv_ctas = (unsigned int)kv;
  const unsigned int grid = (unsigned int)(kv + q);
  const bool neox = p.cos_sin == nullptr || p.neox != 0;
  if (src_dtype == PKV_BF16) {
    if (neox) append_block_kernel<true, true><<<grid, kThreads, 0, stream>>>(p);
    else append_block_kernel<true, false><<<grid, kThreads, 0, stream>>>(p);
  } else {
    if (neox) append_block_kernel<false, true><<<grid, kThreads, 0, stream>>>(p);
    else append_block_kernel<false, false><<<grid, kThreads, 0, stream>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace pkv
