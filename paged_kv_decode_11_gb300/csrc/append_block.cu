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
// Rotation: y1 = x1 c - x2 s, y2 = x2 c + x1 s, each the fp32 value nearest to the
// exact sum, then rounded to the source type. (The plain fp32 sum is off by up to
// its products' rounding, which cancellation makes large against the sum; one element
// in 2^12 of f16 would land on the other side of a midpoint.) Doubles are slow, so the
// sum is carried as an unevaluated pair: the products with their errors (fma), their
// sum with its error (Knuth's two-sum), the parts added up. y1 and y2 of a pair run
// through the packed two-float instructions side by side.
//
// Work decomposition. Tokens of a sequence that fall into one block are
// consecutive rows (a run of at most BS), so a run, not a token, is the unit:
// its first row (the leader) starts a sequence's chunk or a block. A CTA takes
// `window` consecutive rows and one KV head and does the runs whose leaders
// lie among its rows; half of its threads do the keys, the other half the
// values. A group holds 2 x 16 elements of the run per thread in registers from
// the maximum to the codes; of a longer run (more than 32 tokens at head_dim 128)
// what was not kept is loaded and rotated again (holding 4 x 16 spilled registers
// and left room for fewer CTAs: 2,039 tokens of 24 / 8 heads 14.9 us, 13.2 with 2). No two
// CTAs touch one block and head, so nothing is atomic and the result does not depend on
// scheduling. The queries follow in the same grid: one warp or up to eight take a row, a
// thread keeps the angles of its 16 dims and goes over the row's heads.
//
// Bound: when the call is long, the latency of its loads at the 24 warps that an SM holds:
// the chunk kernels are kept to 80 registers a thread for that, and spill 120 to 136 bytes
// (47.4 us with two CTAs an SM, 43.8 with three and two heads in flight). 7 chunks of 150 to 2,100
// tokens, 28 / 4 heads, D = 128, f16, half of each head rotated: 139 MB in 35 us, 4.0 TB/s
// of algorithmic bytes, DRAM 36 % busy; a tensor copy of as many bytes takes 44.6 us.
// (41.6 us with a warp's loads waiting for the stores before them, 91 with a CTA per row
// and doubles for the undecided sums.) For the tokens of a decode batch
// the chain of loads before the first store (sequence, block id, scale) is what
// takes the time, so everything that can be addressed without them is loaded first:
// 128 tokens of 32 / 8 heads 5.4 us, one token 2.6.
#include "block_scale.cuh"
#include "f32x2.cuh"
#include "rope.cuh"
#include "launch_ext.h"

namespace pkv {
namespace {

// A CTA has GROUP threads on the keys of a run and GROUP on its values.
constexpr int kShortGroup = 32, kLongGroup = 128;
constexpr int kKeep = 2;                   // items (16 elements) a thread keeps of a run

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

// Every lane of a warp, each for a row of its own (or -1). Few sequences are looked
// up at once, in one round trip: a lane reads the offsets and the length of one.
__device__ __forceinline__ RowPlace place_of(const AppendBlockParams& p, int row) {
  int n, q0, q1, ctx;
  if (p.num_seqs < 32) {
    const int lane = threadIdx.x & 31;
    const int cu = lane <= p.num_seqs ? p.cu_q_lens[lane] : 0x7FFFFFFF;
    const int len = lane < p.num_seqs ? p.seq_lens[lane] : 0;
    n = -1;                                // the last n with cu_q_lens[n] <= row
    for (int k = 0; k <= p.num_seqs; ++k) n += __shfl_sync(0xffffffffu, cu, k) <= row ? 1 : 0;
    const int at = max(n, 0);
    q0 = __shfl_sync(0xffffffffu, cu, at);
    q1 = __shfl_sync(0xffffffffu, cu, (at + 1) & 31);
    ctx = __shfl_sync(0xffffffffu, len, at);
  } else {
    // a decode batch has row n in sequence n: one round trip to see it
    n = row;
    q0 = q1 = -1;
    ctx = 0;
    if (row >= 0 && row < p.num_seqs) {
      q0 = p.cu_q_lens[row];
      q1 = p.cu_q_lens[row + 1];
      ctx = p.seq_lens[row];
    }
    if (!(q0 <= row && row < q1)) {
      int lo = 0, hi = p.num_seqs + 1;     // cu[lo] <= row (if any), cu[hi] > row
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.cu_q_lens[mid] <= row) lo = mid;
        else hi = mid;
      }
      n = lo;
      if (n < p.num_seqs) {
        q0 = p.cu_q_lens[n];
        q1 = p.cu_q_lens[n + 1];
        ctx = p.seq_lens[n];
      }
    }
  }
  if (n < 0 || n >= p.num_seqs || row < q0 || row >= q1 || !seq_valid(p, q0, q1, ctx))
    return RowPlace{-1, 0, 0, 0};
  return RowPlace{n, ctx - (q1 - row), q0, ctx};
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

// The angles of one item: 8 cosines and 8 sines.
struct Angles {
  float4 c[2], s[2];
};

__device__ __forceinline__ Angles load_angles(const float* cs, int half, int j) {
  const float4* c = reinterpret_cast<const float4*>(cs + 8 * j);
  const float4* s = reinterpret_cast<const float4*>(cs + half + 8 * j);
  return Angles{{c[0], c[1]}, {s[0], s[1]}};
}

// (y1, y2) of each pair of an item, as described above.
template <bool BF16, bool NEOX>
__device__ __forceinline__ Pair8 rotate_pairs(const Pair8& in, const Angles& an) {
  float x1[8], x2[8];
  item_pairs<BF16, NEOX>(in.a, in.b, x1, x2);
  const float c[8] = {an.c[0].x, an.c[0].y, an.c[0].z, an.c[0].w,
                      an.c[1].x, an.c[1].y, an.c[1].z, an.c[1].w};
  const float s[8] = {an.s[0].x, an.s[0].y, an.s[0].z, an.s[0].w,
                      an.s[1].x, an.s[1].y, an.s[1].z, an.s[1].w};
  float y1[8], y2[8];
  f2 finite = pack_f2(0.f, 0.f);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const f2 x = pack_f2(x1[e], x2[e]), z = pack_f2(x2[e], x1[e]);
    const f2 cc = pack_f2(c[e], c[e]), ss = pack_f2(-s[e], s[e]);
    // the rounded products by single multiplications: packed ones were merged into
    // the additions below, whose error terms then belong to another sum
    const float qa = __fmul_rn(x1[e], c[e]), qb = __fmul_rn(x2[e], c[e]);
    const float pa = __fmul_rn(x2[e], -s[e]), pb = __fmul_rn(x1[e], s[e]);
    const f2 nq = pack_f2(-qa, -qb), p = pack_f2(pa, pb), np = pack_f2(-pa, -pb);
    const f2 qe = fma2(x, cc, nq), pe = fma2(z, ss, np);             // what they leave
    const f2 sum = sub2(p, nq);
    const f2 bb = add2(sum, nq);
    const f2 err = sub2(sub2(p, bb), add2(nq, sub2(sum, bb)));       // what the sum leaves
    const f2 rest = add2(err, add2(qe, pe));
    const f2 r = add2(sum, rest);
    finite = fma2(r, pack_f2(0.f, 0.f), finite);
    const float2 y = unpack_f2(r);
    y1[e] = y.x;
    y2[e] = y.y;
  }
  const float2 f = unpack_f2(finite);
  if (!(f.x == 0.f && f.y == 0.f)) {
    // an infinity or NaN among the inputs (the error terms are NaN then)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y1[e] = fmaf(x1[e], c[e], -(x2[e] * s[e]));
      y2[e] = fmaf(x2[e], c[e], x1[e] * s[e]);
    }
  }
  uint32_t w1[4], w2[4];                  // y of pairs 2 i and 2 i + 1
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (NEOX) {
      w1[i] = pack2<BF16>(y1[2 * i], y1[2 * i + 1]);
      w2[i] = pack2<BF16>(y2[2 * i], y2[2 * i + 1]);
    } else {                              // pairs lie side by side: a holds 0..3, b 4..7
      w1[i] = pack2<BF16>(y1[i], y2[i]);
      w2[i] = pack2<BF16>(y1[4 + i], y2[4 + i]);
    }
  }
  return Pair8{make_uint4(w1[0], w1[1], w1[2], w1[3]), make_uint4(w2[0], w2[1], w2[2], w2[3])};
}

// Where the two 8-element halves of item j of a head row lie: the partners of a
// rotated item (rotate-half), or 16 consecutive elements.
template <bool NEOX>
__device__ __forceinline__ void item_offsets(int j, int rot, int& a, int& b) {
  const bool halves = NEOX && j < rot / 16;
  a = halves ? 8 * j : 16 * j;
  b = halves ? 8 * j + rot / 2 : 16 * j + 8;
}

template <bool NEOX>
__device__ __forceinline__ Pair8 load_item(const uint16_t* row, int j, int rot) {
  int a, b;
  item_offsets<NEOX>(j, rot, a, b);
  return Pair8{*reinterpret_cast<const uint4*>(row + a), *reinterpret_cast<const uint4*>(row + b)};
}

template <bool BF16, bool NEOX, int GROUP>
__global__ void __launch_bounds__(2 * GROUP, GROUP == kLongGroup ? 3 : 8)
    append_block_kernel(const __grid_constant__ AppendBlockParams p) {
  constexpr int kGroup = GROUP, kThreads = 2 * GROUP;
  // a decode launched behind this kernel may become resident now; it waits
  // for this grid to finish before it reads anything
  if (threadIdx.x == 0) griddep_launch_dependents();
  __shared__ uint32_t s_max[kThreads / 32];
  const int tid = threadIdx.x;
  const int items_log2 = p.d_log2 - 4, items = 1 << items_log2;     // of a head row

  if (blockIdx.x < p.kv_ctas) {
    const int h = blockIdx.x % p.Hkv;
    const int r0 = (int)(blockIdx.x / p.Hkv) * p.window;
    const bool is_v = tid >= kGroup;
    const int t = tid & (kGroup - 1);
    const uint16_t* src = static_cast<const uint16_t*>(is_v ? p.value : p.key);
    uint8_t* cache = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache);
    uint8_t* scales = is_v ? p.v_scales : p.k_scales;
    const int bs = 1 << p.bs_log2;
    const int rot = is_v || p.cos_sin == nullptr ? 0 : p.rot;
    const int64_t stride = (int64_t)p.Hkv << p.d_log2;
    // a lane looks one row up; then the rows that lead a run are taken in turn
    const int lane = tid & 31;
    const RowPlace mine =
        place_of(p, lane < p.window && r0 + lane < p.rows ? r0 + lane : -1);
    uint32_t leaders = __ballot_sync(
        0xffffffffu, mine.n >= 0 && (r0 + lane == mine.q0 || (mine.pos & (bs - 1)) == 0));
    while (leaders != 0u) {                        // the same for every warp of the CTA
      const int at = __ffs(leaders) - 1;
      leaders &= leaders - 1u;
      const int row = r0 + at;
      const int n = __shfl_sync(0xffffffffu, mine.n, at);
      const int pos = __shfl_sync(0xffffffffu, mine.pos, at);
      const int ctx = __shfl_sync(0xffffffffu, mine.ctx, at);
      const int off = pos & (bs - 1);
      const int run = min(bs - off, ctx - pos);
      const int count = run << items_log2;
      const int id = p.block_tables[(int64_t)n * p.max_blocks + (pos >> p.bs_log2)];
      const uint16_t* rows = src + ((int64_t)row * p.Hkv + h << p.d_log2);
      // items base + t and base + t + kGroup of the run (its chunk of kKeep * kGroup items from
      // base on), rotated
      Pair8 x[kKeep];
      auto take = [&](int base) {
#pragma unroll
        for (int u = 0; u < kKeep; ++u) {
          const int i = base + t + u * kGroup, k = i >> items_log2, j = i & (items - 1);
          x[u] = i < count ? load_item<NEOX>(rows + k * stride, j, rot)
                           : Pair8{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
        }
#pragma unroll
        for (int u = 0; u < kKeep; ++u) {
          const int i = base + t + u * kGroup, k = i >> items_log2, j = i & (items - 1);
          if (i < count && j < rot / 16)
            x[u] = rotate_pairs<BF16, NEOX>(
                x[u], load_angles(p.cos_sin + (int64_t)(pos + k) * p.rot, p.rot / 2, j));
        }
      };
      uint32_t m = 0u;
      int base = 0;
      for (;; base += kKeep * kGroup) {
        take(base);
#pragma unroll
        for (int u = 0; u < kKeep; ++u)
          m = finite_max<BF16>(finite_max<BF16>(m, x[u].a), x[u].b);
        if (base + kKeep * kGroup >= count) break;
      }
      const bool known = id >= 0 && id < p.num_blocks;
      const int64_t unit = known ? (int64_t)id * p.Hkv + h : 0;
      const int stored =
          off == 0 || !known ? -kE8M0Bias : min((int)scales[unit], 254) - kE8M0Bias;
      m = __reduce_max_sync(0xffffffffu, m);
      __syncthreads();                             // the run before has read s_max
      if (lane == 0) s_max[tid >> 5] = m;
      __syncthreads();
      if (!known) {
        if (tid == 0 && h == 0) atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
        continue;
      }
#pragma unroll
      for (int w = 0; w < kGroup / 32; ++w) m = max(m, s_max[(is_v ? kGroup / 32 : 0) + w]);
      const int e = max(stored, block_exponent(widen16<BF16>(m)));

      uint8_t* block = cache + (unit << (p.bs_log2 + p.d_log2));
      if (off != 0 && e > stored) {
        // the slots before and behind the run, to the new scale
        const float f = pow2_any(max(stored - e, -126));
        for (int i = t; i < (bs - run) << items_log2; i += kGroup) {
          int k = i >> items_log2;
          if (k >= off) k += run;
          uint4* c = reinterpret_cast<uint4*>(block + (k << p.d_log2) + 16 * (i & (items - 1)));
          const uint4 w = *c;
          *c = make_uint4(rescale_e4m3x4(w.x, f), rescale_e4m3x4(w.y, f), rescale_e4m3x4(w.z, f),
                          rescale_e4m3x4(w.w, f));
        }
      }
      const float inv = pow2_any(-e);
      for (;;) {                                   // the last chunk is still there
#pragma unroll
        for (int u = 0; u < kKeep; ++u) {
          const int i = base + t + u * kGroup, k = i >> items_log2, j = i & (items - 1);
          if (i >= count) continue;
          int a, b;
          item_offsets<NEOX>(j, rot, a, b);
          uint8_t* dst = block + ((off + k) << p.d_log2);
          const uint2 ca = encode_pow2_x8<BF16>(x[u].a, inv), cb = encode_pow2_x8<BF16>(x[u].b, inv);
          *reinterpret_cast<uint2*>(dst + a) = ca;
          *reinterpret_cast<uint2*>(dst + b) = cb;
        }
        if (base == 0) break;
        base -= kKeep * kGroup;
        take(base);
      }
      if (t == 0) scales[unit] = (uint8_t)(e + kE8M0Bias);
    }
    return;
  }

  // ---- queries --------------------------------------------------------------------------
  const unsigned int cta = blockIdx.x - p.kv_ctas;
  if (cta == 0) {
    // one CTA looks every sequence over and says what is wrong with it
    for (int n = tid; n < p.num_seqs; n += kThreads) {
      const int c0 = p.cu_q_lens[n], c1 = p.cu_q_lens[n + 1], ctx = p.seq_lens[n];
      if (!seq_valid(p, c0, c1, ctx) && c0 != c1) {
        const bool past = p.cos_sin != nullptr && ctx > p.max_position;
        atomicOr(p.err, past ? PKV_DEVERR_POSITION : PKV_DEVERR_QLEN);
      }
    }
  }
  if (p.query_out == nullptr) return;
  const int lane = tid & 31;
  const int64_t task = (int64_t)cta * (kThreads / 32) + (tid >> 5);
  const int row = (int)(task >> p.slices_log2), slices = 1 << p.slices_log2;
  const int slice = (int)task & (slices - 1);
  if (row >= p.rows) return;
  const int64_t o = (int64_t)row * p.Hq << p.d_log2;
  const uint16_t* q = static_cast<const uint16_t*>(p.query) + o;
  uint16_t* out = static_cast<uint16_t*>(p.query_out) + o;
  // the rotated items: lane = (head, item j) with as many heads at a time as fit, j
  // and its angles staying; the warp's heads advance by `step`
  const int R = p.rot / 16, per = 32 / R, step = per * slices;
  const int j = lane % R;
  const int h_end = lane < per * R ? p.Hq : 0;
  int h0 = slice * per + lane / R;
  constexpr int U = 2;
  Pair8 x[U];
  auto load = [&](Pair8 (&to)[U], int h) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h + u * step < h_end) to[u] = load_item<NEOX>(q + ((h + u * step) << p.d_log2), j, p.rot);
  };
  load(x, h0);
  // the dims behind the rotated ones, 8 at a time (in place they are there already)
  const int chunks = (1 << (p.d_log2 - 3)) - 2 * R;
  const int n_rest = q == out ? 0 : p.Hq * chunks;
  constexpr int C = 4;
  uint4 rest[C];
  auto rest_at = [&](int i) {
    const int h = i / chunks;
    return (h << p.d_log2) + p.rot + 8 * (i - h * chunks);
  };
  auto load_rest = [&](int i0) {
#pragma unroll
    for (int u = 0; u < C; ++u)
      if (i0 + 32 * slices * u < n_rest)
        rest[u] = *reinterpret_cast<const uint4*>(q + rest_at(i0 + 32 * slices * u));
  };
  load_rest(slice * 32 + lane);
  const RowPlace at = place_of(p, row);
  if (at.n < 0) return;
  const Angles an = load_angles(p.cos_sin + (int64_t)at.pos * p.rot, p.rot / 2, j);
  for (int i0 = slice * 32 + lane; i0 < n_rest;) {
#pragma unroll
    for (int u = 0; u < C; ++u)
      if (i0 + 32 * slices * u < n_rest)
        *reinterpret_cast<uint4*>(out + rest_at(i0 + 32 * slices * u)) = rest[u];
    i0 += 32 * slices * C;
    load_rest(i0);
  }
  int a, b;
  item_offsets<NEOX>(j, p.rot, a, b);
  while (h0 < h_end) {
    Pair8 next[U];                                 // on their way while x is turned
    load(next, h0 + U * step);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * step;
      if (h >= h_end) continue;
      const Pair8 y = rotate_pairs<BF16, NEOX>(x[u], an);
      *reinterpret_cast<uint4*>(out + (h << p.d_log2) + a) = y.a;
      *reinterpret_cast<uint4*>(out + (h << p.d_log2) + b) = y.b;
    }
    h0 += U * step;
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = next[u];
  }
}

}  // namespace

template <int GROUP>
static void launch_group(AppendBlockParams& p, pkv_dtype src_dtype, unsigned int grid,
                         cudaStream_t stream) {
  const bool neox = p.cos_sin == nullptr || p.neox != 0;
  constexpr int T = 2 * GROUP;
  if (src_dtype == PKV_BF16) {
    if (neox) append_block_kernel<true, true, GROUP><<<grid, T, 0, stream>>>(p);
    else append_block_kernel<true, false, GROUP><<<grid, T, 0, stream>>>(p);
  } else {
    if (neox) append_block_kernel<false, true, GROUP><<<grid, T, 0, stream>>>(p);
    else append_block_kernel<false, false, GROUP><<<grid, T, 0, stream>>>(p);
  }
}

pkv_status launch_append_block(const AppendBlockParams& params, pkv_dtype src_dtype,
                               cudaStream_t stream) {
  AppendBlockParams p = params;
  if (p.rows == 0) return PKV_OK;
  // rows per cache-write CTA: about as many as a run has on average (at most
  // rows / BS + num_seqs rows lead one), rounded up, so that few CTAs meet no leader
  // (spent finding that out) and few meet several (done in turn)
  const int64_t leaders = ((int64_t)p.rows >> p.bs_log2) + p.num_seqs;
  p.window = 1;
  while (p.window < 32 && p.window * leaders < p.rows) p.window *= 2;
  // a warp on the keys of a run while runs may be single tokens, four for chunks
  const bool is_short = p.window == 1;
  const int group = is_short ? kShortGroup : kLongGroup;
  const int64_t kv = (((int64_t)p.rows + p.window - 1) / p.window) * p.Hkv;
  // warps per row of queries: enough that few rows still fill the GPU, while each has
  // two heads' worth of items to do (297 rows of 56 heads: one warp each
  // 12.1 us, eight 5.5)
  const int per = p.cos_sin == nullptr ? 1 : 32 / (p.rot / 16);
  p.slices_log2 = 0;
  while (p.slices_log2 < 3 && ((int64_t)p.rows << p.slices_log2) < 4096 &&
         (per << p.slices_log2) < p.Hq)
    ++p.slices_log2;
  const int64_t warps = (int64_t)p.rows << p.slices_log2, wpc = 2 * group / 32;
  const int64_t q = p.query_out == nullptr ? 1 : (warps + wpc - 1) / wpc;
  if (kv + q > 0x7FFFFFFF) return PKV_ERR_INVALID_ARG;
  p.kv_ctas = (unsigned int)kv;
  if (is_short) launch_group<kShortGroup>(p, src_dtype, (unsigned int)(kv + q), stream);
  else launch_group<kLongGroup>(p, src_dtype, (unsigned int)(kv + q), stream);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace pkv
