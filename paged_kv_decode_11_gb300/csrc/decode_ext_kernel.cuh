// decode_ext_kernel.cuh — decode attention over E4M3 blocks with a scale per
// block and KV head, and with modified scores (a tanh cap, a bias by distance,
// a window of the last keys), instantiated by decode_ext.cu and
// decode_ext_wide.cu.
//
// Mathematics, for a query head with slope a and the position pos of its
// token, over the keys j it sees (pos - j < window):
//   x_j = scale 2^ek(j) <q, kcode_j>;  x_j <- c tanh(x_j / c);  x_j <- x_j - a (pos - j)
//   out = sum_j 2^(x_j log2 e) 2^ev(j) vcode_j / sum_j 2^(x_j log2 e)
// ek, ev are the exponents of the block of key j. The sum and the output are
// kept against references of their own: the probabilities against the largest
// x, the weights of V against the largest x + ev (both in log2). One
// reference for both would push the weights of blocks with a small V scale
// towards f16's subnormals whenever a block with a large one had been seen;
// with two, the P that meets the codes has its largest entry near 1 whatever the
// scales are. The second exponential is 4 per thread and page, which the loads
// hide.
//
// Work decomposition as in decode_kernel.cuh: one CTA per (partition, KV head,
// sequence), its warps taking the partition's 16-token pages in turn, each with
// its own ring of TMA loads; the warps merge on chip, the partitions through
// the workspace in the CTA that finishes last. A window moves the first
// partition to the page that holds its first key, so what lies before it costs
// nothing. A lane keeps the scale bytes of one of the next 32 pages of its warp
// (one byte per 16 to 64 tokens: the bytes of a block's KV heads share a
// sector), fetched while the pages are on their way.
//
// Bound: bytes (codes; 1/(BS D) of that for the scales). 128 sequences of 1,024 to
// 8,192 keys, 32 / 8 heads, D = 128: 205 us, 6.3 TB/s, 0.93 of the measured copy
// rate; a window of 1,024 at D = 256, bf16, 32 sequences: 45 us, 5.8 TB/s. Few and
// short contexts are bound by the chain of a CTA (length, table, pages, merge): one
// sequence of 700 keys 7.4 us.
#pragma once
#include <cuda.h>
#include "block_scale.cuh"
#include "decode_frags.cuh"
#include "launch_ext.h"

namespace pkv {

// Partial results are stored without subnormals (see count_partition).
__device__ __forceinline__ float mul_ftz(float a, float b) {
  float r;
  asm("mul.rn.ftz.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Counts a finished partition of a (sequence, KV head) and returns how many were counted
// before it, out of nparts (at most kMaxDecodeExtParts). The counter is 0 between calls of
// one size, but calls of other sizes that the workspace served may have put partial
// results there. Two of those floats make no number below nparts but 0, as none is
// subnormal: the first CTA to find such a word starts the count in its place, and those
// that added to it meanwhile add again. A word can change under a CTA at most twice for
// each of the other partitions.
__device__ __forceinline__ unsigned int count_partition(unsigned long long* ctr, int nparts,
                                                        unsigned int* err) {
  unsigned long long before = atom_add_acq_rel_gpu(ctr, 1ull);
  for (int i = 0; before >= (unsigned long long)nparts; ++i) {
    if (i > 3 * nparts) {                          // another call is counting here too
      atomicOr(err, PKV_DEVERR_COUNTER);
      return 0u;
    }
    unsigned long long now;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(now) : "l"(ctr) : "memory");
    if (now < (unsigned long long)nparts) before = atom_add_acq_rel_gpu(ctr, 1ull);
    else if (atom_cas_acq_rel_gpu(ctr, now, 1ull) == now) return 0u;
  }
  return (unsigned int)before;
}

template <int D, int KV, int NT, int NW, int NST>
struct DecodeExtCfg {
  using Geo = PageGeom<D, KV>;
  static constexpr int STAGE_BYTES = 2 * Geo::PAGE_BYTES;
  static constexpr int RING_BYTES = NW * NST * STAGE_BYTES;
  static constexpr int OBUF_BYTES = NW * 8 * NT * D * 4;      // warp merge, aliases the ring
  static constexpr int SMEM_BYTES =
      1024 + (RING_BYTES > OBUF_BYTES ? RING_BYTES : OBUF_BYTES);
};

// BSC: E4M3 pages with block scales.
template <int D, int KV, bool BSC, bool QBF16, int NT, int NW, int NST>
__global__ void __launch_bounds__(NW * 32)
    decode_ext_kernel(const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ DecodeExtParams ep) {
  static_assert(!BSC || KV == KV_E4M3, "block scales are for E4M3 codes");
  using Geo = PageGeom<D, KV>;
  using Cfg = DecodeExtCfg<D, KV, NT, NW, NST>;
  constexpr int STAGE = Cfg::STAGE_BYTES;
  constexpr int NH = 8 * NT;                       // head columns of the N dimension
  constexpr int NTH = NW * 32;
  const DecodeParams& p = ep.base;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[NW][NST];
  __shared__ float red_m[NW][NH], red_l[NW][NH];
  __shared__ float red_w[BSC ? NW : 1][BSC ? NH : 1];   // references of the V weights
  __shared__ int s_ids[kMaxPartitionTokens / kBS];
  __shared__ int s_last, s_stuck;
  __shared__ uint64_t s_mbar;     // the merge's bulk copies of the partials

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int G = p.G;
  // launched as a programmatic dependent: resident early, reads nothing
  // before the kernel ahead of it (the cache write) is done
  griddep_wait();

  const int cap = min(p.max_seq_len, p.max_blocks << p.bs_log2);
  const int part_idx = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  int ctx = p.seq_lens[b];
  if (ctx < 0 || ctx > cap) {
    if (tid == 0 && part_idx == 0 && h == 0) atomicOr(p.err, PKV_DEVERR_SEQ_LEN);
    ctx = ctx < 0 ? 0 : cap;
  }
  const int first = ep.window > 0 ? max(0, ctx - ep.window) : 0;   // first key seen
  const int origin = first & ~(kBS - 1);                           // of the partitions
  const int nparts = ctx > 0 ? (ctx - origin + p.part - 1) / p.part : 1;
  if (part_idx >= nparts) return;
  const int tok0 = origin + part_idx * p.part;
  const int tok1 = min(ctx, tok0 + p.part);
  const int npages = (tok1 - tok0 + kBS - 1) / kBS;
  const int page0 = tok0 / kBS;

  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t base = (raw_base + 1023u) & ~1023u;
  uint8_t* basep = smem_raw + (base - raw_base);

  // page rows of the tensor maps: a block of 16 << ppb_shift tokens holds
  // that many consecutive 16-token pages per KV head
  const int sub_mask = (1 << p.ppb_shift) - 1;
  for (int i = tid; i < npages; i += NTH) {
    const int pg = page0 + i;
    int id = p.block_tables[(int64_t)b * p.max_blocks + (pg >> p.ppb_shift)];
    if (id < 0 || id >= p.num_blocks) {
      atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
      id = 0;
    }
    s_ids[i] = ((id * p.Hkv + h) << p.ppb_shift) + (pg & sub_mask);
  }
  if (tid == 0) {
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
#pragma unroll
    for (int w = 0; w < NW; ++w)
#pragma unroll
      for (int s = 0; s < NST; ++s) mbar_init(&bars[w][s], 1);
    mbar_init(&s_mbar, 1);
    fence_barrier_init();
    s_stuck = 0;
  }
  __syncthreads();

  // ---- per-warp ring of TMA loads, issued by lane 0 ------------------------------------
  const uint32_t wbase = base + warp * NST * STAGE;
  uint8_t* wbasep = basep + warp * NST * STAGE;
  const int nmine = warp < npages ? (npages - warp + NW - 1) / NW : 0;
  const uint64_t evict_first = policy_evict_first();   // pages are read once per call
  auto issue = [&](int k) {
    const int st = k % NST;
    uint64_t* bar = &bars[warp][st];
    uint8_t* dst = wbasep + st * STAGE;
    const int z = s_ids[warp + NW * k];
    mbar_arrive_expect_tx(bar, STAGE);
#pragma unroll
    for (int bx = 0; bx < Geo::NBOX; ++bx) {
      tma_load_3d_hint(dst + bx * Geo::BOX_BYTES, &tmK, bar, bx * Geo::BOX_ELEMS, 0, z,
                       evict_first);
      tma_load_3d_hint(dst + Geo::PAGE_BYTES + bx * Geo::BOX_BYTES, &tmV, bar,
                       bx * Geo::BOX_ELEMS, 0, z, evict_first);
    }
  };
  if (lane == 0)
    for (int k = 0; k < NST && k < nmine; ++k) issue(k);
  int issued = min(NST, nmine);

  // scale bytes (K low, V high) of the warp's pages 32 q + lane; a page row
  // shifted down is its block's entry, block * Hkv + head
  auto scales_of = [&](int q) -> uint32_t {
    const int k = 32 * q + lane;
    if (k >= nmine) return 0u;
    const int64_t i = s_ids[warp + NW * k] >> p.ppb_shift;
    return (uint32_t)ep.k_block_scales[i] | ((uint32_t)ep.v_block_scales[i] << 8);
  };
  uint32_t sc_cur = 0u, sc_next = 0u;
  if constexpr (BSC) {
    sc_cur = scales_of(0);
    sc_next = scales_of(1);
  }

  // ---- query fragments (heads in N), straight from global memory --------------------
  const uint16_t* qb = static_cast<const uint16_t*>(p.q) + ((int64_t)b * p.Hq + h * G) * D;
  uint32_t qf[NT][D / 16][2];
  int qshift;
  load_qT_frags<D, KV, QBF16, NT>(qf, qb, G, lane, qshift);

  float oacc[NT][D / 16][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int t = 0; t < D / 16; ++t)
      oacc[nt][t][0] = oacc[nt][t][1] = oacc[nt][t][2] = oacc[nt][t][3] = 0.f;
  // m: reference of the probabilities (and their sum l); mw: of the V weights
  // (the same one without block scales)
  float m[NT][2], mw[NT][2], l[NT][2], slope[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[nt][e] = mw[nt][e] = -INFINITY;
      l[nt][e] = 0.f;
      const int hh = 8 * nt + 2 * c + e;
      slope[nt][e] = ep.slopes != nullptr && hh < G ? ep.slopes[h * G + hh] * kLog2e : 0.f;
    }
  // q was scaled by 2^-qshift for the f16 MMAs: scale the scores back (exact)
  const float sl2 =
      p.qk_scale_log2 * (KV == KV_E4M3 && !BSC ? p.k_scales[h] : 1.f) * pow2f(qshift);
  const int tk0 = st_row_token<KV>(g, 0), tk8 = st_row_token<KV>(g, 1);

  for (int k = 0; k < nmine; ++k) {
    const int st = k % NST;
    bool ok = mbar_wait_bounded(&bars[warp][st], (k / NST) & 1);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) {
      if (lane == 0) atomicOr(p.err, PKV_DEVERR_TIMEOUT);
      // let what this warp still has in flight land (bounded), then stop; if
      // that wait gives up too, a late copy could still land in the ring, so
      // the CTA leaves the ring's space (the merge buffer below) alone
      bool drained = true;
      for (int kk = k + 1; kk < issued; ++kk)
        drained &= mbar_wait_bounded(&bars[warp][kk % NST], (kk / NST) & 1, 1u << 16);
      if (!__all_sync(0xffffffffu, drained) && lane == 0) s_stuck = 1;
      break;
    }
    const uint32_t kpage = wbase + st * STAGE;
    const uint32_t vpage = kpage + Geo::PAGE_BYTES;
    const int tbase = tok0 + (warp + NW * k) * kBS;
    if (tok1 - tbase < kBS || tbase < first) {
      // rows behind the context or before the window get weight 0, and
      // whatever they hold must not turn that into NaN, so zero them in V
      uint8_t* vp = wbasep + st * STAGE + Geo::PAGE_BYTES;
      if (tok1 - tbase < kBS) zero_page_rows<D, KV>(vp, tok1 - tbase, lane);
      if (tbase < first) zero_page_head<D, KV>(vp, first - tbase, lane);
      fence_proxy_async_smem();
      __syncwarp();
    }
    float ksl2 = sl2, evl = 0.f;
    if constexpr (BSC) {
      if (k != 0 && k % 32 == 0) {
        sc_cur = sc_next;
        sc_next = scales_of(k / 32 + 1);
      }
      const uint32_t sc = __shfl_sync(0xffffffffu, sc_cur, k % 32);
      ksl2 = sl2 * e8m0_value(sc & 0xFFu);
      evl = e8m0_log2(sc >> 8);
    }
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
    // E4M3: take the page into registers and refill the stage at once, so the
    // next load is in flight while this page's math runs.
    E4M3PageRegs<D> pr;
    if constexpr (KV == KV_E4M3) {
      load_e4m3_page<D>(pr, kpage, vpage, lane);
      __syncwarp();
      if (lane == 0 && k + NST < nmine) {
        fence_proxy_async_smem();
        issue(k + NST);
      }
      kq_regs<D, NT>(s, qf, pr.k);
    } else {
      kq_page<D, KV, NT>(s, qf, kpage, lane);
    }

    // online softmax in the log2 domain, against references per column that lie
    // kWeightHeadLog2 below a maximum and move only when the page's outgrows that
    // by kRefSlackLog2, so the accumulators are rescaled rarely (weights stay below
    // 2^15)
    const bool v0 = tbase + tk0 < tok1 && tbase + tk0 >= first;
    const bool v8 = tbase + tk8 < tok1 && tbase + tk8 >= first;
    const float back0 = (float)(ctx - 1 - (tbase + tk0)), back8 = (float)(ctx - 1 - (tbase + tk8));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] *= ksl2;
    // up to kCoarseCap the first form is good enough, and it is the faster one beside a
    // page's other work (128 sequences of 1,024 to 8,192 keys 208 us; a choice per score 219)
    if (ep.cap_log2 > kCoarseCap / kLn2) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; e += 2)
          softcap_log2_pair(s[nt][e], s[nt][e + 1], ep.cap_log2, ep.two_over_cap);
    } else if (ep.cap_log2 != 0.f) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          s[nt][e] = softcap_log2(s[nt][e], ep.cap_log2, ep.two_over_cap);
    }
    float pmax[NT][2];
    bool move = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x0 = s[nt][e], x8 = s[nt][2 + e];
        x0 = fmaf(-slope[nt][e], back0, x0);
        x8 = fmaf(-slope[nt][e], back8, x8);
        s[nt][e] = v0 ? x0 : -INFINITY;
        s[nt][2 + e] = v8 ? x8 : -INFINITY;
        pmax[nt][e] = col_max8(fmaxf(s[nt][e], s[nt][2 + e])) - kWeightHeadLog2;
        move |= pmax[nt][e] > m[nt][e] + kRefSlackLog2;
        if constexpr (BSC) move |= pmax[nt][e] + evl > mw[nt][e] + kRefSlackLog2;
      }
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // (a lambda per column, so that the accumulators are indexed by constants)
          auto rescale = [&](float alpha) {
#pragma unroll
            for (int t = 0; t < D / 16; ++t) {
              oacc[nt][t][e] *= alpha;
              oacc[nt][t][2 + e] *= alpha;
            }
          };
          if (pmax[nt][e] > m[nt][e] + kRefSlackLog2) {
            const float alpha = m[nt][e] == -INFINITY ? 0.f : exp2f(m[nt][e] - pmax[nt][e]);
            m[nt][e] = pmax[nt][e];
            l[nt][e] *= alpha;
            if constexpr (!BSC) rescale(alpha);
          }
          if constexpr (BSC) {
            const float top = pmax[nt][e] + evl;
            if (top > mw[nt][e] + kRefSlackLog2) {
              rescale(mw[nt][e] == -INFINITY ? 0.f : exp2f(mw[nt][e] - top));
              mw[nt][e] = top;
            }
          }
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float ms = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
        const float p0 = exp2f(s[nt][e] - ms), p8 = exp2f(s[nt][2 + e] - ms);
        l[nt][e] += p0 + p8;
        if constexpr (BSC) {
          // (a NaN scale makes its weights NaN whatever the reference)
          const float mv = (mw[nt][e] == -INFINITY ? 0.f : mw[nt][e]) - evl;
          s[nt][e] = exp2f(s[nt][e] - mv);
          s[nt][2 + e] = exp2f(s[nt][2 + e] - mv);
        } else {
          s[nt][e] = p0;
          s[nt][2 + e] = p8;
        }
      }
    // weights rounded to the MMA's 16-bit type, by half a step at most (bf16 2^-8, f16
    // 2^-11; the sums took them unrounded), as the output is to the query's
    uint32_t pb[NT][2];
    pT_frags<KV, NT>(pb, s);
    if constexpr (KV == KV_E4M3) {
      vp_regs<D, NT>(oacc, pb, pr.v);
    } else {
      vp_page<D, KV, NT>(oacc, pb, vpage, lane);
      __syncwarp();
      if (lane == 0 && k + NST < nmine) {
        fence_proxy_async_smem();
        issue(k + NST);
      }
    }
    issued = min(k + 1 + NST, nmine);
  }

  // ---- merge the warps of this CTA ----------------------------------------------------
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[nt][e] = col_sum8(l[nt][e]);
      if (g == 0) {
        // (a warp that saw nothing but NaN scores has no reference, but its sum is NaN: any
        // finite reference takes that to the merged sum)
        red_m[warp][8 * nt + 2 * c + e] =
            l[nt][e] != l[nt][e] ? fmaxf(m[nt][e], -3e38f) : m[nt][e];
        red_l[warp][8 * nt + 2 * c + e] = l[nt][e];
        if constexpr (BSC) red_w[warp][8 * nt + 2 * c + e] = mw[nt][e];
      }
    }
  __syncthreads();  // every warp is done with its ring: the ring's space is free
  if (s_stuck) {
    // (after a timeout whose drain gave up; the error word holds the timeout)
    // no output or partial from this CTA, only its count, so that the
    // (b, h) counter still completes and comes back to zero
    if (nparts > 1 && tid == 0) {
      unsigned long long* ctr = p.done + (int64_t)b * p.Hkv + h;
      if ((int)count_partition(ctr, nparts, p.err) + 1 == nparts) *ctr = 0ull;
    }
    return;
  }
  // largest reference over the warps: of the V weights, or (without block
  // scales the same) of the probabilities
  auto top_w = [&](int hh) {
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, BSC ? red_w[BSC ? w : 0][BSC ? hh : 0] : red_m[w][hh]);
    return M;
  };
  float* obuf = reinterpret_cast<float*>(basep);   // [NW][G][D]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int hh = 8 * nt + 2 * c + e;
      if (hh < G) {
        const float mine = BSC ? mw[nt][e] : m[nt][e];
        const float f = mine == -INFINITY ? 0.f : exp2f(mine - top_w(hh));
        float* orow = obuf + (warp * G + hh) * D;
#pragma unroll
        for (int t = 0; t < D / 16; ++t) {
          orow[ot_row_dim<D, KV>(t, g, 0)] = oacc[nt][t][e] * f;
          orow[ot_row_dim<D, KV>(t, g, 1)] = oacc[nt][t][2 + e] * f;
        }
      }
    }
  __syncthreads();

  const float vscale = (KV == KV_E4M3 && !BSC) ? p.v_scales[h] : 1.f;
  const int64_t row0 = (int64_t)b * p.Hq + h * G;
  for (int idx = tid; idx < G * (D / 2); idx += NTH) {
    const int hh = idx / (D / 2), d = 2 * (idx % (D / 2));
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, red_m[w][hh]);
    float L = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (red_m[w][hh] != -INFINITY) L += red_l[w][hh] * exp2f(red_m[w][hh] - M);
      o0 += obuf[(w * G + hh) * D + d];
      o1 += obuf[(w * G + hh) * D + d + 1];
    }
    const bool nonempty = !(L == 0.f);               // (a NaN sum is no empty row)
    float inv = nonempty ? 1.f / L : 0.f;
    if constexpr (BSC) {
      // out = (sum of weights times codes) 2^(their reference) / (L 2^M)
      const float W = top_w(hh);
      inv *= W == -INFINITY ? 0.f : exp2f(W - M);
    }
    if (nparts == 1) {
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + (row0 + hh) * D + d) =
          pack2<QBF16>(o0 * inv * vscale, o1 * inv * vscale);
      if (d == 0 && p.out_lse != nullptr)
        p.out_lse[row0 + hh] = nonempty ? (M + log2f(L)) * kLn2 : -INFINITY;
    } else {
      const int64_t wrow = (row0 + hh) * p.max_parts + part_idx;
      *reinterpret_cast<float2*>(p.ws_o + wrow * D + d) = make_float2(mul_ftz(o0, inv), mul_ftz(o1, inv));
      if (d == 0) p.ws_lse[wrow] = nonempty ? mul_ftz(M + log2f(L), 1.f) : -INFINITY;
    }
  }
  if (nparts == 1) return;

  // ---- the CTA that completes the last partition of (b, h) merges them ------------------
  // (bulk-copied partials as in decode_kernel.cuh)
  __syncthreads();
  unsigned long long* ctr = p.done + (int64_t)b * p.Hkv + h;
  if (tid == 0) s_last = (int)count_partition(ctr, nparts, p.err) + 1 == nparts;
  __syncthreads();
  if (!s_last) return;
  if (tid == 0) *ctr = 0ull;
  // A chunk of CH partitions comes into the ring's space in one bulk copy per
  // head. Then a warp per head turns the chunk's log2-sum-exps into weights
  // 2^(lse - M) against the running maximum M (and says by how much to scale what
  // was summed before), and every thread sums its float4 columns with them: no
  // exponential and no branch in that loop. (With both in it a partition took
  // 0.17 us, and contexts could not be split finely.)
  constexpr int NF = (NH * (D / 4) + NTH - 1) / NTH;   // float4 columns per thread
  constexpr int AVAIL = Cfg::SMEM_BYTES - 1024;         // the ring's space
  const int CH = max(1, min(nparts, (AVAIL - 16) / (G * (D + 1) * 4)));
  float* s_w = reinterpret_cast<float*>(basep);                         // [G][CH]
  float* s_o = reinterpret_cast<float*>(basep + ((G * CH * 4 + 15) & ~15));  // [G][CH][D]
  __shared__ float s_scale[NH];
  float M[(NH + NW - 1) / NW], Z[(NH + NW - 1) / NW];  // of the warp's heads warp, warp + NW, ..
  float4 acc[NF];
#pragma unroll
  for (int i = 0; i < (NH + NW - 1) / NW; ++i) {
    M[i] = -INFINITY;
    Z[i] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < NF; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  const float* lse_rows = p.ws_lse + row0 * (int64_t)p.max_parts;
  for (int c0 = 0, ci = 0; c0 < nparts; c0 += CH, ++ci) {
    const int n = min(CH, nparts - c0);
    if (tid == 0) {
      // the partials were written, and this shared memory read and written, through the
      // generic proxy; the barrier above ordered both before these fences
      fence_proxy_async_global();
      fence_proxy_async_smem();
      mbar_arrive_expect_tx(&s_mbar, (uint32_t)(G * n * D * 4));
      for (int hh = 0; hh < G; ++hh)
        bulk_load(s_o + hh * CH * D, p.ws_o + ((row0 + hh) * p.max_parts + c0) * D,
                  (uint32_t)(n * D * 4), &s_mbar);
    }
#pragma unroll
    for (int i = 0; i < (NH + NW - 1) / NW; ++i) {
      const int hh = warp + NW * i;
      if (hh >= G) continue;
      float top = M[i];
      for (int sp = lane; sp < n; sp += 32) {
        const float v = ldcg_f32(lse_rows + hh * p.max_parts + c0 + sp);
        s_w[hh * CH + sp] = v;
        top = fmaxf(top, v);
      }
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float ref = top == -INFINITY ? 0.f : top;
      float sum = 0.f;
      for (int sp = lane; sp < n; sp += 32) {          // each lane its own values
        const float w = exp2f(s_w[hh * CH + sp] - ref);
        s_w[hh * CH + sp] = w;
        sum += w;
      }
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      const float scale = M[i] == -INFINITY ? 0.f : exp2f(M[i] - ref);
      Z[i] = Z[i] * scale + sum;
      M[i] = top;
      if (lane == 0) s_scale[hh] = scale;
    }
    // the vote is also the barrier that publishes the weights; a CTA whose
    // copies did not all land leaves as one, after waiting once more
    // (bounded), since they target its own shared memory
    const bool landed = mbar_wait_bounded(&s_mbar, ci & 1);
    if (__syncthreads_or(!landed)) {
      if (tid == 0) atomicOr(p.err, PKV_DEVERR_TIMEOUT);
      mbar_wait_bounded(&s_mbar, ci & 1);
      return;
    }
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      const int f = tid + i * NTH;
      if (f < G * (D / 4)) {
        const int hh = f / (D / 4), d4 = f - hh * (D / 4);
        const float sc = s_scale[hh];
        acc[i].x *= sc; acc[i].y *= sc; acc[i].z *= sc; acc[i].w *= sc;
        const float* w = s_w + hh * CH;
        const float4* o = reinterpret_cast<const float4*>(s_o + hh * CH * D) + d4;
#pragma unroll 4
        for (int sp = 0; sp < n; ++sp) {
          const float4 v = o[sp * (D / 4)];
          acc[i].x = fmaf(w[sp], v.x, acc[i].x);
          acc[i].y = fmaf(w[sp], v.y, acc[i].y);
          acc[i].z = fmaf(w[sp], v.z, acc[i].z);
          acc[i].w = fmaf(w[sp], v.w, acc[i].w);
        }
      }
    }
    __syncthreads();   // the next chunk reuses the staging space
  }
#pragma unroll
  for (int i = 0; i < (NH + NW - 1) / NW; ++i) {
    const int hh = warp + NW * i;
    if (hh >= G || lane != 0) continue;
    // (a NaN sum stays one)
    s_scale[hh] = Z[i] == 0.f ? 0.f : vscale / Z[i];
    if (p.out_lse != nullptr)
      p.out_lse[row0 + hh] = Z[i] == 0.f ? -INFINITY : (M[i] + log2f(Z[i])) * kLn2;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NF; ++i) {
    const int f = tid + i * NTH;
    if (f < G * (D / 4)) {
      const int hh = f / (D / 4), d4 = f - hh * (D / 4);
      const float inv = s_scale[hh];
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + (row0 + hh) * D + d4 * 4) =
          make_uint2(pack2<QBF16>(acc[i].x * inv, acc[i].y * inv),
                     pack2<QBF16>(acc[i].z * inv, acc[i].w * inv));
    }
  }
}

template <int D, int KV, bool BSC, bool QBF16, int NT, int NW>
static pkv_status launch_decode_ext_t(const DecodeExtParams& p, const CUtensorMap& tmK,
                                      const CUtensorMap& tmV, cudaStream_t stream) {
  // ring depth per warp: 3 stages of E4M3 pages or 2 of 16-bit ones in CTAs of
  // kDecodeWarps warps (several per SM), 3 of either in whole-context CTAs
  constexpr int NST = NW == kDecodeWideWarps || KV == KV_E4M3 ? 3 : 2;
  using Cfg = DecodeExtCfg<D, KV, NT, NW, NST>;
  auto kern = decode_ext_kernel<D, KV, BSC, QBF16, NT, NW, NST>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PKV_ERR_CUDA;
  static std::atomic<bool> attr_set[64];  // per device; the call is idempotent
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Cfg::SMEM_BYTES) != cudaSuccess)
      return PKV_ERR_CUDA;
    attr_set[dev] = true;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.base.grid_parts, p.base.Hkv, p.base.B);
  cfg.blockDim = dim3(NW * 32);
  cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tmK, tmV, p) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

template <int D, int NW, int KV, bool BSC, bool QBF16>
static pkv_status launch_decode_ext_nt(const DecodeExtParams& p, const CUtensorMap& tmK,
                                       const CUtensorMap& tmV, cudaStream_t stream) {
  if constexpr (D <= 128) {
    if (p.base.G > 8)
      return launch_decode_ext_t<D, KV, BSC, QBF16, 2, NW>(p, tmK, tmV, stream);
  } else {
    if (p.base.G > 8) return PKV_ERR_UNSUPPORTED;        // 16 head columns at D = 256: not built
  }
  return launch_decode_ext_t<D, KV, BSC, QBF16, 1, NW>(p, tmK, tmV, stream);
}

template <int D, int NW>
static pkv_status launch_decode_ext_d(const DecodeExtParams& p, pkv_dtype q_dtype,
                                      pkv_dtype kv_dtype, bool bsc, const CUtensorMap& tmK,
                                      const CUtensorMap& tmV, cudaStream_t stream) {
  const bool qbf = q_dtype == PKV_BF16;
  if (kv_dtype == PKV_FP8_E4M3) {
    if (bsc)
      return qbf ? launch_decode_ext_nt<D, NW, KV_E4M3, true, true>(p, tmK, tmV, stream)
                 : launch_decode_ext_nt<D, NW, KV_E4M3, true, false>(p, tmK, tmV, stream);
    return qbf ? launch_decode_ext_nt<D, NW, KV_E4M3, false, true>(p, tmK, tmV, stream)
               : launch_decode_ext_nt<D, NW, KV_E4M3, false, false>(p, tmK, tmV, stream);
  }
  if (kv_dtype == PKV_BF16)
    return launch_decode_ext_nt<D, NW, KV_BF16, false, true>(p, tmK, tmV, stream);
  return launch_decode_ext_nt<D, NW, KV_F16, false, false>(p, tmK, tmV, stream);
}

}  // namespace pkv
