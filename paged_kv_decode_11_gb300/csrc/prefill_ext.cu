// prefill_ext.cu — chunked-prefill attention over E4M3 blocks with a scale per
// block and KV head, and with modified scores (tanh cap, bias by distance,
// window, prefix): which kernel a call takes, and the one with m16n8k16
// products, for E4M3 caches at head_dim 256 (whose query tile leaves the
// tensor-core kernel's f16 rings no room, as in prefill.cu).
//
// Mathematics: decode_ext_kernel.cuh's for every row of a chunk; row i of a
// chunk of L tokens on P cached ones stands at pos = P + i and sees the keys j
// with j <= pos or j < prefix, j < context and (with a window) pos - j <
// window: one interval [lo, lim] per row, lo = max(0, pos - window + 1),
// lim = max(pos, prefix - 1).
//
// Work decomposition as in prefill.cu: one CTA per (query tile, KV head,
// sequence), the tile's 64 MMA rows being (token, head of the GQA group)
// pairs; a producer warp streams pages by TMA, four consumer warps own 16 rows
// each. The keys start at the page that holds the first key any row sees.
// Each consumer lane keeps the scale bytes of one of the next 32 pages.
#include <cuda.h>
#include "block_scale.cuh"
#include "launch_ext.h"

namespace pkv {
namespace {

constexpr int kConsumers = 4;
constexpr int kRows = 16 * kConsumers;

template <int D, int KV, bool BSC, bool QBF16, int NST, int KT>
__global__ void __launch_bounds__((kConsumers + 1) * 32)
    prefill_ext_kernel(const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV,
                       const __grid_constant__ PrefillExtParams ep) {
  static_assert(!BSC || KV == KV_E4M3, "block scales are for E4M3 codes");
  using Geo = PageGeom<D, KV>;
  constexpr int STAGE = 2 * KT * Geo::PAGE_BYTES;
  constexpr int TILE = kBS * KT;
  const PrefillParams& p = ep.base;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full_bar[NST];
  __shared__ uint64_t empty_bar[NST];

  if (threadIdx.x == 0) griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int qt = blockIdx.x, h = blockIdx.y, n = blockIdx.z;
  const int G = p.G;
  const int q0 = p.cu_q_lens[n];
  const int L = p.cu_q_lens[n + 1] - q0;
  const int ctx = p.seq_lens[n];
  // a chunk longer than its context or than the grid covers, or whose rows are
  // not rows of q and out
  if (L < 0 || L > ctx || L > p.max_q_len || q0 < 0 || q0 > p.q_rows - L ||
      ctx > ((p.max_blocks * kBS) << p.ppb_shift)) {
    if (threadIdx.x == 0 && qt == 0 && h == 0) atomicOr(p.err, PKV_DEVERR_QLEN);
    return;
  }
  const int P = ctx - L;
  const int i0 = qt * p.q_tile;
  if (i0 >= L) return;
  const int i1 = min(L, i0 + p.q_tile);
  const int prefix = ep.prefix_lens != nullptr ? min(max(ep.prefix_lens[n], 0), ctx) : 0;
  const int first = ep.window > 0 ? max(0, P + i0 - ep.window + 1) : 0;  // any row's first key
  const int origin = first & ~(kBS - 1);
  const int key_end = max(P + i1, prefix);             // exclusive
  const int pg0 = origin / kBS;                        // the tiles' first page
  const int n_pages = (key_end - origin + kBS - 1) / kBS;
  const int n_tiles = (key_end - origin + TILE - 1) / TILE;

  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t base = (raw_base + 1023u) & ~1023u;
  uint8_t* basep = smem_raw + (base - raw_base);
  const int32_t* table = p.block_tables + (int64_t)n * p.max_blocks;

  if (threadIdx.x == 0) {
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
    for (int s = 0; s < NST; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], kConsumers);
    }
    fence_barrier_init();
  }
  __syncthreads();

  if (warp == kConsumers) {
    // ---- producer warp: its lanes look up the page rows 32 pages at a time,
    // one chunk ahead; lane 0 issues the loads ----------------------------------------
    static_assert(32 % KT == 0, "a tile's pages lie in one chunk");
    auto page_row = [&](int lp) -> int {
      if (lp >= n_pages) return 0;
      const int pg = pg0 + lp;
      int id = table[pg >> p.ppb_shift];
      if (id < 0 || id >= p.num_blocks) {
        atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
        id = 0;
      }
      return ((id * p.Hkv + h) << p.ppb_shift) + (pg & ((1 << p.ppb_shift) - 1));
    };
    int z_cur = page_row(lane), z_next = page_row(32 + lane), chunk = 0;
    for (int t = 0; t < n_tiles; ++t) {
      const int st = t % NST;
      bool ok = t < NST || mbar_wait_bounded(&empty_bar[st], ((t / NST) - 1) & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        if (lane == 0) atomicOr(p.err, PKV_DEVERR_TIMEOUT);
        break;
      }
      if ((t * KT) / 32 != chunk) {
        z_cur = z_next;
        ++chunk;
        z_next = page_row(32 * (chunk + 1) + lane);
      }
      const int npg = min(KT, n_pages - t * KT);
      if (lane == 0) mbar_arrive_expect_tx(&full_bar[st], npg * 2 * Geo::PAGE_BYTES);
      uint8_t* dst = basep + st * STAGE;
      for (int pg = 0; pg < npg; ++pg) {
        const int z = __shfl_sync(0xffffffffu, z_cur, (t * KT + pg) % 32);
        if (lane == 0) {
#pragma unroll
          for (int bx = 0; bx < Geo::NBOX; ++bx) {
            tma_load_3d(dst + pg * Geo::PAGE_BYTES + bx * Geo::BOX_BYTES, &tmK, &full_bar[st],
                        bx * Geo::BOX_ELEMS, 0, z);
            tma_load_3d(dst + (KT + pg) * Geo::PAGE_BYTES + bx * Geo::BOX_BYTES, &tmV,
                        &full_bar[st], bx * Geo::BOX_ELEMS, 0, z);
          }
        }
      }
    }
    return;
  }

  // ---- consumer warps: 16 rows each ---------------------------------------------
  const int g = lane >> 2, c = lane & 3;
  const int rows_used = p.q_tile * G;
  int qi[2], hq[2], lo[2], lim[2], pos[2];
  bool live[2];
  float slope[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = warp * 16 + g + 8 * e;
    live[e] = r < rows_used && i0 + r / G < i1;
    qi[e] = i0 + r / G;
    hq[e] = h * G + r % G;
    pos[e] = P + qi[e];
    lo[e] = ep.window > 0 ? max(0, pos[e] - ep.window + 1) : 0;
    lim[e] = live[e] ? max(pos[e], prefix - 1) : -1;     // -1: no key
    slope[e] = live[e] && ep.slopes != nullptr ? ep.slopes[hq[e]] * kLog2e : 0.f;
  }
  const uint16_t* qbase = static_cast<const uint16_t*>(p.q);
  const void* rowg = live[0] ? qbase + ((int64_t)(q0 + qi[0]) * p.Hq + hq[0]) * D : nullptr;
  const void* rowg8 = live[1] ? qbase + ((int64_t)(q0 + qi[1]) * p.Hq + hq[1]) * D : nullptr;
  uint32_t qf[D / 16][4];
  int qsh[2];
  load_q_frags<D, KV, QBF16>(qf, rowg, rowg8, lane, qsh[0], qsh[1]);
  const int warp_lim = __reduce_max_sync(0xffffffffu, max(lim[0], lim[1]));
  const int warp_lo = __reduce_min_sync(
      0xffffffffu, min(live[0] ? lo[0] : 0x7FFFFFFF, live[1] ? lo[1] : 0x7FFFFFFF));

  float oacc[D / 8][4];
#pragma unroll
  for (int t = 0; t < D / 8; ++t) oacc[t][0] = oacc[t][1] = oacc[t][2] = oacc[t][3] = 0.f;
  // references of the probabilities and of the V weights, and the sums
  float m[2] = {-INFINITY, -INFINITY}, mw[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  const float sl2 = p.qk_scale_log2 * (KV == KV_E4M3 && !BSC ? p.k_scales[h] : 1.f);
  const float slr[2] = {sl2 * pow2f(qsh[0]), sl2 * pow2f(qsh[1])};

  auto scales_of = [&](int q) -> uint32_t {
    return page_scale_bytes(table, pg0 + 32 * q + lane, pg0 + n_pages, p.ppb_shift, p.num_blocks,
                            p.Hkv, h, ep.k_block_scales, ep.v_block_scales);
  };
  uint32_t sc_cur = 0u, sc_next = 0u;
  if constexpr (BSC) {
    sc_cur = scales_of(0);
    sc_next = scales_of(1);
  }

  for (int t = 0; t < n_tiles; ++t) {
    const int st = t % NST;
    bool ok = mbar_wait_bounded(&full_bar[st], (t / NST) & 1);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) {
      if (lane == 0) atomicOr(p.err, PKV_DEVERR_TIMEOUT);
      break;
    }
    if constexpr (BSC) {
      if (t != 0 && (t * KT) % 32 == 0) {
        sc_cur = sc_next;
        sc_next = scales_of(t * KT / 32 + 1);
      }
    }
    const int kbase = origin + t * TILE;
    if (kbase <= warp_lim && kbase + TILE > warp_lo) {
      const uint32_t kst = base + st * STAGE;
      const uint32_t vst = kst + KT * Geo::PAGE_BYTES;
      const int npg = min(KT, n_pages - t * KT);
      if (kbase < first) {
        // V rows before the first key any row sees (every warp writes the same zeros)
        zero_page_head<D, KV>(basep + st * STAGE + KT * Geo::PAGE_BYTES, first - kbase, lane);
        __syncwarp();
      }
      float s[2 * KT][4];
#pragma unroll
      for (int j = 0; j < 2 * KT; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
      for (int pg = 0; pg < KT; ++pg) {
        if (pg < npg && kbase + pg * kBS <= warp_lim) {
          qk_page<D, KV>(s, 2 * pg, qf, kst + pg * Geo::PAGE_BYTES, lane);
        }
      }
      float mx[2] = {-INFINITY, -INFINITY}, mxw[2] = {-INFINITY, -INFINITY}, evl[KT];
#pragma unroll
      for (int pg = 0; pg < KT; ++pg) {
        float kf = 1.f;
        evl[pg] = 0.f;
        if constexpr (BSC) {
          const uint32_t sc = __shfl_sync(0xffffffffu, sc_cur, (t * KT + pg) % 32);
          kf = e8m0_value(sc & 0xFFu);
          evl[pg] = e8m0_log2(sc >> 8);
        }
        float pm[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int jj = 0; jj < 2; ++jj)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int j = 2 * pg + jj, e = w >> 1;
            const int key = kbase + pg * kBS + s_col_token<KV>(jj, c, w & 1);
            float x = s[j][w] * (slr[e] * kf);
            if (ep.cap_log2 != 0.f) x = softcap_log2(x, ep.cap_log2, ep.two_over_cap);
            x = fmaf(-slope[e], (float)abs(pos[e] - key), x);
            s[j][w] = key <= lim[e] && key >= lo[e] ? x : -INFINITY;
            pm[e] = fmaxf(pm[e], s[j][w]);
          }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[e] = fmaxf(mx[e], pm[e]);
          mxw[e] = fmaxf(mxw[e], pm[e] + evl[pg]);
        }
      }
      float ms[2], mv[2], aw[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mn = fmaxf(m[e], quad_max(mx[e]));
        ms[e] = mn == -INFINITY ? 0.f : mn;
        const float as = exp2f(m[e] - ms[e]);
        m[e] = mn;
        l[e] *= as;
        if constexpr (BSC) {
          const float wn = fmaxf(mw[e], quad_max(mxw[e]));
          mv[e] = wn == -INFINITY ? 0.f : wn;
          aw[e] = exp2f(mw[e] - mv[e]);
          mw[e] = wn;
        } else {
          mv[e] = ms[e];
          aw[e] = as;
        }
      }
#pragma unroll
      for (int j = 0; j < 2 * KT; ++j)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const int e = w >> 1;
          const float pr = exp2f(s[j][w] - ms[e]);
          l[e] += pr;
          // (a masked score has weight 0 even on a page whose scale is NaN)
          if constexpr (BSC)
            s[j][w] = s[j][w] == -INFINITY ? 0.f : exp2f(s[j][w] + (evl[j / 2] - mv[e]));
          else
            s[j][w] = pr;
        }
#pragma unroll
      for (int tt = 0; tt < D / 8; ++tt)
#pragma unroll
        for (int w = 0; w < 4; ++w) oacc[tt][w] *= aw[w >> 1];
#pragma unroll
      for (int pg = 0; pg < KT; ++pg) {
        if (pg < npg && kbase + pg * kBS <= warp_lim) {
          uint32_t pa[4];
          pack_p<KV>(pa, s, 2 * pg);
          pv_page<D, KV>(oacc, pa, vst + pg * Geo::PAGE_BYTES, lane,
                         min(kBS, ctx - (kbase + pg * kBS)));
        }
      }
      if (kbase < first) fence_proxy_async_smem();     // the zeros, before the stage is refilled
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty_bar[st]);
  }

  const float vscale = KV == KV_E4M3 && !BSC ? p.v_scales[h] : 1.f;
  uint16_t* out = static_cast<uint16_t*>(p.out);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float Ls = quad_sum(l[e]);
    float inv = Ls > 0.f ? vscale / Ls : 0.f;
    if constexpr (BSC) inv *= mw[e] == -INFINITY ? 0.f : exp2f(mw[e] - m[e]);
    if (!live[e]) continue;
    const int64_t row = (int64_t)(q0 + qi[e]) * p.Hq + hq[e];
#pragma unroll
    for (int tt = 0; tt < D / 8; ++tt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float v = oacc[tt][2 * e + k] * inv;
        out[row * D + o_col_dim<D, KV>(tt, c, k)] =
            (uint16_t)(pack2<QBF16>(v, v) & 0xFFFFu);
      }
    if (c == 0 && p.out_lse != nullptr)
      p.out_lse[row] = Ls > 0.f ? (m[e] + log2f(Ls)) * kLn2 : -INFINITY;
  }
}

template <int D, int KV, bool BSC, bool QBF16>
pkv_status launch_t(const PrefillExtParams& ep, const CUtensorMap& tmK, const CUtensorMap& tmV,
                    cudaStream_t stream) {
  // D = 256: two pages per tile and two stages keep registers and shared memory in bounds
  constexpr int NST = D > 128 ? 2 : 3;
  constexpr int KT = D > 128 ? 2 : 4;
  constexpr int SMEM = NST * 2 * KT * PageGeom<D, KV>::PAGE_BYTES + 1024;
  auto kern = prefill_ext_kernel<D, KV, BSC, QBF16, NST, KT>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PKV_ERR_CUDA;
  static std::atomic<bool> attr_set[64];  // per device; the call is idempotent
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) !=
        cudaSuccess)
      return PKV_ERR_CUDA;
    attr_set[dev] = true;
  }
  PrefillExtParams p = ep;
  p.base.q_tile = kRows / p.base.G;
  const dim3 grid((p.base.max_q_len + p.base.q_tile - 1) / p.base.q_tile, p.base.Hkv,
                  p.base.num_seqs);
  kern<<<grid, (kConsumers + 1) * 32, SMEM, stream>>>(tmK, tmV, p);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace

pkv_status launch_prefill_ext(const PrefillExtParams& p, int head_dim, pkv_dtype q_dtype,
                              pkv_dtype kv_dtype, bool block_scaled, const CUtensorMap& tmQ,
                              const CUtensorMap& tmK, const CUtensorMap& tmV,
                              cudaStream_t stream) {
  if (prefill_tc_supported(head_dim, kv_dtype))
    return block_scaled
               ? launch_prefill_tc_block(p, head_dim, q_dtype, tmQ, tmK, tmV, stream)
               : launch_prefill_tc_mod(p, head_dim, q_dtype, kv_dtype, tmQ, tmK, tmV, stream);
  if (head_dim != 256 || kv_dtype != PKV_FP8_E4M3) return PKV_ERR_UNSUPPORTED;
  const bool qbf = q_dtype == PKV_BF16;
  if (block_scaled)
    return qbf ? launch_t<256, KV_E4M3, true, true>(p, tmK, tmV, stream)
               : launch_t<256, KV_E4M3, true, false>(p, tmK, tmV, stream);
  return qbf ? launch_t<256, KV_E4M3, false, true>(p, tmK, tmV, stream)
             : launch_t<256, KV_E4M3, false, false>(p, tmK, tmV, stream);
}

}  // namespace pkv
