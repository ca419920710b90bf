// rope_cache.cu — rope_reshape_and_cache: the rotary position embedding of
// the new tokens' queries and keys, fused with the cache write of their keys
// and values ("RoPE + KV cache write -- fused, no intermediate alloc",
// rvLLM: High-performance LLM inference in Rust, Kernel Compiler Stack). The
// rotation is RoFormer's rotary embedding: pair (x1, x2) of a head turned by
// the angle of the token's position, taken from the caller's cos/sin table:
//   y1 = x1 c - x2 s,   y2 = x2 c + x1 s.
//
// Each result is defined as the product terms exact in double, one rounding
// of the sum to double, then one round-to-nearest-even to the 16-bit source
// dtype. Doubles are slow on this part, so a thread first works in fp32:
//   r = fma(xa, ca, +-fl(xb sb)),  |r - exact| <= (ulp(r) + ulp(fl(xb sb))) / 2,
// and rounds r - b and r + b to 16 bits with b = 2 max(ulp(r), ulp(xb sb)),
// both computed so that [r - b, r + b] contains the exact value. Rounding is
// monotone, so when both ends give the same 16-bit value that value is the
// rounding of the exact sum; and the exact sum then lies at least one fp32
// ulp from every 16-bit midpoint, so its rounding to double does not move
// it across one either: the value equals the defined result. Only when the
// ends differ (the exact sum sits near a midpoint, about 1 element in 2^12)
// does the thread redo that element in double.
//
// Work items, per token: for each query head and each key head, rot_dim/16
// rotation items of 16 elements (rotate-half: dims 8j..8j+7 with their
// partners 8j+rot/2..; interleaved: dims 16j..16j+15, eight adjacent pairs);
// for each key head, (D - rot_dim)/8 pass-through chunks of 8; for each value
// head, D/8 chunks of 8. One thread per item, 16-byte loads and stores.
// Query rows are rewritten in place: an item owns both halves of its pairs,
// so no other thread reads what it writes. Rotated keys go straight to the
// cache (bit copy or E4M3 encode, as reshape_and_cache), never to memory in
// between.
#include "rope.cuh"
#include "launch_cache.h"

namespace pkv {

template <bool BF16, bool TO_FP8, bool NEOX>
__global__ void __launch_bounds__(256) rope_cache_kernel(const RopeCacheParams p) {
  // a decode launched behind this kernel may become resident now; it waits
  // for this grid to finish before it reads anything
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int R = p.rot / 16;                 // rotation items per head
  const int PT = (p.D - p.rot) / 8;         // pass-through chunks per key head
  const int C8 = p.D / 8;                   // chunks per value head
  const int nq = p.Hq * R, nk = p.Hkv * (R + PT), nv = p.Hkv * C8;
  const int per_tok = nq + nk + nv;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (int64_t)p.num_tokens * per_tok) return;
  const int64_t t = i / per_tok;
  int r = (int)(i - t * per_tok);
  const int64_t pos = p.positions[t];
  if (pos < 0 || pos >= p.max_position) {
    if (r == 0) atomicOr(p.err, PKV_DEVERR_POSITION);
    return;
  }
  const float* cs = p.cos_sin + pos * p.rot;
  if (r < nq) {                                           // query: rotate in place
    const int h = r / R, j = r - (r / R) * R;
    uint16_t* row = static_cast<uint16_t*>(p.query) + (t * p.Hq + h) * p.D;
    int oa, ob;
    const Pair8 y = rotate_item<BF16, NEOX>(row, cs, p.rot, j, oa, ob);
    *reinterpret_cast<uint4*>(row + oa) = y.a;
    *reinterpret_cast<uint4*>(row + ob) = y.b;
    return;
  }
  const int64_t slot = p.slots[t];
  if (slot < 0) return;
  if (slot >= ((int64_t)p.num_blocks << p.bs_log2)) {
    if (r == nq) atomicOr(p.err, PKV_DEVERR_SLOT);
    return;
  }
  r -= nq;
  if (r < nk) {                                           // key: rotate, then store
    const int per_head = R + PT;
    const int h = r / per_head, j = r - h * per_head;
    const uint16_t* row = static_cast<const uint16_t*>(p.key) + (t * p.Hkv + h) * p.D;
    const float ks = TO_FP8 ? p.k_scales[h] : 1.f;
    const int64_t base = cache_elem(slot, h, p.Hkv, p.D, 0, p.bs_log2);
    if (j < R) {
      int oa, ob;
      const Pair8 y = rotate_item<BF16, NEOX>(row, cs, p.rot, j, oa, ob);
      store_row8<BF16, TO_FP8>(p.k_cache, base + oa, y.a, ks);
      store_row8<BF16, TO_FP8>(p.k_cache, base + ob, y.b, ks);
    } else {
      const int off = p.rot + 8 * (j - R);
      store_row8<BF16, TO_FP8>(p.k_cache, base + off,
                               *reinterpret_cast<const uint4*>(row + off), ks);
    }
    return;
  }
  r -= nk;                                                // value: store
  const int h = r / C8, off = 8 * (r - h * C8);
  const uint16_t* row = static_cast<const uint16_t*>(p.value) + (t * p.Hkv + h) * p.D;
  const float vs = TO_FP8 ? p.v_scales[h] : 1.f;
  store_row8<BF16, TO_FP8>(p.v_cache, cache_elem(slot, h, p.Hkv, p.D, off, p.bs_log2),
                           *reinterpret_cast<const uint4*>(row + off), vs);
}

pkv_status launch_rope_cache(const RopeCacheParams& p, pkv_dtype src_dtype, pkv_dtype kv_dtype,
                             cudaStream_t stream) {
  const int64_t per_tok = (int64_t)p.Hq * (p.rot / 16) +
                          (int64_t)p.Hkv * (p.rot / 16 + (p.D - p.rot) / 8) +
                          (int64_t)p.Hkv * (p.D / 8);
  const int64_t total = (int64_t)p.num_tokens * per_tok;
  if (total == 0) return PKV_OK;
  const int threads = 256;
  const int64_t blocks = (total + threads - 1) / threads;
  if (blocks > 0x7FFFFFFF) return PKV_ERR_INVALID_ARG;
  const bool bf = (src_dtype == PKV_BF16);
  const bool fp8 = (kv_dtype == PKV_FP8_E4M3);
  const unsigned g = (unsigned)blocks;
#define PKV_ROPE_LAUNCH(B, F, N) rope_cache_kernel<B, F, N><<<g, threads, 0, stream>>>(p)
  if (p.neox) {
    if (bf && fp8) PKV_ROPE_LAUNCH(true, true, true);
    else if (bf) PKV_ROPE_LAUNCH(true, false, true);
    else if (fp8) PKV_ROPE_LAUNCH(false, true, true);
    else PKV_ROPE_LAUNCH(false, false, true);
  } else {
    if (bf && fp8) PKV_ROPE_LAUNCH(true, true, false);
    else if (bf) PKV_ROPE_LAUNCH(true, false, false);
    else if (fp8) PKV_ROPE_LAUNCH(false, true, false);
    else PKV_ROPE_LAUNCH(false, false, false);
  }
#undef PKV_ROPE_LAUNCH
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace pkv
