// block_scale.cuh — the arithmetic of E4M3 blocks with one power-of-two scale
// (E8M0) per block and KV head, and of modified attention scores.
//
// A power of two because E4M3 is a floating format: scaling by 2^e moves a
// code's exponent and keeps its bits, so a block loses nothing against a
// scale that fits its largest element exactly, and a block whose scale grows
// is re-encoded without error until a code becomes subnormal. The factor of
// a score, 2^(scale - 127), is exact too.
#pragma once
#include <cstdint>
#include "common.cuh"

namespace pkv {

constexpr int kE8M0Bias = 127;
constexpr int kBlockMinExp = -60;       // smallest exponent the append gives a block

// 2^e for e in [-127, 127] (2^-127 is subnormal).
__device__ __forceinline__ float pow2_any(int e) {
  return __int_as_float(e == -127 ? 0x00400000 : (e + 127) << 23);
}

// The value of an E8M0 scale: 2^(s - 127), NaN for 255.
__device__ __forceinline__ float e8m0_value(uint32_t s) {
  return s == 255u ? __int_as_float(0x7FFFFFFF) : pow2_any((int)s - kE8M0Bias);
}

// Its log2 (NaN for 255).
__device__ __forceinline__ float e8m0_log2(uint32_t s) {
  return s == 255u ? __int_as_float(0x7FFFFFFF) : (float)((int)s - kE8M0Bias);
}

// Smallest e >= kBlockMinExp with amax <= 448 * 2^e = 1.75 * 2^(e + 8), for a
// finite amax >= 0 that a 16-bit type holds: with amax = m 2^k, 1 <= m < 2, e is
// k - 8, or k - 7 where m > 1.75.
__device__ __forceinline__ int block_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(e, kBlockMinExp);
}

// The scale bytes (K low, V high) of the block that holds 16-token page `page` of
// a sequence, for KV head h; 0 for pages at or past `end`. A block id outside the
// pool reads block 0's (the page loads flag it).
__device__ __forceinline__ uint32_t page_scale_bytes(const int32_t* table_row, int page, int end,
                                                     int ppb_shift, int num_blocks, int Hkv, int h,
                                                     const uint8_t* ks, const uint8_t* vs) {
  if (page >= end) return 0u;
  int id = table_row[page >> ppb_shift];
  if (id < 0 || id >= num_blocks) id = 0;
  const int64_t i = (int64_t)id * Hkv + h;
  return (uint32_t)ks[i] | ((uint32_t)vs[i] << 8);
}

// Zeroes rows [0, first) of a page in shared memory: V rows that no query sees
// meet weight 0, and must not turn that into NaN whatever they hold.
template <int D, int KV>
__device__ __forceinline__ void zero_page_head(uint8_t* page, int first, int lane) {
  using Geo = PageGeom<D, KV>;
  constexpr int CPR = Geo::ROW_BYTES / 16;
  for (int i = lane; i < first * CPR; i += 32) {
    const int r = i / CPR, x = (i % CPR) * 16;
    *reinterpret_cast<uint4*>(page + (x / Geo::BOX_ROW_BYTES) * Geo::BOX_BYTES +
                              r * Geo::BOX_ROW_BYTES + x % Geo::BOX_ROW_BYTES) =
        make_uint4(0u, 0u, 0u, 0u);
  }
}

// softcap * tanh(x / softcap), all in log2 units: with E = 2^(2 x / softcap),
// tanh = 1 - 2 / (E + 1). The subtraction loses at most 2^-23 of the cap, an
// error of some 1e-5 in a score at the caps in use; a large E gives 2 / inf = 0.
__device__ __forceinline__ float softcap_log2(float x, float cap_log2, float two_over_cap) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * two_over_cap));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e + 1.f));
  return fmaf(-2.f * cap_log2, r, cap_log2);
}

}  // namespace pkv
