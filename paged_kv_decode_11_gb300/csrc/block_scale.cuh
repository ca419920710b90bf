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
#include "f32x2.cuh"

namespace pkv {

constexpr int kE8M0Bias = 127;
constexpr int kBlockMinExp = -60;       // smallest exponent the append gives a block

// The _ext attentions put a weight's reference this far (log2) below the largest
// score: the weights that are rounded to 16 bits start at 2^7 and may grow to 2^15
// before the reference moves, and f16 holds those down to 2^-21 of the largest in full
// precision (2^-14 with a reference at the maximum). That shows where the largest
// weights meet zeros in V.
constexpr float kWeightHeadLog2 = 7.f;

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

// Up to this cap the error of the first form below, 3e-5 at most, is no more than the
// products behind a score have.
constexpr float kCoarseCap = 128.f;

// softcap * tanh(x / softcap), all in log2 units, in two forms (inv = 1 / cap_log2).
// With E = 2^(2 x / softcap), tanh = 1 - 2 / (E + 1): right to some 2^-23 of the cap,
// which is little beside a score near the cap (a large E gives 2 / inf = 0) and much
// beside a small one.
__device__ __forceinline__ float softcap_log2(float x, float cap_log2, float two_over_cap) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * two_over_cap));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e + 1.f));
  return fmaf(-2.f * cap_log2, r, cap_log2);
}

// Inside (-softcap, softcap), where scores seldom leave, tanh(y) = y P(y^2) with P of
// degree 6 is off by less than 2e-7 of itself (the Chebyshev interpolant of
// tanh(sqrt t) / sqrt t on [0, 1], evaluated in fp32): five packed operations a score,
// where the other form takes two of the special-function unit's, which the softmax
// keeps busy.
__device__ __forceinline__ float2 softcap_log2_inside(float a, float b, float inv) {
  constexpr float kP[7] = {0.99999994f, -0.33332857f, 0.13325398f, -0.053465176f,
                           0.02030552f, -0.0062170699f, 0.0010455536f};
  const f2 v = pack_f2(a, b);
  const f2 y = mul2(v, pack_f2(inv, inv)), t = mul2(y, y);
  f2 h = pack_f2(kP[6], kP[6]);
#pragma unroll
  for (int k = 5; k >= 0; --k) h = fma2(h, t, pack_f2(kP[k], kP[k]));
  return unpack_f2(mul2(v, h));
}

// Two scores, each in its own form.
__device__ __forceinline__ void softcap_log2_pair(float& a, float& b, float cap_log2,
                                                  float two_over_cap) {
  const float inv = two_over_cap * (0.5f * kLn2);
  const float2 r = softcap_log2_inside(a, b, inv);
  const bool in_a = fabsf(a) * inv <= 1.f, in_b = fabsf(b) * inv <= 1.f;
  if (!(in_a && in_b)) {
    a = in_a ? r.x : softcap_log2(a, cap_log2, two_over_cap);
    b = in_b ? r.y : softcap_log2(b, cap_log2, two_over_cap);
  } else {
    a = r.x;
    b = r.y;
  }
}

// N scores, each in its own form. Out of line and in local memory: beside the loop that
// calls it, code that hardly ever runs costs what it displaces (inline 111.6 us on the
// capped window, so 107.8, without it 106.8).
template <int N>
__device__ __noinline__ void softcap_log2_each(float* x, float cap_log2, float two_over_cap) {
  for (int c = 0; c < N; c += 2) {
    float a = x[c], b = x[c + 1];
    softcap_log2_pair(a, b, cap_log2, two_over_cap);
    x[c] = a;
    x[c + 1] = b;
  }
}

// The N scores of a thread's row, of which it sees first..last; the others (left-over
// bytes, maybe) become 0. The row takes one form for all of them, the first where one is
// beyond a cap of up to kCoarseCap. Beyond a larger cap each takes its own: a score below
// -cap weighs nothing, and the others may be small beside 2^-23 of the cap. The choice is
// the row's own, so that its bits depend neither on keys it does not see nor on the
// warp's other rows (the warp choosing for all of its rows, unseen keys included, took
// 103 us on the capped window where a choice by row takes 107).
template <int N>
__device__ __forceinline__ void softcap_log2_row(float (&x)[N], int first, int last,
                                                 float cap_log2, float two_over_cap) {
  const float inv = two_over_cap * (0.5f * kLn2);
  if (first > 0 || last < N - 1) {
    const unsigned span = (unsigned)(last - first);
#pragma unroll
    for (int c = 0; c < N; ++c)
      if ((unsigned)(c - first) > span) x[c] = 0.f;
  }
  float far = 0.f;
#pragma unroll
  for (int c = 0; c < N; ++c) far = fmaxf(far, fabsf(x[c]));
  if (far * inv <= 1.f) {
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      const float2 r = softcap_log2_inside(x[c], x[c + 1], inv);
      x[c] = r.x;
      x[c + 1] = r.y;
    }
  } else {
    if (__builtin_expect(cap_log2 > kCoarseCap / kLn2, 0)) {
      float t[N];
#pragma unroll
      for (int c = 0; c < N; ++c) t[c] = x[c];
      softcap_log2_each<N>(t, cap_log2, two_over_cap);
#pragma unroll
      for (int c = 0; c < N; ++c) x[c] = t[c];
      return;
    }
#pragma unroll
    for (int c = 0; c < N; ++c) x[c] = softcap_log2(x[c], cap_log2, two_over_cap);
  }
}

}  // namespace pkv
