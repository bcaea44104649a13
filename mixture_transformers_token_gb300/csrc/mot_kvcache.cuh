// The paged key-value cache: its layout, the e4m3 form of a vector and the argument checks that its
// entry points share.
//
// K and V pages are [n_pages][Hkv][page][D] in bf16 or e4m3, so the keys of one head in one page are
// consecutive rows. An e4m3 cache has the fp32 scales [n_pages][Hkv][page][2] (K's and V's of a token
// and head side by side: 16 tokens' scales are 128 consecutive bytes). Slot s is token s % page of
// page s / page.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "mot.h"
#include "mot_device.cuh"
#include "mot_host.hpp"

namespace mot {
namespace kv {

constexpr int kMaxPage = 1024;  // tokens of a page, a multiple of 16

// Two floats to two e4m3 codes (the first in the low byte), rounded to nearest even. The callers'
// values are at most 448 in magnitude, or NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two e4m3 codes to two halves: exact, every e4m3 value is a half.
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(codes)));
  return r;
}

__device__ __forceinline__ float2 h2_to_f2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The scale of a vector whose largest magnitude is `a`: 2^e with the smallest e >= -64 that has
// a <= 448 2^e (448 = 1.75 2^8, e4m3's largest value), NaN if a is not finite. A power of two makes
// the division by the scale exact, and costs no accuracy: e4m3's relative step does not depend on
// the scale. The bound -64 keeps 1 / scale finite and sums of it in range; a vector below 2^-55
// loses its low bits to e4m3's subnormals, or becomes zero.
constexpr int kMinScaleExp = -64;

__device__ __forceinline__ float e4m3_scale(float a) {
  const uint32_t b = __float_as_uint(a);
  const int k = int(b >> 23) - 127;  // a = f 2^k with f in [1, 2) (subnormal a: k = -127, below the bound)
  if (k == 128) return __uint_as_float(0x7FC00000u);
  int e = (b & 0x007FFFFFu) <= 0x00600000u ? k - 8 : k - 7;  // f <= 1.75
  e = e < kMinScaleExp ? kMinScaleExp : e;
  return __uint_as_float(uint32_t(e + 127) << 23);
}

// 1 / scale for a scale that e4m3_scale made: 2^-e by its bits (NaN for NaN).
__device__ __forceinline__ float inverse_scale(float scale) {
  const uint32_t b = __float_as_uint(scale);
  return b >= 0x7F800000u ? scale : __uint_as_float(0x7F000000u - b);
}

// Division by a number known to the host. m = floor(2^32 / d) makes the high half of n m either the
// quotient or one less, for every n < 2^32.
struct Div {
  uint32_t d, m;
  Div() = default;
  explicit Div(uint32_t by) : d(by), m(uint32_t((uint64_t(1) << 32) / by - (by == 1 ? 1 : 0))) {}
  __device__ __forceinline__ uint32_t of(uint32_t n) const {
    const uint32_t q = __umulhi(n, m);
    return n - q * d >= d ? q + 1 : q;
  }
};

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Checks of the cache's shape that need no CUDA call.
inline int check_shape(int Hq, int Hkv, int D, int kv_type, int64_t n_pages, int page) {
  if (kv_type != MOT_KV_BF16 && kv_type != MOT_KV_E4M3) return MOT_ERR_ARG;
  if (D != 64 && D != 128) return MOT_ERR_GEOMETRY;
  if (Hq < 1 || Hkv < 1 || Hq > 1024 || Hkv > 1024 || Hq % Hkv != 0) return MOT_ERR_GEOMETRY;
  if (page < 16 || page > kMaxPage || page % 16 != 0) return MOT_ERR_GEOMETRY;
  // rows of the cache are addressed by 32-bit TMA coordinates
  if (n_pages < 1 || n_pages > ((int64_t(1) << 31) - 1) / (int64_t(Hkv) * page)) return MOT_ERR_GEOMETRY;
  return MOT_OK;
}

}  // namespace kv
}  // namespace mot
