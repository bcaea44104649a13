// AdamW over many tensors in one launch, states in 32 or in 8 bits.
//
// Source: [RFC][BAGEL-7B-MoT][CUDA/ROCm] WS1/WS2 kernel roadmap and integration plan #435 (§3 BAGEL-specific rules: phase A
// updates the gen weight set). The update is the decoupled-weight-decay Adam of Loshchilov and Hutter (ICLR 2019); 8-bit
// states in blocks with a scale of their own are those of Dettmers et al. (ICLR 2022), here in e4m3 and rounded at random
// (Philox4x32 of Salmon, Moraes, Dror and Shaw, SC 2011): rounded to nearest, a second moment that changes by 1 - beta2
// a step would stay where it is, for its neighbours are 6 to 12 % away.
//
// Every element is read and written once: 30 bytes with fp32 states, fp32 gradients and the bf16 copy, 16.06 with 8-bit states
// and bf16 gradients. The bound is memory. fp32 states reach a plain copy's rate and more (985 us for 233 million elements, 30 bytes
// each). 8-bit ones take 73 instructions an element, so that a warp's loads have to come while others compute: 233 million
// elements in 599 us, 93% of the copy's rate, with the next block's lines asked for ahead and 32 warps an SM (without the
// first 701 us, with 24 warps 654, with neither 789 and more).

#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>

#include "mot.h"
#include "mot_device.cuh"
#include "mot_host.hpp"
#include "mot_kvcache.cuh"

namespace mot {
namespace adamw {

constexpr int THREADS = 256;
constexpr int BLOCK = MOT_ADAMW_BLOCK;
constexpr int WARPS = THREADS / 32;
constexpr int kMaxTensors = 128;  // of one launch: its table is part of the launch's parameters
constexpr int ROUNDS = 7;         // of Philox

struct Table {
  mot_adamw_tensor t[kMaxTensors];
  uint32_t first[kMaxTensors + 1];  // first CTA of each tensor
  int n;
  int base;                         // index of t[0] in the caller's array
  int blocks;                       // of 256 elements a warp
  const float* hyper;
  uint32_t key[2 * ROUNDS];         // of each round
  uint32_t* err;
};

// words of the step's row
enum { LR, B1, C1, B2, C2, LR1, R2, EPS, GS, STEP };

struct Hyper {
  float lr, b1, c1, b2, c2, lr1, r2, eps, gs;
  uint32_t step;
};

__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u; }

__device__ __forceinline__ bool load_hyper(const float* row, Hyper& h) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(row)), b = __ldg(reinterpret_cast<const float4*>(row) + 1),
               c = __ldg(reinterpret_cast<const float4*>(row) + 2);
  h = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, __float_as_uint(c.y)};
  return h.lr >= 0.0f && finite(h.lr) && h.b1 >= 0.0f && h.b1 < 1.0f && h.c1 > 0.0f && h.c1 <= 1.0f && h.b2 >= 0.0f &&
         h.b2 < 1.0f && h.c2 > 0.0f && h.c2 <= 1.0f && h.lr1 >= 0.0f && finite(h.lr1) && h.r2 >= 1.0f && finite(h.r2) &&
         h.eps > 0.0f && finite(h.eps) && finite(h.gs) && h.step >= 1u && h.step < 0x80000000u;
}

// Eight elements: m and v become the new moments, r the square roots of v, p the new weights. Products two at a time.
__device__ __forceinline__ void update(const Hyper& h, float wl, float (&g)[8], float (&m)[8], float (&v)[8], float (&r)[8],
                                       float (&p)[8]) {
  float a[8], b[8];
  mul_each(g, h.gs, g);
  mul_each(m, h.b1, m);
  mul_each(g, h.c1, a);
#pragma unroll
  for (int i = 0; i < 8; ++i) m[i] = __fadd_rn(m[i], a[i]);
  mul_each(v, h.b2, v);
  mul_each(g, g, a);
  mul_each(a, h.c2, a);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = __fadd_rn(v[i], a[i]);
    r[i] = __fsqrt_rn(v[i]);
  }
  mul_each(r, h.r2, a);
  mul_each(m, h.lr1, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = __fdiv_rn(b[i], __fadd_rn(a[i], h.eps));
  mul_each(p, wl, a);
#pragma unroll
  for (int i = 0; i < 8; ++i) p[i] = __fsub_rn(p[i], __fadd_rn(b[i], a[i]));
}

__device__ __forceinline__ void philox_round(uint32_t (&x)[4], uint32_t k0, uint32_t k1) {
  const uint64_t a = uint64_t(x[0]) * 0xD2511F53u, b = uint64_t(x[2]) * 0xCD9E8D57u;
  x[0] = uint32_t(b >> 32) ^ x[1] ^ k0;
  x[1] = uint32_t(b);
  x[2] = uint32_t(a >> 32) ^ x[3] ^ k1;
  x[3] = uint32_t(a);
}

// Philox4x32-7: the words of elements 4 b .. 4 b + 3.
__device__ __forceinline__ void random_words(uint32_t (&x)[4], uint64_t b, uint32_t tensor, uint32_t step,
                                             const uint32_t* key) {
  x[0] = uint32_t(b);
  x[1] = uint32_t(b >> 32);
  x[2] = tensor;
  x[3] = step;
#pragma unroll
  for (int i = 0; i < ROUNDS; ++i) philox_round(x, key[2 * i], key[2 * i + 1]);
}

// A block's quantiser from its largest magnitude's bits (whose order is the floats', infinities and NaNs last).
struct Scale {
  float scale, inv;
};
__device__ __forceinline__ Scale block_scale(uint32_t top) {
  const float a = __uint_as_float(top);
  if (top >= 0x7F800000u) return {__uint_as_float(0x7FC00000u), 0.0f};
  if (!(a >= 0x1p-100f)) return {0.0f, 0.0f};
  return {__fmul_rn(a, 1.0f / 448.0f), __fmul_rn(__frcp_rn(a), 448.0f)};
}

// y = x inv (at most 448 and a few units in magnitude) rounded to one of its e4m3 neighbours by 16 random bits below the last kept
// one; the sign bit stays, and what is a few units above 448 keeps 448's bits. FULL false: no magnitude is under 2^-6. FULL: those
// (e4m3's subnormals) move up by 2^-6, where fp32 values have the subnormals' step in the same bit.
template <bool FULL>
__device__ __forceinline__ float round_at_random(float y, uint32_t bits16) {
  if constexpr (FULL) {
    const float lift = fabsf(y) < 0x1p-6f ? 0x1p-6f : 0.0f;
    const uint32_t z = (__float_as_uint(__fadd_rn(fabsf(y), lift)) + (bits16 << 4)) & 0xFFF00000u;
    return copysignf(__fsub_rn(__uint_as_float(z), lift), y);
  } else {
    return __uint_as_float((__float_as_uint(y) + (bits16 << 4)) & 0xFFF00000u);
  }
}

// Elements [0, 8) of a lane, of which the first `have` are there (ALL: all of them).
template <bool ALL, bool BF16>
__device__ __forceinline__ void load_grad(const void* g, int64_t e, int have, float (&x)[8]) {
  if (ALL || have == 8) {
    if constexpr (BF16) {
      const uint4 w = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(g) + e));
      x[0] = bf_lo(w.x), x[1] = bf_hi(w.x), x[2] = bf_lo(w.y), x[3] = bf_hi(w.y);
      x[4] = bf_lo(w.z), x[5] = bf_hi(w.z), x[6] = bf_lo(w.w), x[7] = bf_hi(w.w);
    } else {
      const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(g) + e);
      const float4 a = __ldcs(s), b = __ldcs(s + 1);
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = i >= have ? 0.0f : BF16 ? bf_to_f(static_cast<const uint16_t*>(g)[e + i]) : static_cast<const float*>(g)[e + i];
  }
}

template <bool ALL>
__device__ __forceinline__ void load8(const float* s, int have, float (&x)[8]) {
  if (ALL || have == 8) {
    const float4 a = *reinterpret_cast<const float4*>(s), b = *(reinterpret_cast<const float4*>(s) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i < have ? s[i] : 0.0f;
  }
}

template <bool ALL>
__device__ __forceinline__ void store8(float* d, int have, const float (&x)[8]) {
  if (ALL || have == 8) {
    *reinterpret_cast<float4*>(d) = make_float4(x[0], x[1], x[2], x[3]);
    *(reinterpret_cast<float4*>(d) + 1) = make_float4(x[4], x[5], x[6], x[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < have) d[i] = x[i];
  }
}

template <bool ALL>
__device__ __forceinline__ void store_bf16(uint16_t* d, int have, const float (&x)[8]) {
  if (ALL || have == 8) {
    *reinterpret_cast<uint4*>(d) =
        make_uint4(cvt_bf2(x[0], x[1]), cvt_bf2(x[2], x[3]), cvt_bf2(x[4], x[5]), cvt_bf2(x[6], x[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < have) d[i] = f_to_bf(x[i]);
  }
}

template <bool ALL>
__device__ __forceinline__ void load_codes(const uint8_t* s, int have, float scale, float (&x)[8]) {
  uint32_t w[2] = {0u, 0u};
  if (ALL || have == 8) {
    const uint2 c = *reinterpret_cast<const uint2*>(s);
    w[0] = c.x, w[1] = c.y;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < have) w[i >> 2] |= uint32_t(s[i]) << (8 * (i & 3));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = kv::h2_to_f2(kv::e4m3x2_to_h2((w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu));
    x[2 * i] = v.x;
    x[2 * i + 1] = v.y;
  }
  mul_each(x, scale, x);
}

template <bool ALL>
__device__ __forceinline__ void store_codes(uint8_t* d, int have, uint32_t lo, uint32_t hi) {
  if (ALL || have == 8) {
    *reinterpret_cast<uint2*>(d) = make_uint2(lo, hi);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < have) d[i] = uint8_t((i < 4 ? lo : hi) >> (8 * (i & 3)));
  }
}

__device__ __forceinline__ uint32_t warp_max(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }

// The largest magnitude of eight values; a NaN if there is one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t top_of(const float (&x)[8]) {
  float a = fabsf(x[0]), b = fabsf(x[1]);
#pragma unroll
  for (int i = 2; i < 8; i += 2) a = max_nan(a, fabsf(x[i])), b = max_nan(b, fabsf(x[i + 1]));
  return __float_as_uint(max_nan(a, b));
}

// The codes of 8 values scaled to e4m3's range, by the low or the high halves of the elements' words. `keep` (sqrt(v)): values that
// are positive in v keep a code (a magnitude of at least 2^-6 has one anyway).
template <bool FULL, bool HIGH>
__device__ __forceinline__ void codes_of(const float (&y)[8], const uint32_t (&w)[2][4], bool keep, const float (&v)[8],
                                         uint32_t (&code)[2]) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    float z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[i] = round_at_random<FULL>(y[4 * q + i], HIGH ? w[q][i] >> 16 : w[q][i] & 0xFFFFu);
      if (FULL && keep && v[4 * q + i] > 0.0f) z[i] = fmaxf(z[i], 0x1p-9f);
    }
    code[q] = kv::e4m3x2(z[0], z[1]) | (kv::e4m3x2(z[2], z[3]) << 16);
  }
}

// A warp takes a block of 256 elements, eight consecutive ones a lane: the block's scales need no shared memory.
template <bool ALL, bool BF16, bool E4M3>
__device__ __forceinline__ void warp_block(const Table& a, const Hyper& h, const mot_adamw_tensor& t, float wl, int id,
                                           int64_t block, int lane) {
  const int64_t e = block * BLOCK + lane * 8;
  int have = 8;
  if constexpr (!ALL) {
    const int64_t left = t.n - e;
    have = left >= 8 ? 8 : left > 0 ? int(left) : 0;
  }
  float g[8], m[8], v[8], r[8], p[8];
  load_grad<ALL, BF16>(t.g, e, have, g);
  load8<ALL>(t.p + e, have, p);
  if constexpr (E4M3) {
    const float2 s = *reinterpret_cast<const float2*>(t.scales + 2 * block);
    load_codes<ALL>(static_cast<const uint8_t*>(t.m) + e, have, s.x, m);
    load_codes<ALL>(static_cast<const uint8_t*>(t.v) + e, have, s.y, v);
    mul_each(v, v, v);
  } else {
    load8<ALL>(static_cast<const float*>(t.m) + e, have, m);
    load8<ALL>(static_cast<const float*>(t.v) + e, have, v);
  }
  update(h, wl, g, m, v, r, p);
  store8<ALL>(t.p + e, have, p);
  if (t.p16) store_bf16<ALL>(t.p16 + e, have, p);
  if constexpr (E4M3) {
    uint32_t w[2][4], cm[2], cr[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) random_words(w[q], uint64_t(e) / 4 + q, uint32_t(id), h.step, a.key);
    // elements past the end are zero
    const Scale sm = block_scale(warp_max(top_of(m))), sr = block_scale(warp_max(top_of(r)));
    mul_each(m, sm.inv, m);
    mul_each(r, sr.inv, r);
    float least = fminf(fabsf(m[0]), r[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) least = fminf(least, fminf(fabsf(m[i]), r[i]));
    // few blocks reach 2^-15 below their largest value (`least` is a number also where one state's values are all NaN)
    if (__all_sync(0xffffffffu, least >= 0x1p-6f && sm.scale < INFINITY && sr.scale < INFINITY)) {
      codes_of<false, false>(m, w, false, v, cm);
      codes_of<false, true>(r, w, false, v, cr);
    } else {
      codes_of<true, false>(m, w, false, v, cm);
      codes_of<true, true>(r, w, sr.scale > 0.0f, v, cr);
      if (!(sm.scale > 0.0f)) cm[0] = cm[1] = 0u;  // a NaN, or zero, where negative values have become -0
      if (!(sr.scale > 0.0f)) cr[0] = cr[1] = 0u;
    }
    store_codes<ALL>(static_cast<uint8_t*>(t.m) + e, have, cm[0], cm[1]);
    store_codes<ALL>(static_cast<uint8_t*>(t.v) + e, have, cr[0], cr[1]);
    if (lane == 0) *reinterpret_cast<float2*>(t.scales + 2 * block) = make_float2(sm.scale, sr.scale);
  } else {
    store8<ALL>(static_cast<float*>(t.m) + e, have, m);
    store8<ALL>(static_cast<float*>(t.v) + e, have, v);
  }
}

// The lines of a whole block with 8-bit states into L2, one a lane.
template <bool BF16>
__device__ __forceinline__ void prefetch_block(const mot_adamw_tensor& t, int64_t block, int lane) {
  constexpr int G = BF16 ? 4 : 8;  // lines of the gradient
  const int64_t e = block * BLOCK;
  const uint8_t* at = nullptr;
  if (lane < 8) at = reinterpret_cast<const uint8_t*>(t.p + e) + 128 * lane;
  else if (lane < 8 + G) at = static_cast<const uint8_t*>(t.g) + e * (BF16 ? 2 : 4) + 128 * (lane - 8);
  else if (lane < 10 + G) at = static_cast<const uint8_t*>(t.m) + e + 128 * (lane - 8 - G);
  else if (lane < 12 + G) at = static_cast<const uint8_t*>(t.v) + e + 128 * (lane - 10 - G);
  if (at != nullptr) asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
}

template <bool BF16, bool E4M3>
__device__ __forceinline__ void warp_blocks(const Table& a, const Hyper& h, const mot_adamw_tensor& t, int id, int64_t block,
                                            int lane) {
  const float wl = __fmul_rn(h.lr, t.weight_decay);
#pragma unroll 1
  for (int i = 0; i < a.blocks; ++i, block += WARPS) {
    if ((block + 1) * BLOCK <= t.n) {
      if (E4M3 && i + 1 < a.blocks && (block + WARPS + 1) * BLOCK <= t.n) prefetch_block<BF16>(t, block + WARPS, lane);
      warp_block<true, BF16, E4M3>(a, h, t, wl, id, block, lane);
    } else {
      if (block * BLOCK < t.n) warp_block<false, BF16, E4M3>(a, h, t, wl, id, block, lane);
      break;
    }
  }
}

// E4M3 false: no tensor has 8-bit states.
template <bool E4M3>
__global__ void __launch_bounds__(THREADS, 4) adamw_kernel(const __grid_constant__ Table a) {
  Hyper h;
  if (!load_hyper(a.hyper, h)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.err, MOT_DEV_BAD_HYPER);
    return;
  }
  int lo = 0, hi = a.n;  // the tensor of this CTA
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.first[mid] <= blockIdx.x) lo = mid;
    else hi = mid;
  }
  const mot_adamw_tensor& t = a.t[lo];
  const int64_t block = int64_t(blockIdx.x - a.first[lo]) * (WARPS * a.blocks) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, id = a.base + lo;
  const bool bf16 = (t.flags & MOT_ADAMW_GRAD_BF16) != 0;
  if (E4M3 && (t.flags & MOT_ADAMW_STATE_E4M3) != 0) {
    if (bf16) warp_blocks<true, E4M3>(a, h, t, id, block, lane);
    else warp_blocks<false, E4M3>(a, h, t, id, block, lane);
  } else {
    if (bf16) warp_blocks<true, false>(a, h, t, id, block, lane);
    else warp_blocks<false, false>(a, h, t, id, block, lane);
  }
}

inline bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

// check_ptr for many pointers that lie in few allocations: an allocation that a pointer was found in vouches for the next ones.
// (560 pointers of 112 tensors, one by one, took 45 us of the host's time.)
class Allocations {
 public:
  explicit Allocations(int dev) : dev_(dev) {}
  int check(const void* p) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    for (int i = 0; i < n_; ++i)
      if (at - from_[i] < size_[i]) return MOT_OK;
    const int st = check_ptr(p, dev_);
    if (st != MOT_OK) return st;
    static std::atomic<void*> fn{nullptr};
    auto range = driver_fn<CUresult (*)(CUdeviceptr*, size_t*, CUdeviceptr)>("cuMemGetAddressRange", 3020, fn);
    CUdeviceptr from = 0;
    size_t size = 0;
    if (range != nullptr && range(&from, &size, CUdeviceptr(at)) == CUDA_SUCCESS) {
      const int i = n_ < kMax ? n_++ : next_++ % kMax;
      from_[i] = uintptr_t(from);
      size_[i] = size;
    }
    return MOT_OK;
  }

 private:
  static constexpr int kMax = 8;
  int dev_, n_ = 0, next_ = 0;
  uintptr_t from_[kMax];
  size_t size_[kMax];
};

}  // namespace adamw
}  // namespace mot

using namespace mot;

extern "C" int mot_adamw_hyper_host(double lr, double beta1, double beta2, double eps, double grad_scale, int64_t step,
                                    float* host_row) {
  if (!host_row) return MOT_ERR_NULL;
  if (!std::isfinite(lr) || !(lr >= 0) || !(beta1 >= 0) || !(beta1 < 1) || !(beta2 >= 0) || !(beta2 < 1) ||
      !std::isfinite(eps) || !std::isfinite(grad_scale) || step < 1 || step >= (int64_t(1) << 31))
    return MOT_ERR_ARG;
  const double t = double(step);
  float row[MOT_ADAMW_HYPER_WORDS] = {};
  row[adamw::LR] = float(lr);
  row[adamw::B1] = float(beta1);
  row[adamw::C1] = float(1 - beta1);
  row[adamw::B2] = float(beta2);
  row[adamw::C2] = float(1 - beta2);
  row[adamw::LR1] = float(lr / (1 - std::pow(beta1, t)));
  row[adamw::R2] = float(1 / std::sqrt(1 - std::pow(beta2, t)));
  row[adamw::EPS] = float(eps);
  row[adamw::GS] = float(grad_scale);
  // what rounds out of range in fp32 is refused like what is out of range itself
  if (!(row[adamw::EPS] > 0) || row[adamw::B1] >= 1 || row[adamw::B2] >= 1 || !std::isfinite(row[adamw::LR]) ||
      !std::isfinite(row[adamw::LR1]) || !std::isfinite(row[adamw::EPS]) || !std::isfinite(row[adamw::GS]))
    return MOT_ERR_ARG;
  const uint32_t word = uint32_t(step);
  static_assert(sizeof(row) == 4 * MOT_ADAMW_HYPER_WORDS, "a row of 32-bit words");
  __builtin_memcpy(&row[adamw::STEP], &word, 4);
  __builtin_memcpy(host_row, row, sizeof(row));
  return MOT_OK;
}

extern "C" int mot_adamw_step(const mot_adamw_tensor* tensors, int n_tensors, const float* hyper, uint64_t seed, void* ws,
                              size_t ws_bytes, void* stream) {
  if (!tensors || !hyper || !ws) return MOT_ERR_NULL;
  if (n_tensors < 1 || n_tensors > 65536) return MOT_ERR_GEOMETRY;
  for (int i = 0; i < n_tensors; ++i) {
    const mot_adamw_tensor& t = tensors[i];
    const bool e4m3 = (t.flags & MOT_ADAMW_STATE_E4M3) != 0;
    if (!t.p || !t.g || !t.m || !t.v || (e4m3 && !t.scales)) return MOT_ERR_NULL;
    if (t.n < 1 || t.n > (int64_t(1) << 40)) return MOT_ERR_GEOMETRY;
    if ((t.flags & ~(MOT_ADAMW_GRAD_BF16 | MOT_ADAMW_STATE_E4M3)) != 0 || !(t.weight_decay >= 0.0f) ||
        !(t.weight_decay <= 3.4e38f))
      return MOT_ERR_ARG;
    if (!aligned16(t.p) || !aligned16(t.p16) || !aligned16(t.g) || !aligned16(t.m) || !aligned16(t.v) ||
        (e4m3 && !adamw::aligned8(t.scales)))
      return MOT_ERR_ALIGN;
  }
  if (!aligned16(hyper) || !aligned16(ws)) return MOT_ERR_ALIGN;
  if (ws_bytes < sizeof(PlanHeader)) return MOT_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const void* ptrs[] = {hyper, ws};
  int dev = -1;
  int st = check_device(s, ptrs, 2, &dev);
  if (st != MOT_OK) return st;
  DeviceGuard guard(dev);
  adamw::Allocations known(dev);
  int64_t all = 0;  // blocks
  bool e4m3 = false;
  for (int i = 0; i < n_tensors; ++i) {
    const mot_adamw_tensor& t = tensors[i];
    const void* mine[] = {t.p, t.p16, t.g, t.m, t.v, (t.flags & MOT_ADAMW_STATE_E4M3) ? t.scales : nullptr};
    for (const void* p : mine)
      if (p != nullptr && (st = known.check(p)) != MOT_OK) return st;
    all += (t.n + adamw::BLOCK - 1) / adamw::BLOCK;
    e4m3 |= (t.flags & MOT_ADAMW_STATE_E4M3) != 0;
  }
  adamw::Table a;
  a.hyper = hyper;
  uint32_t k0 = uint32_t(seed), k1 = uint32_t(seed >> 32);
  for (int i = 0; i < adamw::ROUNDS; ++i, k0 += 0x9E3779B9u, k1 += 0xBB67AE85u) a.key[2 * i] = k0, a.key[2 * i + 1] = k1;
  // With 8-bit states a warp takes several blocks, whose lines come ahead but for the first's, and its setting up (the step's numbers,
  // its tensor) costs about an eighth of a block: up to 16 a warp, as long as every SM has eight CTAs (4 a warp 706 us for 656, 32
  // a warp 666). fp32 states, bound by memory, lose by it: 1019 us for 987.
  const int64_t waves = all / (int64_t(sm_count(dev)) * 8 * adamw::WARPS);
  a.blocks = e4m3 && waves > 1 ? int(waves < 16 ? waves : 16) : 1;
  const int64_t per = int64_t(a.blocks) * adamw::WARPS * adamw::BLOCK;
  a.err = &static_cast<PlanHeader*>(ws)->error;
  for (int i = 0; i < n_tensors;) {
    a.n = 0;
    a.base = i;
    int64_t ctas = 0;
    for (; i < n_tensors && a.n < adamw::kMaxTensors; ++i) {
      const int64_t mine = (tensors[i].n + per - 1) / per;
      if (ctas + mine > (int64_t(1) << 31) - 1) break;  // one tensor has at most 2^29
      a.t[a.n] = tensors[i];
      a.first[a.n++] = uint32_t(ctas);
      ctas += mine;
    }
    a.first[a.n] = uint32_t(ctas);
    if (e4m3) adamw::adamw_kernel<true><<<unsigned(ctas), adamw::THREADS, 0, s>>>(a);
    else adamw::adamw_kernel<false><<<unsigned(ctas), adamw::THREADS, 0, s>>>(a);
    if (cudaGetLastError() != cudaSuccess) return MOT_ERR_CUDA;
  }
  return MOT_OK;
}
