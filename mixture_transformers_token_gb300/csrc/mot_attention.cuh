// What joint attention's forward and backward kernels share: the check of a sequence's descriptor (q_start, k_start, nq, nk,
// n_causal) and the arithmetic of a pair of scores.
#pragma once

#include <cstdint>

#include "mot.h"

namespace mot {
namespace attn {

// 2^x: CUDA's exp2f (the library's accurate function, with subnormal results; this code is
// built without fast-math options).
__device__ __forceinline__ float ex2(float x) { return exp2f(x); }

// Packed pairs of fp32 (Blackwell f32x2 arithmetic: two IEEE operations per instruction, each
// rounded as the scalar one would be).
__device__ __forceinline__ unsigned long long f2_pack(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_unpack(unsigned long long v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ unsigned long long f2_mul(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ unsigned long long f2_add(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ bool bad_seq(const int32_t* d, int T) {
  const int q0 = d[0], k0 = d[1], nq = d[2], nk = d[3], c = d[4];
  return q0 < 0 || k0 < 0 || nq < 0 || nk < 1 || c < 0 || c > nq || (c > 0 && nk < nq) ||
         int64_t(q0) + nq > T || int64_t(k0) + nk > T;
}

// Up to this many sequences a pack's work is put in the order of its weight; more are taken as they come.
constexpr int kSortedSeqs = 64;

}  // namespace attn
}  // namespace mot
