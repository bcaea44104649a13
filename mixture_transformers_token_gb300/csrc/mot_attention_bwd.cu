// Gradient of joint attention with respect to its fused QKV rows.
//
// Sources: [RFC][BAGEL-7B-MoT][CUDA/ROCm] WS1/WS2 kernel roadmap and integration plan #435 (§1 Motivation item 2, §2 Reference
// hazards: the masks, as in the forward; §3 BAGEL-specific rules: dX passes through the frozen und operators; §3 Numerical
// contract: fixed accumulation order, no atomics).
//
// Per query i and visible key j: P = 2^((S - lse / scale) c) with c = scale log2 e, dP = dout_i . v_j, delta_i = dout_i . out_i,
// dS = P (dP - delta_i); dq_i = scale sum_j dS k_j, dk_j = scale sum_i dS q_i, dv_j = sum_i P dout_i.
//
// One warp per query row and head (dq) and per key row and KV head (dk, dv), in fp32: the plain kernels.

#include <cuda_runtime.h>

#include "mot.h"
#include "mot_device.cuh"
#include "mot_host.hpp"

namespace mot {
namespace attnb {

constexpr int WARPS = 8, THREADS = 32 * WARPS;

struct Args {
  const uint16_t* dout;
  const uint16_t* qkv;
  const uint16_t* out;
  const float* lse;
  const int32_t* seqs;
  int n_seq, T, Hq, Hkv;
  float c, scale, rscale;
  float* delta;  // [Hq][T]
  uint16_t* dqkv;
  uint32_t* err;
};

__device__ __forceinline__ bool bad_seq(const int32_t* d, int T) {
  const int q0 = d[0], k0 = d[1], nq = d[2], nk = d[3], c = d[4];
  return q0 < 0 || k0 < 0 || nq < 0 || nk < 1 || c < 0 || c > nq || (c > 0 && nk < nq) ||
         int64_t(q0) + nq > T || int64_t(k0) + nk > T;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}

// A lane's D / 32 values of a head, or their dot product with another row's.
template <int D>
__device__ __forceinline__ void load(const uint16_t* p, int lane, float (&x)[D / 32]) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i) x[i] = bf_to_f(p[lane + 32 * i]);
}
template <int D>
__device__ __forceinline__ float dot(const float (&a)[D / 32], const float (&b)[D / 32]) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) s = __fadd_rn(s, __fmul_rn(a[i], b[i]));
  return warp_sum(s);
}
template <int D>
__device__ __forceinline__ void add(float (&s)[D / 32], float f, const float (&x)[D / 32]) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i) s[i] = __fadd_rn(s[i], __fmul_rn(f, x[i]));
}
template <int D>
__device__ __forceinline__ void store(uint16_t* p, int lane, float f, const float (&x)[D / 32]) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i) p[lane + 32 * i] = f_to_bf(__fmul_rn(f, x[i]));
}

template <int D>
__global__ void __launch_bounds__(THREADS) dq_kernel(const Args a) {
  const int lane = threadIdx.x & 31;
  const int64_t item = int64_t(blockIdx.x) * WARPS + (threadIdx.x >> 5);
  if (item >= int64_t(a.T) * a.Hq) return;
  const int row = int(item / a.Hq), h = int(item % a.Hq), g = h / (a.Hq / a.Hkv);
  const int64_t N = int64_t(a.Hq + 2 * a.Hkv) * D;
  for (int s = 0; s < a.n_seq; ++s) {
    const int32_t* d = a.seqs + 5 * s;
    if (bad_seq(d, a.T)) {
      if (item == 0 && lane == 0) atomicOr(a.err, MOT_DEV_BAD_SEQUENCE);
      continue;
    }
    const int i = row - d[0];
    if (i < 0 || i >= d[2]) continue;
    float q[D / 32], dy[D / 32], o[D / 32], sum[D / 32] = {};
    load<D>(a.qkv + row * N + h * D, lane, q);
    load<D>(a.dout + (int64_t(row) * a.Hq + h) * D, lane, dy);
    load<D>(a.out + (int64_t(row) * a.Hq + h) * D, lane, o);
    const float delta = dot<D>(dy, o);
    if (lane == 0) a.delta[int64_t(h) * a.T + row] = delta;
    const float l = __fmul_rn(a.lse[int64_t(h) * a.T + row], a.rscale);
    const int lim = i < d[4] ? d[3] - d[2] + i + 1 : d[3];
    for (int j = 0; j < lim; ++j) {
      float k[D / 32], v[D / 32];
      load<D>(a.qkv + int64_t(d[1] + j) * N + (a.Hq + g) * D, lane, k);
      load<D>(a.qkv + int64_t(d[1] + j) * N + (a.Hq + a.Hkv + g) * D, lane, v);
      const float p = exp2f(__fmul_rn(__fsub_rn(dot<D>(q, k), l), a.c));
      add<D>(sum, __fmul_rn(p, __fsub_rn(dot<D>(dy, v), delta)), k);
    }
    store<D>(a.dqkv + row * N + h * D, lane, a.scale, sum);
  }
}

template <int D>
__global__ void __launch_bounds__(THREADS) dkv_kernel(const Args a) {
  const int lane = threadIdx.x & 31;
  const int64_t item = int64_t(blockIdx.x) * WARPS + (threadIdx.x >> 5);
  if (item >= int64_t(a.T) * a.Hkv) return;
  const int row = int(item / a.Hkv), g = int(item % a.Hkv), G = a.Hq / a.Hkv;
  const int64_t N = int64_t(a.Hq + 2 * a.Hkv) * D;
  float k[D / 32], v[D / 32], dk[D / 32] = {}, dv[D / 32] = {};
  load<D>(a.qkv + row * N + (a.Hq + g) * D, lane, k);
  load<D>(a.qkv + row * N + (a.Hq + a.Hkv + g) * D, lane, v);
  bool key = false;
  for (int s = 0; s < a.n_seq; ++s) {
    const int32_t* d = a.seqs + 5 * s;
    if (bad_seq(d, a.T)) continue;
    const int j = row - d[1];
    if (j < 0 || j >= d[3]) continue;
    key = true;
    for (int h = g * G; h < (g + 1) * G; ++h)
      for (int i = 0; i < d[2]; ++i) {
        if (i < d[4] && j > d[3] - d[2] + i) continue;
        const int64_t r = d[0] + i;
        float q[D / 32], dy[D / 32];
        load<D>(a.qkv + r * N + h * D, lane, q);
        load<D>(a.dout + (r * a.Hq + h) * D, lane, dy);
        const float l = __fmul_rn(a.lse[int64_t(h) * a.T + r], a.rscale);
        const float p = exp2f(__fmul_rn(__fsub_rn(dot<D>(q, k), l), a.c));
        add<D>(dv, p, dy);
        add<D>(dk, __fmul_rn(p, __fsub_rn(dot<D>(dy, v), a.delta[int64_t(h) * a.T + r])), q);
      }
  }
  if (!key) return;
  store<D>(a.dqkv + row * N + (a.Hq + g) * D, lane, a.scale, dk);
  store<D>(a.dqkv + row * N + (a.Hq + a.Hkv + g) * D, lane, 1.0f, dv);
}

inline bool shape_ok(int64_t T, int Hq, int Hkv, int D, int n_seq) {
  return T >= 1 && T <= MOT_MAX_TOKENS && (D == 64 || D == 128) && Hq >= 1 && Hkv >= 1 && Hq <= 1024 && Hkv <= 1024 &&
         Hq % Hkv == 0 && n_seq >= 1 && n_seq <= MOT_MAX_TOKENS;
}

}  // namespace attnb
}  // namespace mot

using namespace mot;

extern "C" size_t mot_joint_attention_backward_workspace_bytes(int64_t T, int Hq, int Hkv, int D, int n_seq) {
  if (!attnb::shape_ok(T, Hq, Hkv, D, n_seq)) return 0;
  return sizeof(PlanHeader) + (size_t(T) * Hq * sizeof(float) + 15) / 16 * 16;
}

extern "C" int mot_joint_attention_backward(const mot_bf16* dout, const mot_bf16* qkv, const mot_bf16* out,
                                            const float* lse, int64_t T, int Hq, int Hkv, int D, const int32_t* seqs,
                                            int n_seq, float scale, void* ws, size_t ws_bytes, mot_bf16* dqkv,
                                            void* stream) {
  if (!dout || !qkv || !out || !lse || !seqs || !ws || !dqkv) return MOT_ERR_NULL;
  if (!attnb::shape_ok(T, Hq, Hkv, D, n_seq)) return MOT_ERR_GEOMETRY;
  const float c = scale * 1.4426950408889634f;
  if (!(c >= 0x1p-100f) || !(c <= 0x1p100f)) return MOT_ERR_ARG;
  if (!aligned16(dout) || !aligned16(qkv) || !aligned16(out) || !aligned16(lse) || !aligned16(seqs) || !aligned16(ws) ||
      !aligned16(dqkv))
    return MOT_ERR_ALIGN;
  if (ws_bytes < mot_joint_attention_backward_workspace_bytes(T, Hq, Hkv, D, n_seq)) return MOT_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const void* ptrs[] = {dout, qkv, out, lse, seqs, ws, dqkv};
  int dev = -1;
  const int st = check_device(s, ptrs, 7, &dev);
  if (st != MOT_OK) return st;
  DeviceGuard guard(dev);
  attnb::Args a{};
  a.dout = dout;
  a.qkv = qkv;
  a.out = out;
  a.lse = lse;
  a.seqs = seqs;
  a.n_seq = n_seq;
  a.T = int(T);
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.c = c;
  a.scale = scale;
  a.rscale = 1.0f / scale;
  a.delta = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + sizeof(PlanHeader));
  a.dqkv = dqkv;
  a.err = &static_cast<PlanHeader*>(ws)->error;
  const int64_t nq = (T * Hq + attnb::WARPS - 1) / attnb::WARPS, nkv = (T * Hkv + attnb::WARPS - 1) / attnb::WARPS;
  if (nq > (int64_t(1) << 31) - 1) return MOT_ERR_GEOMETRY;
  if (D == 64) {
    attnb::dq_kernel<64><<<unsigned(nq), attnb::THREADS, 0, s>>>(a);
    attnb::dkv_kernel<64><<<unsigned(nkv), attnb::THREADS, 0, s>>>(a);
  } else {
    attnb::dq_kernel<128><<<unsigned(nq), attnb::THREADS, 0, s>>>(a);
    attnb::dkv_kernel<128><<<unsigned(nkv), attnb::THREADS, 0, s>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? MOT_OK : MOT_ERR_CUDA;
}
