// Gradient through the QKV projection's epilogue: the RoPE rotation and the per-head RMSNorm of Q and K.
//
// Sources: [RFC][BAGEL-7B-MoT][CUDA/ROCm] WS1/WS2 kernel roadmap and integration plan #435 (§2 Reference hazards: QK norm in
// FP32, RoPE; §3 BAGEL-specific rules: the frozen und operators still need dX); [WS1][CUDA][Qwen3-Next] MoE route/combine
// contract ... #503 (gated-norm commit: the backward from deterministic pieces).
//
// Per head of D values, with h = D / 2 and (c, s) the table's entry of the row's position:
//   forward   xh = x rstd, u = xh w, out_i = u_i c - u_{i+h} s, out_{i+h} = u_{i+h} c + u_i s
//   backward  du_i = d_i c + d_{i+h} s, du_{i+h} = d_{i+h} c - d_i s, g = du w,
//             dx = rstd (g - xh (sum g xh) / D), dw += du xh
// in fp32, each operation rounded on its own, the forward's casts differentiated as the identity.
//
// A row is read and written once: 2 N + (Hq + Hkv) D values of bf16, its position and its table entries (16.5 us for 4096 rows
// of 28/4 heads of 128 at the measured copy rate): the bound is memory. D / 16 lanes hold a head, each 8 values and their 8
// partners, so that the rotation needs no exchange and a warp has four 16-byte loads a lane in flight.
//
// The weights' gradients: each CTA takes a run of the plan's positions, so that its rows are of one weight set, but for the run
// that holds the border; a lane adds its columns over the warp's rows, the warps' sums are added in order, and a second kernel
// adds the CTAs' sums in order.

#include <cuda_runtime.h>

#include <type_traits>

#include "mot.h"
#include "mot_device.cuh"
#include "mot_host.hpp"

namespace mot {
namespace qkvb {

constexpr int WARPS = 8, THREADS = 32 * WARPS;
constexpr int kMaxCtas = 608;  // runs of positions: four for each of 152 SMs

struct Args {
  const uint16_t* d;
  const uint16_t* x;
  const uint16_t* w[2];  // q's and k's, [2][D]
  const int32_t* pos;
  const void* cs;
  int P, T, Hq, Hkv;
  float eps;
  const uint8_t* ws;
  uint32_t* err;
  uint16_t* dx;
  float* part;  // [CTAs][2 kinds][2 sets][D], or null
  float* dw;    // [2][2][D]
  int sets;
  int ctas;
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  x[0] = bf_lo(v.x), x[1] = bf_hi(v.x), x[2] = bf_lo(v.y), x[3] = bf_hi(v.y);
  x[4] = bf_lo(v.z), x[5] = bf_hi(v.z), x[6] = bf_lo(v.w), x[7] = bf_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(cvt_bf2(x[0], x[1]), cvt_bf2(x[2], x[3]), cvt_bf2(x[4], x[5]), cvt_bf2(x[6], x[7]));
}

// cos and sin of the lane's 8 pairs
template <bool F32>
__device__ __forceinline__ void load_table(const void* cs, int64_t pair, float (&c)[8], float (&s)[8]) {
  if constexpr (F32) {
    const float4* t = reinterpret_cast<const float4*>(static_cast<const float*>(cs) + 2 * pair);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = __ldg(t + i);
      c[2 * i] = v.x, s[2 * i] = v.y, c[2 * i + 1] = v.z, s[2 * i + 1] = v.w;
    }
  } else {
    const uint4* t = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(cs) + 2 * pair);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 v = __ldg(t + i);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) c[4 * i + k] = bf_lo(w[k]), s[4 * i + k] = bf_hi(w[k]);
    }
  }
}

template <int LANES>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int off = LANES / 2; off >= 1; off >>= 1) x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}

template <int D, bool F32>
__global__ void __launch_bounds__(THREADS) qk_norm_rope_bwd_kernel(const Args a) {
  constexpr int LANES = D / 16, HEADS = 32 / LANES, H2 = D / 2;  // lanes of a head, heads of a warp
  __shared__ float sums[WARPS][2][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % LANES, grp = lane / LANES;
  const PlanHeader* hdr = reinterpret_cast<const PlanHeader*>(a.ws);
  if (hdr->magic != kPlanMagic || hdr->T != a.T) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.err, MOT_DEV_PLAN_MISMATCH);
    return;
  }
  if (hdr->count[0] + hdr->count[1] != a.T) return;  // no plan (bad modality): nothing is defined
  const int32_t* perm = reinterpret_cast<const int32_t*>(a.ws + perm_offset());
  const int nqk = a.Hq + a.Hkv, N = (nqk + a.Hkv) * D;
  const int begin = int(int64_t(a.T) * blockIdx.x / a.ctas), end = int(int64_t(a.T) * (blockIdx.x + 1) / a.ctas);
  const bool copy_v = a.dx != a.d;
  for (int e = 0; e < 2; ++e) {
    const int lo = e == 0 ? begin : max(begin, hdr->count[0]), hi = e == 0 ? min(end, hdr->count[0]) : end;
    float acc[2][2][8] = {};  // [q, k][half][column]
    for (int at = lo + warp; at < hi; at += WARPS) {
      const int64_t row = perm[at];
      int pos = a.pos[row];
      if (pos < 0 || pos >= a.P) {
        if (lane == 0) atomicOr(a.err, MOT_DEV_BAD_POSITION);
        pos = 0;
      }
      float c[8], s[8];
      load_table<F32>(a.cs, int64_t(pos) * H2 + 8 * sub, c, s);
      for (int h0 = 0; h0 < nqk; h0 += HEADS) {
        const int h = h0 + grp;
        const bool has = h < nqk;
        const int kind = h < a.Hq ? 0 : 1;
        const int64_t off = row * N + int64_t(has ? h : 0) * D + 8 * sub;
        float d0[8], d1[8], x0[8], x1[8], w0[8], w1[8];
        unpack8(*reinterpret_cast<const uint4*>(a.d + off), d0);
        unpack8(*reinterpret_cast<const uint4*>(a.d + off + H2), d1);
        unpack8(__ldg(reinterpret_cast<const uint4*>(a.x + off)), x0);
        unpack8(__ldg(reinterpret_cast<const uint4*>(a.x + off + H2)), x1);
        const uint16_t* w = a.w[kind] + e * D + 8 * sub;
        unpack8(__ldg(reinterpret_cast<const uint4*>(w)), w0);
        unpack8(__ldg(reinterpret_cast<const uint4*>(w + H2)), w1);
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __fadd_rn(ss, __fadd_rn(__fmul_rn(x0[i], x0[i]), __fmul_rn(x1[i], x1[i])));
        const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(group_sum<LANES>(ss), float(D)), a.eps)));
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float u0 = __fadd_rn(__fmul_rn(d0[i], c[i]), __fmul_rn(d1[i], s[i]));
          const float u1 = __fsub_rn(__fmul_rn(d1[i], c[i]), __fmul_rn(d0[i], s[i]));
          x0[i] = __fmul_rn(x0[i], rstd);
          x1[i] = __fmul_rn(x1[i], rstd);
          // a head past the last adds zero; both kinds are added to, so that the sums stay in registers
          const float p0 = has ? __fmul_rn(u0, x0[i]) : 0.0f, p1 = has ? __fmul_rn(u1, x1[i]) : 0.0f;
          acc[0][0][i] = __fadd_rn(acc[0][0][i], kind == 0 ? p0 : 0.0f);
          acc[0][1][i] = __fadd_rn(acc[0][1][i], kind == 0 ? p1 : 0.0f);
          acc[1][0][i] = __fadd_rn(acc[1][0][i], kind == 1 ? p0 : 0.0f);
          acc[1][1][i] = __fadd_rn(acc[1][1][i], kind == 1 ? p1 : 0.0f);
          d0[i] = __fmul_rn(u0, w0[i]);
          d1[i] = __fmul_rn(u1, w1[i]);
          dot = __fadd_rn(dot, __fadd_rn(__fmul_rn(d0[i], x0[i]), __fmul_rn(d1[i], x1[i])));
        }
        const float mean = __fdiv_rn(group_sum<LANES>(dot), float(D));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          d0[i] = __fmul_rn(rstd, __fsub_rn(d0[i], __fmul_rn(x0[i], mean)));
          d1[i] = __fmul_rn(rstd, __fsub_rn(d1[i], __fmul_rn(x1[i], mean)));
        }
        if (has) {
          *reinterpret_cast<uint4*>(a.dx + off) = pack8(d0);
          *reinterpret_cast<uint4*>(a.dx + off + H2) = pack8(d1);
        }
      }
      if (copy_v)
        for (int i = lane; i < a.Hkv * D / 8; i += 32)
          *reinterpret_cast<uint4*>(a.dx + row * N + nqk * D + 8 * i) =
              *reinterpret_cast<const uint4*>(a.d + row * N + nqk * D + 8 * i);
    }
    if (a.part == nullptr || ((a.sets >> e) & 1) == 0) continue;
    // the warp's heads, then the warps, in order
#pragma unroll
    for (int kind = 0; kind < 2; ++kind)
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float v = acc[kind][half][i];
#pragma unroll
          for (int off = LANES; off < 32; off <<= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, off));
          if (grp == 0) sums[warp][kind][half * H2 + 8 * sub + i] = v;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += THREADS) {
      float v = sums[0][i / D][i % D];
      for (int k = 1; k < WARPS; ++k) v = __fadd_rn(v, sums[k][i / D][i % D]);
      a.part[((int64_t(blockIdx.x) * 2 + i / D) * 2 + e) * D + i % D] = v;
    }
    __syncthreads();
  }
}

// Adds the CTAs' sums: a CTA takes 32 columns of one kind and set, warp k the runs k, k + 8, ...
template <int D>
__global__ void __launch_bounds__(THREADS) qk_dweight_fold_kernel(const Args a) {
  __shared__ float sums[WARPS][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = int(blockIdx.x) / (D / 32), col = int(blockIdx.x) % (D / 32) * 32 + lane;  // kind * 2 + set
  if (((a.sets >> (group & 1)) & 1) == 0) return;
  const PlanHeader* hdr = reinterpret_cast<const PlanHeader*>(a.ws);
  if (hdr->magic != kPlanMagic || hdr->T != a.T || hdr->count[0] + hdr->count[1] != a.T) return;
  float v = 0.0f;
  for (int i = warp; i < a.ctas; i += WARPS) v = __fadd_rn(v, a.part[(int64_t(i) * 4 + group) * D + col]);
  sums[warp][lane] = v;
  __syncthreads();
  if (warp == 0) {
    v = sums[0][lane];
#pragma unroll
    for (int k = 1; k < WARPS; ++k) v = __fadd_rn(v, sums[k][lane]);
    a.dw[group * D + col] = v;
  }
}

inline int ctas_of(int64_t T) { return int(T < kMaxCtas ? T : kMaxCtas); }

template <bool F32>
static int run(const uint16_t* d, const uint16_t* x, const uint16_t* qw, const uint16_t* kw, const int32_t* pos,
               const void* cs, int P, int64_t T, int Hq, int Hkv, int D, float eps, void* ws, size_t ws_bytes, uint16_t* dx,
               float* dw, int sets, void* scratch, size_t scratch_bytes, void* stream) {
  if (!d || !x || !qw || !kw || !pos || !cs || !ws || !dx || (dw && !scratch)) return MOT_ERR_NULL;
  if (T < 1 || T > MOT_MAX_TOKENS) return MOT_ERR_GEOMETRY;
  if ((D != 64 && D != 128) || Hq < 1 || Hkv < 1 || Hq > 1024 || Hkv > 1024) return MOT_ERR_GEOMETRY;
  if (P < 1 || !(eps > 0.0f) || !(eps <= 3.4e38f) || (dw && (sets < 1 || sets > 3))) return MOT_ERR_ARG;
  if (!aligned16(d) || !aligned16(x) || !aligned16(qw) || !aligned16(kw) || !aligned16(pos) || !aligned16(cs) ||
      !aligned16(ws) || !aligned16(dx) || !aligned16(dw) || (dw && !aligned16(scratch)))
    return MOT_ERR_ALIGN;
  if (ws_bytes < size_t(plan_bytes(T))) return MOT_ERR_WORKSPACE;
  if (dw && scratch_bytes < mot_qk_norm_rope_backward_workspace_bytes(T, D)) return MOT_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const void* ptrs[] = {d, x, qw, kw, pos, cs, ws, dx, dw, dw ? scratch : nullptr};
  int dev = -1;
  const int st = check_device(s, ptrs, 10, &dev);
  if (st != MOT_OK) return st;
  DeviceGuard guard(dev);
  Args a{};
  a.d = d;
  a.x = x;
  a.w[0] = qw;
  a.w[1] = kw;
  a.pos = pos;
  a.cs = cs;
  a.P = P;
  a.T = int(T);
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.eps = eps;
  a.ws = static_cast<const uint8_t*>(ws);
  a.err = &static_cast<PlanHeader*>(ws)->error;
  a.dx = dx;
  a.part = dw ? static_cast<float*>(scratch) : nullptr;
  a.dw = dw;
  a.sets = sets;
  a.ctas = ctas_of(T);
  if (D == 64) qk_norm_rope_bwd_kernel<64, F32><<<a.ctas, THREADS, 0, s>>>(a);
  else qk_norm_rope_bwd_kernel<128, F32><<<a.ctas, THREADS, 0, s>>>(a);
  if (dw) {
    if (D == 64) qk_dweight_fold_kernel<64><<<4 * 64 / 32, THREADS, 0, s>>>(a);
    else qk_dweight_fold_kernel<128><<<4 * 128 / 32, THREADS, 0, s>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? MOT_OK : MOT_ERR_CUDA;
}

}  // namespace qkvb
}  // namespace mot

using namespace mot;

extern "C" size_t mot_qk_norm_rope_backward_workspace_bytes(int64_t T, int D) {
  if (T < 1 || T > MOT_MAX_TOKENS || (D != 64 && D != 128)) return 0;
  return size_t(qkvb::ctas_of(T)) * 4 * D * sizeof(float);
}

extern "C" int mot_qk_norm_rope_backward(const mot_bf16* d_out, const mot_bf16* x, const mot_bf16* q_norm_w,
                                         const mot_bf16* k_norm_w, const int32_t* pos, const mot_bf16* rope_cs, int P,
                                         int64_t T, int Hq, int Hkv, int D, float eps, void* ws, size_t ws_bytes,
                                         mot_bf16* dx, float* dw, int sets, void* scratch, size_t scratch_bytes,
                                         void* stream) {
  return qkvb::run<false>(d_out, x, q_norm_w, k_norm_w, pos, rope_cs, P, T, Hq, Hkv, D, eps, ws, ws_bytes, dx, dw, sets,
                          scratch, scratch_bytes, stream);
}

extern "C" int mot_qk_norm_rope_backward_fp32(const mot_bf16* d_out, const mot_bf16* x, const mot_bf16* q_norm_w,
                                              const mot_bf16* k_norm_w, const int32_t* pos, const float* rope_cs_f32, int P,
                                              int64_t T, int Hq, int Hkv, int D, float eps, void* ws, size_t ws_bytes,
                                              mot_bf16* dx, float* dw, int sets, void* scratch, size_t scratch_bytes,
                                              void* stream) {
  return qkvb::run<true>(d_out, x, q_norm_w, k_norm_w, pos, rope_cs_f32, P, T, Hq, Hkv, D, eps, ws, ws_bytes, dx, dw, sets,
                         scratch, scratch_bytes, stream);
}
