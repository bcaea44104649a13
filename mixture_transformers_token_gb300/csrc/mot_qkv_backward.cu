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
// of 28/4 heads of 128 at the measured copy rate): the bound is memory. D / 8 lanes hold a head, each 4 values and their 4
// partners, so that the rotation needs no exchange. Loads into registers kept too little under way for the memory's latency (two
// CTAs of 8 warps, the next heads' loads ahead: 36 us on that pack): each warp has a ring of slots in shared memory for a row's
// next heads, their projection and the table entries, filled by bulk copies. 24 warps with two slots, 33.1 us there and 177 us
// (83% of that rate) for 36001 rows of the FP32 profile; 16 warps with three 35.3 and 192 us, 20 with two 34.4 and 194 us, 32 with
// slots of half the size 37.5 and 207 us. With D / 16 lanes a head a thread's registers allow 16 warps: 35.7 and 198 us. What is
// left on the small pack is the start (header, row numbers, positions, first rows: each waits for the one before) and the second
// kernel: a pack of 64 rows takes 13 us.
//
// The weights' gradients: each CTA takes a run of the plan's positions, so that its rows are of one weight set, but for the run
// that holds the border; a lane adds its columns over the warp's rows, the warps' sums are added in order, and a second kernel,
// already launched, adds the CTAs' sums in order.

#include <cuda_runtime.h>

#include "mot.h"
#include "mot_device.cuh"
#include "mot_host.hpp"

namespace mot {
namespace qkvb {

constexpr int WARPS = 24, THREADS = 32 * WARPS;
constexpr int kMaxCtas = 152;           // runs of positions: one for each SM
constexpr int PIECE = 1024;             // values of a slot: the heads of an item
constexpr int SLOTS = 2;
constexpr uint32_t SLOT = 2 * PIECE * 2 + 512 + 16;  // gradient, projection, table entries of a position, the row
constexpr uint32_t RING = WARPS * SLOTS * SLOT;
constexpr uint32_t WEIGHTS = RING, BARS = WEIGHTS + 4 * 128 * 4;
constexpr size_t SMEM = BARS + 8 * WARPS * SLOTS + 16;

struct Args {
  const uint16_t* d;
  const uint16_t* x;
  const uint16_t* qw;    // [2][D]
  const uint16_t* kw;
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

// Four of a lane's values.
__device__ __forceinline__ void unpack4(const uint2& v, float (&x)[4]) {
  x[0] = bf_lo(v.x), x[1] = bf_hi(v.x), x[2] = bf_lo(v.y), x[3] = bf_hi(v.y);
}
__device__ __forceinline__ uint2 pack4(const float (&x)[4]) { return make_uint2(cvt_bf2(x[0], x[1]), cvt_bf2(x[2], x[3])); }

// cos and sin of the lane's 4 pairs
template <bool F32>
__device__ __forceinline__ void load_table(const void* cs, int pair, float (&c)[4], float (&s)[4]) {
  if constexpr (F32) {
    const float4* t = reinterpret_cast<const float4*>(static_cast<const float*>(cs) + 2 * pair);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 v = t[i];
      c[2 * i] = v.x, s[2 * i] = v.y, c[2 * i + 1] = v.z, s[2 * i + 1] = v.w;
    }
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(cs) + 2 * pair);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) c[k] = bf_lo(w[k]), s[k] = bf_hi(w[k]);
  }
}

template <int LANES>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int off = LANES / 2; off >= 1; off >>= 1) x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}

template <int D, bool F32>
__global__ void __launch_bounds__(THREADS, 1) qk_norm_rope_bwd_kernel(const Args a) {
  constexpr int LANES = D / 8, HEADS = 32 / LANES, H2 = D / 2;  // lanes of a head, heads of a warp
  constexpr int ITEM = PIECE / D;                                // heads of an item
  constexpr uint32_t TABLE = D * (F32 ? 4 : 2);                  // bytes of a position's table entries
  extern __shared__ __align__(128) uint8_t smem[];
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % LANES, grp = lane / LANES;
  uint8_t* ring = smem + warp * SLOTS * SLOT;
  float* weights = reinterpret_cast<float*>(smem + WEIGHTS);  // [q, k][2][D]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + BARS) + warp * SLOTS;
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + BARS + 8 * WARPS * SLOTS);
  const int begin = int(int64_t(a.T) * blockIdx.x / a.ctas), end = int(int64_t(a.T) * (blockIdx.x + 1) / a.ctas);
  const int32_t* perm = reinterpret_cast<const int32_t*>(a.ws + perm_offset());
  if (begin + threadIdx.x < end) {  // the first rows' numbers and positions into the caches while the header is read
    const int row = perm[begin + threadIdx.x];
    if (row >= 0 && row < a.T) asm volatile("prefetch.global.L1 [%0];" ::"l"(a.pos + row));
  }
  const float weight = threadIdx.x < 4 * D ? bf_to_f((threadIdx.x < 2 * D ? a.qw : a.kw)[threadIdx.x % (2 * D)]) : 0.0f;
  const PlanHeader* hdr = reinterpret_cast<const PlanHeader*>(a.ws);
  if (hdr->magic != kPlanMagic || hdr->T != a.T) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.err, MOT_DEV_PLAN_MISMATCH);
    return;
  }
  const int count0 = hdr->count[0];
  if (count0 + hdr->count[1] != a.T) return;  // no plan (bad modality): nothing is defined
  if (lane == 0) {
    for (int i = 0; i < SLOTS; ++i) mbar_init(smem_u32(&full[i]), 1);
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (threadIdx.x == 0) *abort_flag = 0u;
  static_assert(4 * D <= THREADS, "a thread a weight");
  if (threadIdx.x < 4 * D) weights[threadIdx.x] = weight;
  __syncthreads();
  const int nqk = a.Hq + a.Hkv, n_heads = nqk + a.Hkv;
  // items of a row: the normed heads, and, where the result is elsewhere, the value heads to copy
  const int normed = (nqk + ITEM - 1) / ITEM, items = normed + (a.dx != a.d ? (a.Hkv + ITEM - 1) / ITEM : 0);
  int issued = 0, taken = 0;  // of all this warp's items
  bool ok = true;
  for (int e = 0; e < 2; ++e) {
    const int lo = e == 0 ? begin : max(begin, count0), hi = e == 0 ? min(end, count0) : end;
    float acc[2][2][4] = {};  // [q, k][half][column]
    const int all = hi > lo ? (hi - lo) * items : 0;                 // less than 2^26
    const int n = ok && all > warp ? (all - warp + WARPS - 1) / WARPS : 0;  // this warp's items: warp, warp + WARPS, ...
    int my_row = 0, my_pos = 0;                                      // of its items that a lane looks up, 32 at once
    int next_item = warp % items, this_item = next_item;             // of the row: the next one to issue, and to take
    auto issue = [&](int j) {
      if ((j & 31) == 0 && j + lane < n) {
        my_row = perm[lo + (warp + (j + lane) * WARPS) / items];
        my_pos = a.pos[my_row];
        if (my_pos < 0 || my_pos >= a.P) {
          atomicOr(a.err, MOT_DEV_BAD_POSITION);
          my_pos = 0;
        }
      }
      const int row = __shfl_sync(0xffffffffu, my_row, j & 31), pos = __shfl_sync(0xffffffffu, my_pos, j & 31);
      if (lane == 0) {
        const int item = next_item, s = issued % SLOTS;
        const int h = item < normed ? item * ITEM : nqk + (item - normed) * ITEM, to = item < normed ? nqk : n_heads;
        const uint32_t bytes = uint32_t(to - h < ITEM ? to - h : ITEM) * D * 2, bar = smem_u32(&full[s]);
        uint8_t* slot = ring + s * SLOT;
        const int64_t off = (int64_t(row) * n_heads + h) * D;
        *reinterpret_cast<int*>(slot + 4 * PIECE + 512) = row;
        mbar_arrive_expect_tx(bar, item < normed ? 2 * bytes + TABLE : bytes);
        bulk_load(smem_u32(slot), a.d + off, bytes, bar);
        if (item < normed) {
          bulk_load(smem_u32(slot + 2 * PIECE), a.x + off, bytes, bar);
          bulk_load(smem_u32(slot + 4 * PIECE), static_cast<const uint8_t*>(a.cs) + int64_t(pos) * TABLE, TABLE, bar);
        }
      }
      ++issued;
      next_item = (next_item + WARPS) % items;
    };
    for (int j = 0; j < n && j < SLOTS - 1; ++j) issue(j);
    for (int j = 0; j < n; ++j, ++taken) {
      __syncwarp();  // every lane has read the slot that is filled next
      if (j + SLOTS - 1 < n) issue(j + SLOTS - 1);
      const int s = taken % SLOTS;
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&full[s]), uint32_t(taken / SLOTS) & 1u, abort_flag, a.err));
      if (!ok) break;
      const uint8_t* slot = ring + s * SLOT;
      const int item = this_item;
      this_item = (this_item + WARPS) % items;
      const int64_t row = *reinterpret_cast<const int*>(slot + 4 * PIECE + 512);
      if (item >= normed) {
        const int h = (item - normed) * ITEM, pieces = min(a.Hkv - h, ITEM) * D / 8;
        uint4* to = reinterpret_cast<uint4*>(a.dx + (row * n_heads + nqk + h) * D);
        for (int i = lane; i < pieces; i += 32) to[i] = reinterpret_cast<const uint4*>(slot)[i];
        continue;
      }
      float c[4], sn[4];
      load_table<F32>(slot + 4 * PIECE, 4 * sub, c, sn);
#pragma unroll 1
      for (int h0 = item * ITEM; h0 < min((item + 1) * ITEM, nqk); h0 += HEADS) {
        const int h = h0 + grp, at = (h - item * ITEM) * D + 4 * sub;  // a head past the last reads what was in the slot
        const bool has = h < nqk, key = h >= a.Hq;
        float d0[4], d1[4], x0[4], x1[4];
        const uint16_t* ds = reinterpret_cast<const uint16_t*>(slot) + at;
        unpack4(*reinterpret_cast<const uint2*>(ds), d0);
        unpack4(*reinterpret_cast<const uint2*>(ds + H2), d1);
        unpack4(*reinterpret_cast<const uint2*>(ds + PIECE), x0);
        unpack4(*reinterpret_cast<const uint2*>(ds + PIECE + H2), x1);
        float ss = 0.0f, p0[4], p1[4];
        mul_each(x0, x0, p0);
        mul_each(x1, x1, p1);
#pragma unroll
        for (int k = 0; k < 4; ++k) ss = __fadd_rn(ss, __fadd_rn(p0[k], p1[k]));
        const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fmul_rn(group_sum<LANES>(ss), 1.0f / D), a.eps)));
        float u0[4], u1[4], dot = 0.0f;
        mul_each(d0, c, u0);
        mul_each(d1, sn, p0);
        mul_each(d1, c, u1);
        mul_each(d0, sn, p1);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          u0[k] = __fadd_rn(u0[k], p0[k]);
          u1[k] = __fsub_rn(u1[k], p1[k]);
        }
        mul_each(x0, rstd, x0);
        mul_each(x1, rstd, x1);
        mul_each(u0, x0, p0);
        mul_each(u1, x1, p1);
        if (!__all_sync(0xffffffffu, has)) {  // heads past the last add zero
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            p0[k] = has ? p0[k] : 0.0f;
            p1[k] = has ? p1[k] : 0.0f;
          }
        }
        // q's heads, k's, or some of both
        if (__all_sync(0xffffffffu, !key)) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            acc[0][0][k] = __fadd_rn(acc[0][0][k], p0[k]);
            acc[0][1][k] = __fadd_rn(acc[0][1][k], p1[k]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            acc[0][0][k] = __fadd_rn(acc[0][0][k], key ? 0.0f : p0[k]);
            acc[0][1][k] = __fadd_rn(acc[0][1][k], key ? 0.0f : p1[k]);
            acc[1][0][k] = __fadd_rn(acc[1][0][k], key ? p0[k] : 0.0f);
            acc[1][1][k] = __fadd_rn(acc[1][1][k], key ? p1[k] : 0.0f);
          }
        }
        const float* w = weights + ((key ? 2 : 0) + e) * D + 4 * sub;
        float w0[4], w1[4];
        *reinterpret_cast<float4*>(w0) = *reinterpret_cast<const float4*>(w);
        *reinterpret_cast<float4*>(w1) = *reinterpret_cast<const float4*>(w + H2);
        mul_each(u0, w0, u0);
        mul_each(u1, w1, u1);
        mul_each(u0, x0, p0);
        mul_each(u1, x1, p1);
#pragma unroll
        for (int k = 0; k < 4; ++k) dot = __fadd_rn(dot, __fadd_rn(p0[k], p1[k]));
        const float mean = __fmul_rn(group_sum<LANES>(dot), 1.0f / D);  // D is a power of two
        mul_each(x0, mean, x0);
        mul_each(x1, mean, x1);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          d0[k] = __fsub_rn(u0[k], x0[k]);
          d1[k] = __fsub_rn(u1[k], x1[k]);
        }
        mul_each(d0, rstd, d0);
        mul_each(d1, rstd, d1);
        if (has) {
          uint16_t* to = a.dx + (row * n_heads + h) * D + 4 * sub;
          *reinterpret_cast<uint2*>(to) = pack4(d0);
          *reinterpret_cast<uint2*>(to + H2) = pack4(d1);
        }
      }
    }
    if (a.part == nullptr || ((a.sets >> e) & 1) == 0) continue;
    // the warp's heads, then the warps, in order; through the rings, whose copies have all been taken
    __syncthreads();
    float* sums = reinterpret_cast<float*>(smem);  // [WARPS][2][D]
#pragma unroll
    for (int kind = 0; kind < 2; ++kind)
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v = acc[kind][half][i];
#pragma unroll
          for (int off = LANES; off < 32; off <<= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, off));
          if (grp == 0 && ok) sums[(warp * 2 + kind) * D + half * H2 + 4 * sub + i] = v;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += THREADS) {
      float v = sums[i];
#pragma unroll
      for (int k = 1; k < WARPS; ++k) v = __fadd_rn(v, sums[k * 2 * D + i]);
      a.part[((int64_t(blockIdx.x) * 2 + i / D) * 2 + e) * D + i % D] = v;
    }
    fence_proxy_async_smem();  // before the next set's copies land here
    __syncthreads();
  }
  // after a timeout: no copy may still land when the CTA exits
  if (!ok && lane == 0)
    for (int j = taken; j < issued; ++j) mbar_drain(smem_u32(&full[j % SLOTS]), uint32_t(j / SLOTS) & 1u);
}

// Adds the CTAs' sums: a CTA takes 32 columns of one kind and set, warp k the runs k, k + 32, ... (at most five) in ascending
// order, then the warps' sums in theirs.
constexpr int FOLD_WARPS = 32, FOLD_THREADS = 32 * FOLD_WARPS;

template <int D>
__global__ void __launch_bounds__(FOLD_THREADS) qk_dweight_fold_kernel(const Args a) {
  __shared__ float sums[FOLD_WARPS][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = int(blockIdx.x) / (D / 32), col = int(blockIdx.x) % (D / 32) * 32 + lane;  // kind * 2 + set
  // the plan is older than the grid before this one
  const PlanHeader* hdr = reinterpret_cast<const PlanHeader*>(a.ws);
  const bool plan = hdr->magic == kPlanMagic && hdr->T == a.T && hdr->count[0] + hdr->count[1] == a.T;
  pdl_wait();  // also where nothing is written: this grid ends after the one before it
  if (((a.sets >> (group & 1)) & 1) == 0 || !plan) return;
  float v = 0.0f;
  for (int i = warp; i < a.ctas; i += FOLD_WARPS) v = __fadd_rn(v, __ldcg(a.part + (int64_t(i) * 4 + group) * D + col));
  sums[warp][lane] = v;
  __syncthreads();
  if (warp == 0) {
    v = sums[0][lane];
#pragma unroll
    for (int k = 1; k < FOLD_WARPS; ++k) v = __fadd_rn(v, sums[k][lane]);
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
  a.qw = qw;
  a.kw = kw;
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
  static_assert(SMEM <= 227 * 1024 && WARPS * 2 * 128 * 4 <= RING, "shared memory");
  if (cudaFuncSetAttribute(D == 64 ? qk_norm_rope_bwd_kernel<64, F32> : qk_norm_rope_bwd_kernel<128, F32>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, int(SMEM)) != cudaSuccess)
    return MOT_ERR_CUDA;
  if (D == 64) qk_norm_rope_bwd_kernel<64, F32><<<a.ctas, THREADS, SMEM, s>>>(a);
  else qk_norm_rope_bwd_kernel<128, F32><<<a.ctas, THREADS, SMEM, s>>>(a);
  if (cudaGetLastError() != cudaSuccess) return MOT_ERR_CUDA;
  if (dw) {
    const cudaError_t fold =
        D == 64 ? launch_dependent(qk_dweight_fold_kernel<64>, dim3(4 * 64 / 32), dim3(FOLD_THREADS), 0, s, a)
                : launch_dependent(qk_dweight_fold_kernel<128>, dim3(4 * 128 / 32), dim3(FOLD_THREADS), 0, s, a);
    if (fold != cudaSuccess) return MOT_ERR_CUDA;
  }
  return MOT_OK;
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
