// Attention of single new tokens over a paged key-value cache.
//
// Sources: [RFC][BAGEL-7B-MoT][CUDA/ROCm] WS1/WS2 kernel roadmap and integration plan #435 (§1
// Motivation item 2: queries over the cached prompt KV; §3 Numerical contract: fixed accumulation
// order, a row's bits do not depend on the pack). The attention is the textbook scaled dot-product
// softmax with grouped KV heads.

#include <cuda_runtime.h>

#include "mot_kvcache.cuh"

namespace mot {
namespace decode {

constexpr int WARPS = 8;

struct Args {
  const uint16_t* qkv;   // [R][(Hq + 2 Hkv) D]
  const int32_t* table;  // [R][max_pages]
  const int32_t* lens;   // [R]
  const uint8_t* k;
  const uint8_t* v;
  const float* scales;
  int64_t n_pages;
  int max_pages, page;
  int Hq, Hkv;
  float c;  // scale * log2(e)
  uint16_t* out;  // [R][Hq D]
  uint32_t* err;
};

template <int D, bool E4M3>
__device__ __forceinline__ void load_vec(const uint8_t* base, int64_t row, int lane, float (&x)[D / 32]) {
  if (E4M3) {
    const uint8_t* p = base + row * D + lane * (D / 32);
#pragma unroll
    for (int i = 0; i < D / 32; i += 2) {
      const float2 f = kv::h2_to_f2(kv::e4m3x2_to_h2(*reinterpret_cast<const uint16_t*>(p + i)));
      x[i] = f.x;
      x[i + 1] = f.y;
    }
  } else {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(base) + row * D + lane * (D / 32);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) x[i] = bf_to_f(p[i]);
  }
}

// One CTA per (row, query head); each warp takes every eighth key with its own running maximum and
// sum, the warps' results are joined in order.
template <int D, bool E4M3>
__global__ void __launch_bounds__(32 * WARPS) decode_kernel(const Args a) {
  constexpr int E = D / 32;
  __shared__ float sm[WARPS], sl[WARPS], so[WARPS][D];
  const int64_t row = blockIdx.x / a.Hq;
  const int h = int(blockIdx.x % a.Hq), g = h / (a.Hq / a.Hkv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = a.lens[row];
  if (len < 0 || len > int64_t(a.max_pages) * a.page) {
    if (threadIdx.x == 0) atomicOr(a.err, MOT_DEV_BAD_PAGE);
    return;
  }
  float q[E], o[E];
  const uint16_t* qp = a.qkv + (row * (a.Hq + 2 * a.Hkv) + h) * D + lane * E;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] = bf_to_f(qp[i]);
    o[i] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int j = warp; j < len; j += WARPS) {
    int p = a.table[row * a.max_pages + j / a.page];
    if (p < 0 || p >= a.n_pages) {
      if (lane == 0) atomicOr(a.err, MOT_DEV_BAD_PAGE);
      p = 0;
    }
    const int64_t r = (int64_t(p) * a.Hkv + g) * a.page + j % a.page;
    float x[E], s = 0.0f;
    load_vec<D, E4M3>(a.k, r, lane, x);
#pragma unroll
    for (int i = 0; i < E; ++i) s = __fadd_rn(s, __fmul_rn(q[i], x[i]));
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, off));
    if (E4M3) s = __fmul_rn(s, a.scales[2 * r]);
    s = __fmul_rn(s, a.c);
    const float mn = s > m || isnan(s) ? s : m;
    const float alpha = m == -INFINITY ? 0.0f : exp2f(__fsub_rn(m, mn));
    float w = mn == -INFINITY ? 0.0f : exp2f(__fsub_rn(s, mn));
    m = mn;
    l = __fadd_rn(__fmul_rn(l, alpha), w);
    load_vec<D, E4M3>(a.v, r, lane, x);
    if (E4M3) w = __fmul_rn(w, a.scales[2 * r + 1]);
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = __fadd_rn(__fmul_rn(o[i], alpha), __fmul_rn(w, x[i]));
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < E; ++i) so[warp][lane * E + i] = o[i];
  __syncthreads();
  if (threadIdx.x < D) {
    float top = sm[0];
    for (int w = 1; w < WARPS; ++w) top = sm[w] > top || isnan(sm[w]) ? sm[w] : top;
    float sum = 0.0f, acc = 0.0f;
    for (int w = 0; w < WARPS; ++w) {
      const float f = sm[w] == -INFINITY ? 0.0f : exp2f(__fsub_rn(sm[w], top));
      sum = __fadd_rn(sum, __fmul_rn(sl[w], f));
      acc = __fadd_rn(acc, __fmul_rn(so[w][threadIdx.x], f));
    }
    a.out[(row * a.Hq + h) * D + threadIdx.x] = f_to_bf(sum == 0.0f ? 0.0f : __fdiv_rn(acc, sum));
  }
}

}  // namespace decode
}  // namespace mot

using namespace mot;

extern "C" size_t mot_paged_decode_workspace_bytes(int64_t R, int Hq, int Hkv, int D, int max_pages, int page) {
  if (kv::check_shape(Hq, Hkv, D, MOT_KV_BF16, 1, page) != MOT_OK) return 0;
  if (R < 1 || R > MOT_MAX_TOKENS || max_pages < 1 || int64_t(max_pages) * page > (int64_t(1) << 30)) return 0;
  return sizeof(PlanHeader);
}

extern "C" int mot_paged_decode_attention(const mot_bf16* qkv, int64_t R, int Hq, int Hkv, int D, const int32_t* table,
                                          const int32_t* lens, int max_pages, int kv_type, int64_t n_pages, int page,
                                          const void* k_cache, const void* v_cache, const float* scales, float scale,
                                          void* ws, size_t ws_bytes, mot_bf16* out, void* stream) {
  const bool e4m3 = kv_type == MOT_KV_E4M3;
  if (!qkv || !table || !lens || !k_cache || !v_cache || !ws || !out || (e4m3 && !scales)) return MOT_ERR_NULL;
  int st = kv::check_shape(Hq, Hkv, D, kv_type, n_pages, page);
  if (st != MOT_OK) return st;
  const size_t need = mot_paged_decode_workspace_bytes(R, Hq, Hkv, D, max_pages, page);
  if (need == 0 || R * Hq > (int64_t(1) << 31) - 1) return MOT_ERR_GEOMETRY;
  if (!(scale > 0.0f) || !(scale < 3.0e38f)) return MOT_ERR_ARG;
  if (!aligned16(qkv) || !aligned16(table) || !aligned16(lens) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned16(ws) || !aligned16(out) || (e4m3 && !aligned16(scales)))
    return MOT_ERR_ALIGN;
  if (ws_bytes < need) return MOT_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const void* ptrs[] = {qkv, table, lens, k_cache, v_cache, ws, out, e4m3 ? scales : nullptr};
  int dev = -1;
  st = check_device(s, ptrs, 8, &dev);
  if (st != MOT_OK) return st;
  DeviceGuard guard(dev);
  decode::Args a{};
  a.qkv = qkv;
  a.table = table;
  a.lens = lens;
  a.k = static_cast<const uint8_t*>(k_cache);
  a.v = static_cast<const uint8_t*>(v_cache);
  a.scales = scales;
  a.n_pages = n_pages;
  a.max_pages = max_pages;
  a.page = page;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.c = scale * 1.4426950408889634f;
  a.out = out;
  a.err = &static_cast<PlanHeader*>(ws)->error;
  const unsigned grid = unsigned(R * Hq);
  if (D == 64 && e4m3) decode::decode_kernel<64, true><<<grid, 32 * decode::WARPS, 0, s>>>(a);
  else if (D == 64) decode::decode_kernel<64, false><<<grid, 32 * decode::WARPS, 0, s>>>(a);
  else if (e4m3) decode::decode_kernel<128, true><<<grid, 32 * decode::WARPS, 0, s>>>(a);
  else decode::decode_kernel<128, false><<<grid, 32 * decode::WARPS, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? MOT_OK : MOT_ERR_CUDA;
}
