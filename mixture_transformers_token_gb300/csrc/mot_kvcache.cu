// Writing the K and V columns of fused QKV rows into a paged cache, and reading them back.
//
// Sources: [RFC][BAGEL-7B-MoT][CUDA/ROCm] WS1/WS2 kernel roadmap and integration plan #435 (§1
// Motivation item 2: latent tokens query the prompt KV at every step; §2 Reference hazards: cached
// prefill). The pages name the cached prompt KV and fix no cache layout.
//
// Both directions move each (row, head) pair of vectors once: a group of D / 8 lanes takes one
// vector of D bf16 in 16-byte pieces, K's group beside V's of the same token and head.

#include <cuda_runtime.h>

#include "mot_kvcache.cuh"

namespace mot {
namespace kv {

struct MoveArgs {
  uint16_t* qkv;         // [T][(Hq + 2 Hkv) D]
  const int32_t* slots;  // [T]
  uint8_t* k;
  uint8_t* v;
  float* scales;
  int64_t vectors;  // T * Hkv * 2
  int64_t n_slots;
  int Hq, Hkv, page;
  uint32_t* err;
};

// Vector u of the call: K (u even) or V (u odd) of head (u / 2) % Hkv of row u / (2 Hkv).
struct Vec {
  int64_t src;   // element offset of the vector in qkv
  int64_t slot;  // row index of the vector in the cache, < 0: skipped
};

template <int D>
__device__ __forceinline__ Vec locate(const MoveArgs& a, int64_t u) {
  const int64_t t = u >> 1;
  const int64_t row = t / a.Hkv;
  const int h = int(t - row * a.Hkv);
  const int s = a.slots[row];
  Vec r;
  r.src = (row * (a.Hq + 2 * a.Hkv) + a.Hq + (u & 1 ? a.Hkv : 0) + h) * D;
  r.slot = -1;
  if (s >= 0 && s < a.n_slots) {
    const int p = s / a.page;
    r.slot = (int64_t(p) * a.Hkv + h) * a.page + (s - p * a.page);
  } else if (s != -1) {
    atomicOr(a.err, MOT_DEV_BAD_PAGE);
  }
  return r;
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(256) kv_write_kernel(const MoveArgs a) {
  constexpr int LANES = D / 8;  // of one vector
  const int lane = threadIdx.x % LANES;
  const int64_t step = int64_t(gridDim.x) * (256 / LANES);
  for (int64_t u0 = int64_t(blockIdx.x) * (256 / LANES) + threadIdx.x / LANES;; u0 += step) {
    // whole warps leave together: the lanes exchange maxima
    if (__all_sync(0xffffffffu, u0 >= a.vectors)) break;
    Vec w{0, -1};
    if (u0 < a.vectors) w = locate<D>(a, u0);
    uint4 x = make_uint4(0, 0, 0, 0);
    if (w.slot >= 0) x = __ldg(reinterpret_cast<const uint4*>(a.qkv + w.src) + lane);
    uint8_t* dst = u0 & 1 ? a.v : a.k;
    if (!E4M3) {
      if (w.slot >= 0) reinterpret_cast<uint4*>(dst + w.slot * (2 * D))[lane] = x;
      continue;
    }
    const uint32_t r[4] = {x.x, x.y, x.z, x.w};
    // magnitudes as bits: their order is the floats', infinities and NaNs last
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = (r[i] << 16) & 0x7FFFFFFFu, hi = r[i] & 0x7FFF0000u;
      top = max(top, max(lo, hi));
    }
#pragma unroll
    for (int off = LANES / 2; off >= 1; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float scale = e4m3_scale(__uint_as_float(top));
    const float inv = inverse_scale(scale);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = e4m3x2(__fmul_rn(bf_lo(r[i]), inv), __fmul_rn(bf_hi(r[i]), inv));
    if (w.slot >= 0) {
      reinterpret_cast<uint2*>(dst + w.slot * D)[lane] = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
      if (lane == 0) a.scales[w.slot * 2 + (u0 & 1)] = scale;
    }
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(256) kv_read_kernel(const MoveArgs a) {
  constexpr int LANES = D / 8;
  const int lane = threadIdx.x % LANES;
  const int64_t step = int64_t(gridDim.x) * (256 / LANES);
  for (int64_t u = int64_t(blockIdx.x) * (256 / LANES) + threadIdx.x / LANES; u < a.vectors; u += step) {
    const Vec w = locate<D>(a, u);
    if (w.slot < 0) continue;
    const uint8_t* src = u & 1 ? a.v : a.k;
    uint4 x;
    if (!E4M3) {
      x = __ldg(reinterpret_cast<const uint4*>(src + w.slot * (2 * D)) + lane);
    } else {
      const uint2 c = __ldg(reinterpret_cast<const uint2*>(src + w.slot * D) + lane);
      const float scale = __ldg(a.scales + w.slot * 2 + (u & 1));
      const uint32_t codes[4] = {c.x & 0xFFFFu, c.x >> 16, c.y & 0xFFFFu, c.y >> 16};
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = h2_to_f2(e4m3x2_to_h2(codes[i]));
        o[i] = pack_bf2(__fmul_rn(f.x, scale), __fmul_rn(f.y, scale));
      }
      x = make_uint4(o[0], o[1], o[2], o[3]);
    }
    reinterpret_cast<uint4*>(a.qkv + w.src)[lane] = x;
  }
}

static int move(bool write, uint16_t* qkv, int64_t T, int Hq, int Hkv, int D, const int32_t* slots, int kv_type,
                int64_t n_pages, int page, void* k, void* v, float* scales, void* ws, size_t ws_bytes, void* stream) {
  const bool e4m3 = kv_type == MOT_KV_E4M3;
  if (!qkv || !slots || !k || !v || !ws || (e4m3 && !scales)) return MOT_ERR_NULL;
  int st = check_shape(Hq, Hkv, D, kv_type, n_pages, page);
  if (st != MOT_OK) return st;
  if (T < 1 || T > MOT_MAX_TOKENS) return MOT_ERR_GEOMETRY;
  if (!aligned16(qkv) || !aligned16(slots) || !aligned16(k) || !aligned16(v) || !aligned16(ws) ||
      (e4m3 && !aligned16(scales)))
    return MOT_ERR_ALIGN;
  if (ws_bytes < sizeof(PlanHeader)) return MOT_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const void* ptrs[] = {qkv, slots, k, v, ws, e4m3 ? scales : nullptr};
  int dev = -1;
  st = check_device(s, ptrs, 6, &dev);
  if (st != MOT_OK) return st;
  DeviceGuard guard(dev);
  MoveArgs a{};
  a.qkv = qkv;
  a.slots = slots;
  a.k = static_cast<uint8_t*>(k);
  a.v = static_cast<uint8_t*>(v);
  a.scales = scales;
  a.vectors = T * Hkv * 2;
  a.n_slots = n_pages * page;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.page = page;
  a.err = &static_cast<PlanHeader*>(ws)->error;
  const int64_t per_cta = 256 / (D / 8);
  const int64_t want = (a.vectors + per_cta - 1) / per_cta, most = int64_t(8) * sm_count(dev);
  const unsigned grid = unsigned(want < most ? want : most);
#define MOT_KV_LAUNCH(KERNEL)                                    \
  do {                                                           \
    if (D == 64 && e4m3) KERNEL<64, true><<<grid, 256, 0, s>>>(a);   \
    else if (D == 64) KERNEL<64, false><<<grid, 256, 0, s>>>(a);     \
    else if (e4m3) KERNEL<128, true><<<grid, 256, 0, s>>>(a);        \
    else KERNEL<128, false><<<grid, 256, 0, s>>>(a);                 \
  } while (0)
  if (write) MOT_KV_LAUNCH(kv_write_kernel);
  else MOT_KV_LAUNCH(kv_read_kernel);
#undef MOT_KV_LAUNCH
  return cudaGetLastError() == cudaSuccess ? MOT_OK : MOT_ERR_CUDA;
}

}  // namespace kv
}  // namespace mot

using namespace mot;

extern "C" int mot_kv_cache_write(const mot_bf16* qkv, int64_t T, int Hq, int Hkv, int D, const int32_t* slots,
                                  int kv_type, int64_t n_pages, int page, void* k_cache, void* v_cache, float* scales,
                                  void* ws, size_t ws_bytes, void* stream) {
  return kv::move(true, const_cast<mot_bf16*>(qkv), T, Hq, Hkv, D, slots, kv_type, n_pages, page, k_cache, v_cache,
                  scales, ws, ws_bytes, stream);
}

extern "C" int mot_kv_cache_read(const void* k_cache, const void* v_cache, const float* scales, int kv_type,
                                 int64_t n_pages, int page, const int32_t* slots, int64_t T, int Hq, int Hkv, int D,
                                 mot_bf16* qkv, void* ws, size_t ws_bytes, void* stream) {
  return kv::move(false, qkv, T, Hq, Hkv, D, slots, kv_type, n_pages, page, const_cast<void*>(k_cache),
                  const_cast<void*>(v_cache), const_cast<float*>(scales), ws, ws_bytes, stream);
}
