// Writing the K and V columns of fused QKV rows into a paged cache, and reading them back.
//
// Sources: [RFC][BAGEL-7B-MoT][CUDA/ROCm] WS1/WS2 kernel roadmap and integration plan #435 (§1
// Motivation item 2: latent tokens query the prompt KV at every step; §2 Reference hazards: cached
// prefill). The pages name the cached prompt KV and fix no cache layout.
//
// Both directions move each (row, head) pair of vectors once: a group of D / 16 lanes takes one vector of
// D bf16, two 16-byte pieces a lane, K's group beside V's of the same token and head. HBM bounds them. A group
// walks its vectors by additions: a 64-bit division a vector cost as much as the quantiser. On 36864
// rows of 4 heads of 128 in e4m3 (115 MB to read and write, 16.9 us at the copy's rate) the write takes
// 18.8 us and the read 20.7; with one piece a lane (twice the shuffles, address sums and groups) they took
// 28.3 and 25.3, with two vectors of one piece in flight 25.9 and 22.2.

#include <cuda_runtime.h>

#include "mot_kvcache.cuh"

namespace mot {
namespace kv {

constexpr int THREADS = 256;
constexpr int PIECES = 2;  // 16-byte pieces of a vector that a lane takes

// Lanes of a vector's group: lane l takes the pieces l and l + LANES.
template <int D>
constexpr int kLanes = D / (8 * PIECES);

struct MoveArgs {
  uint16_t* qkv;         // [T][(Hq + 2 Hkv) D]
  const int32_t* slots;  // [T]
  uint8_t* k;
  uint8_t* v;
  float* scales;
  int T, Hq, Hkv, page;
  uint32_t n_slots;
  Div by_page;
  int step_row, step_j;  // the grid's groups, as rows and a rest of vectors
  uint32_t* err;
};

// A vector of the call: K (j even) or V (j odd) of head j / 2 of a row. The groups of the grid take
// consecutive vectors; the next of a group is the grid's groups further on.
struct Pos {
  int row, j;
  __device__ __forceinline__ void next(const MoveArgs& a) {
    row += a.step_row;
    j += a.step_j;
    if (j >= 2 * a.Hkv) {
      j -= 2 * a.Hkv;
      ++row;
    }
  }
};

template <int D>
__device__ __forceinline__ Pos first_pos(const MoveArgs& a) {
  const int64_t u = int64_t(blockIdx.x) * (THREADS / kLanes<D>) + threadIdx.x / kLanes<D>;
  Pos p;
  p.row = int(u / (2 * a.Hkv));
  p.j = int(u - int64_t(p.row) * (2 * a.Hkv));
  return p;
}

// Element offset of a vector in qkv.
template <int D>
__device__ __forceinline__ int64_t in_rows(const MoveArgs& a, const Pos& p) {
  return (int64_t(p.row) * (a.Hq + 2 * a.Hkv) + a.Hq + (p.j & 1 ? a.Hkv : 0) + (p.j >> 1)) * D;
}

// Row of a vector in the cache, < 0 if the row has no slot (reported unless it is -1).
__device__ __forceinline__ int64_t in_cache(const MoveArgs& a, const Pos& p, int slot) {
  if (uint32_t(slot) < a.n_slots) {
    const uint32_t page = a.by_page.of(uint32_t(slot));
    return (int64_t(page) * a.Hkv + (p.j >> 1)) * a.page + int(uint32_t(slot) - page * uint32_t(a.page));
  }
  if (slot != -1) atomicOr(a.err, MOT_DEV_BAD_PAGE);
  return -1;
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(THREADS) kv_write_kernel(const MoveArgs a) {
  constexpr int LANES = kLanes<D>;
  const int lane = threadIdx.x % LANES;
  Pos p = first_pos<D>(a);
  pdl_wait();
  // whole warps leave together: the lanes exchange maxima
  for (; __any_sync(0xffffffffu, p.row < a.T); p.next(a)) {
    uint32_t x[PIECES][4] = {};
    int64_t to = -1;
    if (p.row < a.T) {
      const uint4* src = reinterpret_cast<const uint4*>(a.qkv + in_rows<D>(a, p)) + lane;
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const uint4 u = __ldg(src + i * LANES);
        x[i][0] = u.x; x[i][1] = u.y; x[i][2] = u.z; x[i][3] = u.w;
      }
      to = in_cache(a, p, __ldg(a.slots + p.row));
    }
    uint8_t* dst = p.j & 1 ? a.v : a.k;
    if constexpr (!E4M3) {
      if (to >= 0)
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
          reinterpret_cast<uint4*>(dst + to * (2 * D))[lane + i * LANES] =
              make_uint4(x[i][0], x[i][1], x[i][2], x[i][3]);
    } else {
      // magnitudes as bits, two at a time: their order is the floats', infinities and NaNs last
      uint32_t top2 = 0;
#pragma unroll
      for (int i = 0; i < PIECES; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) top2 = __vmaxu2(top2, x[i][k] & 0x7FFF7FFFu);
#pragma unroll
      for (int off = LANES / 2; off >= 1; off >>= 1) top2 = __vmaxu2(top2, __shfl_xor_sync(0xffffffffu, top2, off));
      const float scale = e4m3_scale(__uint_as_float(max(top2 << 16, top2 & 0xFFFF0000u)));
      const float inv = inverse_scale(scale);
      if (to >= 0) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
          uint32_t c[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) c[k] = e4m3x2(__fmul_rn(bf_lo(x[i][k]), inv), __fmul_rn(bf_hi(x[i][k]), inv));
          reinterpret_cast<uint2*>(dst + to * D)[lane + i * LANES] = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
        }
        if (lane == 0) a.scales[to * 2 + (p.j & 1)] = scale;
      }
    }
  }
}

// a b to fp32 with the last bit set where bits were dropped, so that a rounding to bf16 that follows has the
// exact product's result: a code times a scale has up to 28 bits (all within fp32's range down to 2^-122).
__device__ __forceinline__ float product_to_odd(float a, float b) {
  const float p = __fmul_rz(a, b);
  return __uint_as_float(__float_as_uint(p) | (__fmaf_rn(a, b, -p) != 0.0f ? 1u : 0u));
}

// Eight codes times a scale that is no power of two, rounded once.
__device__ __forceinline__ void store_to_odd(uint4* dst, uint2 c, float scale) {
  const uint32_t codes[4] = {c.x & 0xFFFFu, c.x >> 16, c.y & 0xFFFFu, c.y >> 16};
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 v = h2_to_f2(e4m3x2_to_h2(codes[k]));
    o[k] = pack_bf2(product_to_odd(v.x, scale), product_to_odd(v.y, scale));
  }
  *dst = make_uint4(o[0], o[1], o[2], o[3]);
}

// Eight blocks an SM, as many as its threads allow: with 40 registers instead of 32 the 36864 rows took 23.7 us.
template <int D, bool E4M3>
__global__ void __launch_bounds__(THREADS, 8) kv_read_kernel(const MoveArgs a) {
  constexpr int LANES = kLanes<D>;
  const int lane = threadIdx.x % LANES;
  Pos p = first_pos<D>(a);
  pdl_wait();
  for (; p.row < a.T; p.next(a)) {
    const int64_t from = in_cache(a, p, __ldg(a.slots + p.row));
    if (from < 0) continue;
    const uint8_t* src = p.j & 1 ? a.v : a.k;
    uint4* dst = reinterpret_cast<uint4*>(a.qkv + in_rows<D>(a, p)) + lane;
    if constexpr (!E4M3) {
      uint4 x[PIECES];
#pragma unroll
      for (int i = 0; i < PIECES; ++i) x[i] = __ldg(reinterpret_cast<const uint4*>(src + from * (2 * D)) + lane + i * LANES);
#pragma unroll
      for (int i = 0; i < PIECES; ++i) dst[i * LANES] = x[i];
    } else {
      uint2 c[PIECES];
#pragma unroll
      for (int i = 0; i < PIECES; ++i) c[i] = __ldg(reinterpret_cast<const uint2*>(src + from * D) + lane + i * LANES);
      const float scale = __ldg(a.scales + from * 2 + (p.j & 1));
      // a power of two is exact. The others apart, a whole vector: as a choice an element 36864 rows took 21.5 us, as
      // two equal branches 777 rows 1.9 instead of 1.7
      if (__builtin_expect((__float_as_uint(scale) & 0x007FFFFFu) != 0u, 0)) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) store_to_odd(dst + i * LANES, c[i], scale);
        continue;
      }
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const uint32_t codes[4] = {c[i].x & 0xFFFFu, c[i].x >> 16, c[i].y & 0xFFFFu, c[i].y >> 16};
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 v = h2_to_f2(e4m3x2_to_h2(codes[k]));
          o[k] = pack_bf2(__fmul_rn(v.x, scale), __fmul_rn(v.y, scale));
        }
        dst[i * LANES] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

static int move(bool write, uint16_t* qkv, int64_t T, int Hq, int Hkv, int D, const int32_t* slots, int kv_type,
                int64_t n_pages, int page, void* k, void* v, float* scales, void* ws, size_t ws_bytes, void* stream) {
  const bool e4m3 = kv_type == MOT_KV_E4M3;
  if (!qkv || !slots || !k || !v || !ws || (e4m3 && !scales)) return MOT_ERR_NULL;
  int st = check_shape(Hq, Hkv, D, kv_type, n_pages, page);
  if (st != MOT_OK) return st;
  if (T < 1 || T > MOT_MAX_TOKENS) return MOT_ERR_GEOMETRY;
  if (!aligned16(qkv) || !aligned4(slots) || !aligned16(k) || !aligned16(v) || !aligned16(ws) ||
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
  a.T = int(T);
  a.n_slots = uint32_t(n_pages * page);
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.page = page;
  a.by_page = Div(uint32_t(page));
  a.err = &static_cast<PlanHeader*>(ws)->error;
  const int64_t groups = THREADS / (D / (8 * PIECES)), vectors = T * Hkv * 2;
  const int64_t want = (vectors + groups - 1) / groups, most = int64_t(16) * sm_count(dev);
  const unsigned grid = unsigned(want < most ? want : most);
  a.step_row = int(int64_t(grid) * groups / (2 * Hkv));
  a.step_j = int(int64_t(grid) * groups % (2 * Hkv));
  cudaError_t e;
#define MOT_KV_LAUNCH(KERNEL)                                                                        \
  (D == 64 ? (e4m3 ? launch_dependent(KERNEL<64, true>, dim3(grid), dim3(THREADS), 0, s, a)          \
                   : launch_dependent(KERNEL<64, false>, dim3(grid), dim3(THREADS), 0, s, a))        \
           : (e4m3 ? launch_dependent(KERNEL<128, true>, dim3(grid), dim3(THREADS), 0, s, a)         \
                   : launch_dependent(KERNEL<128, false>, dim3(grid), dim3(THREADS), 0, s, a)))
  if (write) e = MOT_KV_LAUNCH(kv_write_kernel);
  else e = MOT_KV_LAUNCH(kv_read_kernel);
#undef MOT_KV_LAUNCH
  return e == cudaSuccess ? MOT_OK : MOT_ERR_CUDA;
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
