// Attention of single new tokens over a paged key-value cache, split over the keys and joined.
//
// Sources: [RFC][BAGEL-7B-MoT][CUDA/ROCm] WS1/WS2 kernel roadmap and integration plan #435 (§1
// Motivation item 2: queries over the cached prompt KV; §3 Numerical contract: fixed accumulation
// order, a row's bits do not depend on the pack). The attention is the textbook scaled dot-product
// softmax with grouped KV heads.
//
// Splitting. A row's keys are cut into ranges of span(len) keys, a function of the row's own length
// and the head geometry alone, so a row's bits do not depend on the batch. The span is the shortest
// multiple of a CTA's round (8 warps x TOK keys), 512 keys at least, that cuts one row into no more
// (range, KV head) items than there are SMs: a single long row then fills the machine in one wave, and
// each long row of a batch gives every SM about one item. Of the shortest spans 256, 512, 768 and 1024,
// 512 was taken over 20 batches: 1024 is 12 % faster on 12 rows of 2000 keys, 7 % on 128 of 750 and 2 % on 64
// of up to 8192, but 24 % slower on one row of 4000 and 13 % on 33 of 750; 256 is 9 % faster on one row of 4000
// and 28 % slower on 256 e4m3 rows of up to 4096. A persistent CTA per SM takes every 152nd item.
//
// Arithmetic of an item (a key range of one KV head, up to 8 of its query heads): warp w of 8 takes
// the range's tiles w, w + 8, ... of TOK keys. Per tile S^T = K Q^T with mma.sync (m16n8k16: 16 keys x
// 8 heads), x = S c in powers of two, then w = 2^(x - ref) where a head's reference starts from the
// tile's maximum and moves only when a tile's maximum is 2^8 above the one that set it (e4m3: the largest w is
// at least 2^6, and w <= 2^14); sums of w in fp32 per lane; O^T += V^T W^T (m16n8k16: 16 dims x 8
// heads), the weights turned by movmatrix. The 8 warps' (ref, sum, O) are joined in a fixed order, the
// ranges' in a fixed order by join_kernel. Every fp32 operation is rounded on its own.
// bf16 cache: w goes into the product as two bf16 (w and what its rounding leaves), so the weights
// keep 16 bits: one bf16 each would put an error the size of the output's own rounding beside it. Two bf16
// have fp32's exponents, so w needs no headroom above the smallest: with n keys in the item w <= 2^-m, m the
// smallest that has n <= 2^m. An item's weights then add up to at most 1, and O is finite wherever the values are.
// e4m3 cache: codes become halves (exact), the query too, scaled by a power of two that takes its largest
// element into [2^14, 2^15) (exact but for elements below 2^-24 of it), and a weight is a half. A token's
// V scale belongs into its weight, so the reference follows x + log2(scale): the halves' range is then
// spent on what the products contribute, however the scales differ. The sums take the same exponential over
// the scale. That is in range while the scales are 2^-64 to 2^17: a key whose score leads, with the smallest
// scale (a zero vector has it) beside the largest, is at 2^-80 of the largest product. Beside a scale of 2^17
// and more it could fall below fp32's range and out of the sum, so a warp that has met one takes its sums from
// the scores alone, in a second pass over its keys (loud_sums).
//
// What bounds it: HBM. A key costs 4 G flop per 4 bytes, far below the tensor cores' rate even on
// mma.sync (tcgen05's smallest M is 64 rows; here there are 8 heads, and a tile's 16 to 32 keys), so the
// design is about bytes in flight: every consumer warp owns a ring of STAGES tiles in shared memory (24 KB
// a warp, 192 KB an SM, several times the 54 KB an SM needs to cover HBM's latency at full rate), and what
// is not a tile's arithmetic is done by other warps. Four producer warps walk the items, look the pages up
// one round ahead and fill the rings with TMA copies (16 or 32 keys, hardware swizzle, so ldmatrix reads are
// free of bank conflicts; they leave L2 first); the first also sends the items' descriptors and queries.
// Four joiner warps turn e4m3 queries into halves an item ahead, and join the consumers' results while
// these run on. What each step brought, on 64 ragged bf16 rows of up to 8192 keys and 256 e4m3 rows of up
// to 4096 (28 / 4 heads of 128; floors 93 and 90 us at the copy's rate): every warp walking and copying for
// itself 157 and 294 us; producers 111 and 219; joiners, one warp a head in narrow joins, spans of
// 512 110 and 130; queries by the joiners, two heads a joiner 107 and 118; the L2 policy 103 and 116;
// K Q^T 103 and 115; maxima exchanged only when a reference moves 103 and 114; a walk that loads its lengths
// at once and a join whose loads do not wait for one another 102 and 109 (6.2 and 5.6 TB/s); sums that no scale
// takes out of range 102 and 110. One e4m3 row of 131072 keys takes 27 us (floor 20), one bf16 row of 500 7. (Times
// of calls in a replayed graph; from Python that row takes 10.) A KV head's query heads beyond 8 are
// items of their own, which read the tiles again through L2: 64 rows of up to 4096 keys of 2 KV heads take
// 34 and 23 us with 8 heads each, 48 and 35 with 16; items of 16 heads took 41 and 34 there, but 9.6 us
// instead of 6.9 on one row of 500 and up to 13 % more on 12 to 40 rows. What is above the floors now: the
// start (lengths, page table, first tiles one after the other: 3 us), the join (2 us, 5 on 256 rows) and the last
// CTAs' rest. With the products and weights left out, the 256 e4m3 rows take 3 us less and the 64 bf16 rows
// the same. What waits for arithmetic are rows of one or two tiles a warp (256 e4m3 rows of up to 300: 21 us, floor
// 9) and e4m3 heads of 64, whose tiles have half the bytes for the same keys (64 rows of up to 8192 over 8 KV heads:
// 88 us, floor 50; in bf16 102, floor 93).

#include <cuda.h>
#include <cuda_runtime.h>

#include <cfloat>

#include "mot_kvcache.cuh"

namespace mot {
namespace decode {

constexpr int WARPS = 8;                  // consumers
constexpr int PRODUCERS = 4;              // warps 8 .. 11, two consumers each
constexpr int JOINERS = 4;                // warps 12 .. 15, two heads each
constexpr int THREADS = 32 * (WARPS + PRODUCERS + JOINERS);
// Registers of a thread: at launch, then of each kind of warp. The consumers' share waits for what the
// others give up, so the sum has to be the launch's; the host checks the compiled kernel's count.
constexpr int LAUNCH_REGS = 128, CONSUMER_REGS = 160, PRODUCER_REGS = 80, JOINER_REGS = 112;
static_assert(WARPS * CONSUMER_REGS + PRODUCERS * PRODUCER_REGS + JOINERS * JOINER_REGS ==
                  (WARPS + PRODUCERS + JOINERS) * LAUNCH_REGS,
              "register split");
constexpr int ITEMS = 4;                  // item descriptors in flight
constexpr int WINDOW = 256;               // rows whose item counts the producer holds at a time
constexpr int HEADS = 8;      // query heads of an item
constexpr int SPLIT_ITEMS = 152;  // items that one row is cut into, at most: one for each SM
// e4m3: the largest weight, and the largest weight of the tile that sets a reference, as powers of two. bf16: the
// same distance, shifted (see `above` and `below`)
constexpr float kAbove = 14.0f, kBelow = 6.0f;
constexpr float kLoud = 0x1p-17f;  // one over the V scales from which on loud_sums has the sums

template <int D, bool E4M3>
struct Cfg {
  static constexpr int ROW = D * (E4M3 ? 1 : 2);            // bytes of a cached vector
  static constexpr int TOK = ROW == 256 ? 16 : 32;          // keys of a tile: 4 KB of K (2 KB at 64-byte rows)
  static constexpr int KT = TOK * ROW;                      // bytes of a tile's K
  static constexpr int BOX = ROW < 128 ? ROW : 128;         // bytes of a TMA box's row, the swizzle's width
  static constexpr int HALVES = ROW / BOX;                  // boxes across a row
  static constexpr int SC = E4M3 ? TOK * 8 : 0;             // bytes of a tile's scales
  static constexpr int STAGES = KT == 2048 ? 6 : 3;
  static constexpr int ROUND = WARPS * TOK;                 // keys a CTA takes at a time
  static constexpr int MIN_SPAN = 512;                      // shortest range
  static constexpr uint32_t TILES = 0;                      // [WARPS][STAGES][K tile, V tile]
  static constexpr uint32_t SCALES = TILES + WARPS * STAGES * 2 * KT;
  static constexpr uint32_t Q = SCALES + WARPS * STAGES * SC;         // [ITEMS][HEADS][D] bf16
  static constexpr uint32_t ZERO = Q + ITEMS * HEADS * D * 2;         // [HEADS][D] float: the O of a warp without tiles
  static constexpr uint32_t DESC = ZERO + HEADS * D * 4;              // [ITEMS] Item
  static constexpr uint32_t ML = DESC + ITEMS * 32;                   // [2][2][WARPS][HEADS] float
  static constexpr uint32_t QC = ML + 4 * WARPS * HEADS * 4;          // [ITEMS][HEADS] float: c over the query's scale
  static constexpr uint32_t SLOT = QC + ITEMS * HEADS * 4;            // [2][WARPS] the slot that holds a warp's O
  // [PRODUCERS][3][WINDOW]: items up to a row, its length, its span
  static constexpr uint32_t ROWS = SLOT + 2 * WARPS * 4;
  static constexpr uint32_t BARS = ROWS + PRODUCERS * 3 * WINDOW * 4; // full, empty [WARPS][STAGES] each
  // full, empty, qready [ITEMS] each, jfull, jread [2] each
  static constexpr uint32_t IBARS = BARS + 2 * WARPS * STAGES * 8;
  static constexpr uint32_t ABORT = IBARS + (3 * ITEMS + 4) * 8;
  static constexpr size_t BYTES = 1024 + size_t(ABORT) + 16;
  static_assert(HEADS * D * 4 <= KT, "a warp's O fits into a tile's K");
};

struct Args {
  const uint16_t* qkv;   // [R][(Hq + 2 Hkv) D]
  const int32_t* table;  // [R][max_pages]
  const int32_t* lens;   // [R]
  const float* scales;
  const uint8_t* k;      // K as the copies take it
  int64_t n_pages;
  int R, max_pages, page;
  int Hq, Hkv, G;        // G = Hq / Hkv
  int HC;                // groups of up to 8 heads that share a KV head
  int max_split;         // ranges of a row that the workspace has room for
  int box;               // keys of a copy: 16, or 32 where a tile's 32 lie in one page
  kv::Div by_page, by_heads, by_hc, by_most;  // page, Hkv * HC, HC, most ranges of a row
  float c;               // scale * log2(e)
  float2* ml;            // [R][max_split][Hq] (reference, sum) of a range
  float* part;           // [R][max_split][Hq][D]
  uint16_t* out;         // [R][Hq D]
  uint32_t* err;
};

// Ranges that one row is cut into, at most.
inline int most_of(int heads) { return SPLIT_ITEMS / heads > 1 ? SPLIT_ITEMS / heads : 1; }

// How many ranges a row of len keys has, and their keys (an empty row has one empty range, which writes its
// zeros). C: the Cfg.
template <typename C>
__device__ __forceinline__ int ranges_of(const Args& a, int len, int& span) {
  const int each = int(a.by_most.of(uint32_t(len) + a.by_most.d - 1));
  span = (each + C::ROUND - 1) / C::ROUND * C::ROUND;
  if (span <= C::MIN_SPAN) {
    span = C::MIN_SPAN;
    return len == 0 ? 1 : (len + C::MIN_SPAN - 1) / C::MIN_SPAN;
  }
  return (len + span - 1) / span;
}

// ---------------------------------------------------------------------------
// small wrappers
// ---------------------------------------------------------------------------
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool HALF>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if (HALF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// The transposed 8 x 8 matrix of 16-bit elements whose row g lane (g, t) holds columns 2 t, 2 t + 1 of.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %1, %2;" : "=r"(r) : "r"(a), "r"(sel));
  return r;
}

// Rows y .. of an array of vectors, whole: vectors of 256 bytes as two halves of 128, one behind the other
// (a 3D map whose third dimension is the half), the others as one box. `policy`: an L2 cache policy.
template <int HALVES>
__device__ __forceinline__ void tma_load_vectors(uint32_t dst, const void* tmap, int32_t y, uint32_t bar,
                                                 uint64_t policy) {
  if (HALVES == 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, "
        "{%2, %3}], [%4], %5;" ::"r"(dst),
        "l"(tmap), "r"(0), "r"(y), "r"(bar), "l"(policy)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, "
        "{%2, %3, %4}], [%5], %6;" ::"r"(dst),
        "l"(tmap), "r"(0), "r"(y), "r"(0), "r"(bar), "l"(policy)
        : "memory");
}
__device__ __forceinline__ uint64_t policy_evict_first() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint64_t policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// ---------------------------------------------------------------------------
// items
// ---------------------------------------------------------------------------
struct alignas(16) Item {
  int row, g, hc, split;
  int t0, t1;    // keys [t0, t1) of the row
  int split_up;  // the row has more than one range
  int pad;
};
static_assert(sizeof(Item) == 32, "a descriptor is 32 bytes");

// Finds items in ascending order; used by the producer warp, warp-uniform results. The item counts of
// WINDOW rows at a time lie in shared memory, summed up.
template <int D, bool E4M3>
struct Walk {
  using C = Cfg<D, E4M3>;
  int64_t base;  // items of the rows before the window
  int w0, nw;    // the window's first row and its rows
  int hint;      // no row of the window before this one holds an item still to come
  int* upto;     // items of the window's rows up to and with row i
  int* lens;
  int* spans;

  __device__ void load(const Args& a) {
    const int lane = threadIdx.x & 31, heads = a.Hkv * a.HC;
    nw = min(WINDOW, a.R - w0);
    hint = 0;
    // all loads on their way at once, then a lane takes neighbouring rows: one exchange sums up the lanes'
    int len[WINDOW / 32];
#pragma unroll
    for (int k = 0; k < WINDOW / 32; ++k) len[k] = 32 * k + lane < nw ? a.lens[w0 + 32 * k + lane] : 0;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < WINDOW / 32; ++k)
      if (32 * k + lane < nw) lens[32 * k + lane] = len[k];
    __syncwarp();
    const int each = (nw + 31) / 32, first = min(lane * each, nw), last = min(first + each, nw);
    int mine = 0;
    for (int i = first; i < last; ++i) {
      const int n = lens[i];
      if (n < 0 || n > int64_t(a.max_pages) * a.page) {
        if (blockIdx.x == 0 && threadIdx.x / 32 == WARPS) atomicOr(a.err, MOT_DEV_BAD_PAGE);
      } else {
        int span;
        mine += ranges_of<C>(a, n, span) * heads;
        spans[i] = span;
      }
      upto[i] = mine;
    }
    int before = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, before, off);
      if (lane >= off) before += o;
    }
    before -= mine;
    for (int i = first; i < last; ++i) upto[i] += before;
    __syncwarp();
  }
  __device__ void init(const Args& a, int* rows) {
    base = 0;
    w0 = 0;
    upto = rows;
    lens = rows + WINDOW;
    spans = lens + WINDOW;
    load(a);
  }
  __device__ bool find(const Args& a, int64_t it, Item& m) {
    while (it >= base + upto[nw - 1]) {
      if (w0 + nw >= a.R) return false;
      base += upto[nw - 1];
      w0 += nw;
      load(a);
    }
    const int lane = threadIdx.x & 31, k = int(it - base);
    uint32_t hit;
    while ((hit = __ballot_sync(0xffffffffu, hint + lane < nw && upto[min(hint + lane, nw - 1)] > k)) == 0u) hint += 32;
    hint += __ffs(hit) - 1;
    const int first = hint > 0 ? upto[hint - 1] : 0, span = spans[hint], nk = lens[hint];
    const int local = k - first;
    m.row = w0 + hint;
    m.split = int(a.by_heads.of(local));
    const int hh = local - m.split * int(a.by_heads.d);
    m.g = int(a.by_hc.of(hh));
    m.hc = hh - m.g * a.HC;
    m.split_up = (upto[hint] - first) > int(a.by_heads.d);
    m.t0 = m.split * span;
    m.t1 = m.t0 + span < nk ? m.t0 + span : nk;
    return true;
  }
};

// Shared-memory offset of the 16-byte chunk c of row r in a tile (the TMA's swizzle).
template <int D, bool E4M3>
__device__ __forceinline__ uint32_t chunk(int r, int c) {
  using C = Cfg<D, E4M3>;
  if (C::BOX == 64) return uint32_t(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
  // boxes of 16 rows, one behind the other per 16 keys: [16-key block][half][16 rows][128 bytes]
  return uint32_t(((r >> 4) * C::HALVES + (c >> 3)) * 2048 + (r & 15) * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// The sums of a warp's weights in an item of an e4m3 cache from the scores alone: for each head the sum of
// 2^score. A lane takes a tile's key; K comes from memory again, the queries (halves, [half][8 heads][128 bytes],
// swizzled) and their factors from shared memory. refs, sums and o (the warp's references, sums and O, [HEADS][D])
// become e, the sum over 2^e, in [1/2, 1), and O under 2^e: then O is the warp's own output times that number, so in
// range wherever the values are. It stands beside the loop, for values that no model has, because there a second
// exponential a weight, or a vote a tile, cost every row time: 256 rows of up to 4096 keys took 113.3 or 111.4 us, 256
// of up to 300 23.4 or 22.2; with the sums' one reference alone they take 110.0 and 20.6, with this 110.3 and 21.3.
// Loud rows take up to five times theirs (537 us a call instead of 122; 5.9 us a round of 256 keys, which is 0.4 s in
// a range of 2^24 keys, while a wait is given up after one).
template <int D>
__device__ __forceinline__ void loud_sums(const Args& a, int row, int g, int t0, int t1, const uint8_t* q,
                                          const float* qc, float* refs, float* sums, float* o) {
  using C = Cfg<D, true>;
  static_assert(C::TOK == 32, "a lane for each key of a tile");
  const int lane = threadIdx.x & 31;
  float top[HEADS], sum[HEADS];  // a lane's references, moved as the tiles' are, and sums
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    top[h] = -INFINITY;
    sum[h] = 0.0f;
  }
#pragma unroll 1
  for (int key = t0 + lane; key < t1; key += C::ROUND) {
    const int nth = a.by_page.of(key), at = key - nth * a.page;
    int page = a.table[int64_t(row) * a.max_pages + nth];
    if (page < 0 || page >= a.n_pages) page = 0;  // reported where it was copied
    const int64_t y = (int64_t(page) * a.Hkv + g) * a.page + at;
    const float scale = a.scales[2 * y];
    const uint2* codes = reinterpret_cast<const uint2*>(a.k + y * D);
    uint2 u = codes[0];
    float x[HEADS] = {};
#pragma unroll 1
    for (int c = 0; c < D / 8; ++c) {
      const float2 k[4] = {kv::h2_to_f2(kv::e4m3x2_to_h2(u.x & 0xFFFFu)), kv::h2_to_f2(kv::e4m3x2_to_h2(u.x >> 16)),
                           kv::h2_to_f2(kv::e4m3x2_to_h2(u.y & 0xFFFFu)), kv::h2_to_f2(kv::e4m3x2_to_h2(u.y >> 16))};
      if (c + 1 < D / 8) u = codes[c + 1];
#pragma unroll
      for (int h = 0; h < HEADS; ++h) {
        const uint4 w = *reinterpret_cast<const uint4*>(q + (c >> 3) * 1024 + h * 128 + (((c & 7) ^ h) << 4));
        const uint32_t e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = kv::h2_to_f2(e[i]);  // a half times a code is exact: one rounding an addition
          x[h] = __fmaf_rn(k[i].y, f.y, __fmaf_rn(k[i].x, f.x, x[h]));
        }
      }
    }
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
      const float s = __fmul_rn(x[h], __fmul_rn(qc[h], scale));
      if (s > __fadd_rn(top[h], kAbove)) {
        const float next = __fsub_rn(s, kBelow);
        sum[h] = __fmul_rn(sum[h], top[h] == -INFINITY ? 0.0f : exp2f(__fsub_rn(top[h], next)));
        top[h] = next;
      }
      sum[h] = __fadd_rn(sum[h], exp2f(top[h] == -INFINITY ? s : __fsub_rn(s, top[h])));
    }
  }
  __syncwarp();
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    float t = top[h];
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, off));
    float v = top[h] == -INFINITY ? sum[h] : __fmul_rn(sum[h], exp2f(__fsub_rn(top[h], t)));
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, off));
    const uint32_t u = __float_as_uint(v);
    const float e = __fadd_rn(t, __fsub_rn(__uint_as_float((u >> 23) | 0x4B000000u), 8388734.0f));  // 2^23 + 126
    // O 2^(its reference - e), as a root twice: the power may lie outside fp32's range
    const float ref = refs[h];
    const float root = ref == -INFINITY || t == -INFINITY ? 0.0f : exp2f(__fmul_rn(0.5f, __fsub_rn(ref, e)));
#pragma unroll
    for (int d = 0; d < D; d += 32) o[h * D + d + lane] = __fmul_rn(__fmul_rn(o[h * D + d + lane], root), root);
    __syncwarp();
    if (lane == 0) {
      refs[h] = e;
      sums[h] = __fmul_rn(v, __uint_as_float(0x7E800000u - (u & 0x7F800000u)));
    }
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(THREADS, 1)
    decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ CUtensorMap tm_q, const Args a) {
  using C = Cfg<D, E4M3>;
  constexpr int TOK = C::TOK, NB = TOK / 16, KS = D / 16, STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, t4 = lane & 3;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BARS);   // [WARPS][STAGES] full, then empty
  uint64_t* ifull = reinterpret_cast<uint64_t*>(smem + C::IBARS);
  uint64_t* iempty = ifull + ITEMS;
  uint64_t* qready = iempty + ITEMS;  // e4m3: the queries are halves now
  uint64_t* jfull = qready + ITEMS;  // the consumers' results of an item are there (by the item's parity)
  uint64_t* jread = jfull + 2;       // and have been read
  Item* desc = reinterpret_cast<Item*>(smem + C::DESC);
  float* s_ref = reinterpret_cast<float*>(smem + C::ML);
  float* s_sum = s_ref + 2 * WARPS * HEADS;
  float* s_qc = reinterpret_cast<float*>(smem + C::QC);
  int* s_slot = reinterpret_cast<int*>(smem + C::SLOT);
  volatile uint32_t* abort_flag = reinterpret_cast<uint32_t*>(smem + C::ABORT);

  {
    // a barrier a thread
    const int i = int(threadIdx.x), n = 2 * WARPS * STAGES;
    if (i < n) mbar_init(smem_u32(&bars[i]), 1);
    else if (i < n + ITEMS) mbar_init(smem_u32(&ifull[i - n]), 1);
    else if (i < n + 2 * ITEMS) mbar_init(smem_u32(&iempty[i - n - ITEMS]), WARPS + JOINERS);
    else if (i < n + 3 * ITEMS) mbar_init(smem_u32(&qready[i - n - 2 * ITEMS]), JOINERS);
    else if (i < n + 3 * ITEMS + 2) mbar_init(smem_u32(&jfull[i - n - 3 * ITEMS]), WARPS);
    else if (i < n + 3 * ITEMS + 4) mbar_init(smem_u32(&jread[i - n - 3 * ITEMS - 2]), JOINERS);
    if (i < n + 3 * ITEMS + 4) fence_mbar_init();
    static_assert(n + 3 * ITEMS + 4 < THREADS, "a thread for each barrier");
  }
  for (int i = int(threadIdx.x); i < HEADS * D / 4; i += THREADS)
    reinterpret_cast<float4*>(smem + C::ZERO)[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (threadIdx.x == THREADS - 1) {
    *abort_flag = 0u;
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_q);
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();

  if (warp >= WARPS && warp < WARPS + PRODUCERS) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PRODUCER_REGS));
    // ---------------- producers: a lane for each copy's keys of the two tiles that a warp copies ----------------
    const int pw = warp - WARPS;
    const int per = TOK / a.box;  // copies of a tile: 1 or 2
    const int cw = (WARPS / PRODUCERS) * pw + (per == 2 ? lane >> 1 : lane), sub = per == 2 ? lane & 1 : 0;
    const bool works = lane < (WARPS / PRODUCERS) * per;  // whose tile, which copy of it
    uint64_t* full = bars + cw * STAGES;
    uint64_t* empty = full + WARPS * STAGES;
    uint8_t* ring = smem + C::TILES + cw * STAGES * 2 * C::KT;
    uint8_t* ring_sc = smem + C::SCALES + cw * STAGES * C::SC;
    Walk<D, E4M3> walk;
    walk.init(a, reinterpret_cast<int*>(smem + C::ROWS) + pw * 3 * WINDOW);
    // K and V pass through once (unless several groups of heads share them): they leave L2 first, and the
    // partial results, the page tables and the kernels' own instructions stay
    const uint64_t keep = policy_evict_normal(), stream = a.HC == 1 ? policy_evict_first() : keep;
    int issued = 0, items = 0;  // tiles of warp cw, items
    bool ok = true;
    int64_t it = blockIdx.x;
    Item m{}, nx{};
    bool more = walk.find(a, it, m);
    int r0 = m.t0;  // the round's first key
    auto lookup = [&](const Item& w, int first) {  // the page of this lane's keys
      const int key = first + cw * TOK + a.box * sub;
      return works && key < w.t1 ? __ldg(a.table + int64_t(w.row) * a.max_pages + a.by_page.of(key)) : 0;
    };
    int pg = more ? lookup(m, r0) : 0;
    while (more) {
      // the round after this one, its lookup on the way while this one's copies go out
      bool nmore = true;
      int n0 = r0 + C::ROUND;
      nx = m;
      if (n0 >= m.t1) {
        it += gridDim.x;
        nmore = walk.find(a, it, nx);
        n0 = nx.t0;
      }
      const int npg = nmore ? lookup(nx, n0) : 0;

      if (pw == 0 && r0 == m.t0) {
        // a new item: its descriptor and its queries
        const int is = items % ITEMS;
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&iempty[is]), (uint32_t(items / ITEMS) & 1u) ^ 1u, abort_flag,
                                               a.err));
        if (!ok) break;
        if (lane == 0) {
          desc[is] = m;
          const int h0 = m.g * a.G + m.hc * HEADS;
          // 8 heads whatever the group has: the rows behind are not used
          mbar_arrive_expect_tx(smem_u32(&ifull[is]), HEADS * D * 2);
          tma_load_vectors<D / 64>(smem_u32(smem + C::Q + is * HEADS * D * 2), &tm_q,
                                   m.row * (a.Hq + 2 * a.Hkv) + h0, smem_u32(&ifull[is]), keep);
        }
        ++items;
        __syncwarp();
      }
      const int tile = r0 + cw * TOK;
      if (works && tile < m.t1) {
        const int st = issued % STAGES;
        const uint32_t bar = smem_u32(&full[st]);
        ok = mbar_wait(smem_u32(&empty[st]), (uint32_t(issued / STAGES) & 1u) ^ 1u, abort_flag, a.err);
        if (ok) {
          const int copies = m.t1 - tile > a.box ? per : 1;
          if (sub == 0) mbar_arrive_expect_tx(bar, copies * a.box * (2 * C::ROW + (E4M3 ? 8 : 0)));
          if (sub < copies) {
            int page = pg;
            if (page < 0 || page >= a.n_pages) {
              atomicOr(a.err, MOT_DEV_BAD_PAGE);
              page = 0;
            }
            const int key = tile + a.box * sub;
            const int y = (page * a.Hkv + m.g) * a.page + (key - int(a.by_page.of(key)) * a.page);
            const uint32_t dst = smem_u32(ring + st * 2 * C::KT) + sub * (16 * C::ROW);
            tma_load_vectors<C::HALVES>(dst, &tm_k, y, bar, stream);
            if (E4M3) bulk_load(smem_u32(ring_sc + st * C::SC) + sub * 128, a.scales + 2 * int64_t(y), a.box * 8, bar);
            tma_load_vectors<C::HALVES>(dst + C::KT, &tm_v, y, bar, stream);
          }
          ++issued;
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      more = nmore;
      m = nx;
      r0 = n0;
      pg = npg;
    }
    if (ok && pw == 0) {
      // no more items
      const int is = items % ITEMS;
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&iempty[is]), (uint32_t(items / ITEMS) & 1u) ^ 1u, abort_flag,
                                             a.err));
      if (ok) {
        if (lane == 0) {
          desc[is].row = -1;
          mbar_arrive(smem_u32(&ifull[is]));
        }
        ++items;
      }
    }
    // every copy has landed before the CTA can exit: the last phase of each slot
    if (works)
      for (int i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i)
        mbar_drain(smem_u32(&full[i % STAGES]), uint32_t(i / STAGES) & 1u);
    for (int i = items > ITEMS ? items - ITEMS : 0; i < items; ++i)
      mbar_drain(smem_u32(&ifull[i % ITEMS]), uint32_t(i / ITEMS) & 1u);
    return;
  }

  if (warp >= WARPS + PRODUCERS) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(JOINER_REGS));
    // ---------------- joiners: half a warp a head, the consumers' results in warp order ----------------
    // The two heads of a warp share every instruction: this code runs once an item, from cold instruction
    // caches, so its length is its time (a head after the other it took 3400 cycles an item, and the
    // joiners were what bounded the e4m3 cache).
    static_assert(HEADS == 2 * JOINERS, "a joiner's halves");
    constexpr int P = D / 64;  // pieces of 4 dims of a lane: 64 i + 4 l16
    const int jw = warp - WARPS - PRODUCERS, l16 = lane & 15, hd = 2 * jw + (lane >> 4);
    // e4m3: the queries of item i become halves, each head scaled by a power of two that takes its largest
    // element into [2^14, 2^15) (exact but for elements below 2^-24 of it); false after a wait that gave up
    auto convert = [&](int i) -> bool {
      const int is = i % ITEMS;
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&ifull[is]), uint32_t(i / ITEMS) & 1u, abort_flag, a.err)))
        return false;
      if (desc[is].row >= 0) {
        // in place: [half][8 heads][128 bytes] with the 128-byte swizzle, 16 bytes of a vector a lane (D = 64: 8)
        const uint32_t byte = (D / 16) * l16 * 2;
        uint32_t* at = reinterpret_cast<uint32_t*>(smem + C::Q + is * HEADS * D * 2 + (byte >> 7) * 1024 + hd * 128 +
                                                   ((((byte >> 4) & 7) ^ hd) << 4) + (byte & 15));
        uint32_t w[D / 32], top2 = 0;
        if constexpr (D == 128) {
          const uint4 u = *reinterpret_cast<const uint4*>(at);
          w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(at);
          w[0] = u.x; w[1] = u.y;
        }
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
          top2 = __vmaxu2(top2, w[k] & 0x7FFF7FFFu);  // magnitudes by their bits: infinities above, then NaNs
        uint32_t top = max(top2 << 16, top2 & 0xFFFF0000u);
#pragma unroll
        for (int off = 8; off >= 1; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
        const int e = min(14 - (int(top >> 23) - 127), 100);
        const float f = __uint_as_float(uint32_t(e + 127) << 23);
#pragma unroll
        for (int k = 0; k < D / 32; ++k) w[k] = pack_h2(__fmul_rn(bf_lo(w[k]), f), __fmul_rn(bf_hi(w[k]), f));
        if constexpr (D == 128) *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
        if (l16 == 0) s_qc[is * HEADS + hd] = __fmul_rn(a.c, __uint_as_float(uint32_t(127 - e) << 23));
      }
      fence_proxy_async_smem();  // the place goes back to the copies
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&qready[is]));
      return true;
    };
    if (E4M3 && !convert(0)) return;
    for (int item = 0;; ++item) {
      const int is = item % ITEMS, par = item & 1;
      const uint32_t phase = uint32_t(item / 2) & 1u;
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&ifull[is]), uint32_t(item / ITEMS) & 1u, abort_flag, a.err)))
        return;
      const Item m = desc[is];
      if (m.row < 0) return;
      if (E4M3 && !convert(item + 1)) return;
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&jfull[par]), phase, abort_flag, a.err))) return;
      const int nh = min(HEADS, a.G - m.hc * HEADS);
      const int st = lane < WARPS ? s_slot[par * WARPS + lane] : -1;
      const uint32_t off = st >= 0 ? C::TILES + ((lane & 7) * STAGES + st) * 2 * C::KT : C::ZERO;
      float4 v[WARPS][P];
#pragma unroll
      for (int k = 0; k < WARPS; ++k) {
        const float* src = reinterpret_cast<const float*>(smem + __shfl_sync(0xffffffffu, off, k)) + hd * D;
#pragma unroll
        for (int i = 0; i < P; ++i) v[k][i] = *reinterpret_cast<const float4*>(src + ((64 * i + 4 * l16) ^ (8 * (hd >> 1))));
      }
      // lane k of 8 has warp k's reference and sum: one exponential each, the factors go round by shuffles
      const float ref = s_ref[(par * WARPS + (lane & 7)) * HEADS + hd], sum = s_sum[(par * WARPS + (lane & 7)) * HEADS + hd];
      float top = ref;
#pragma unroll
      for (int o = 4; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      // a warp without tiles has -inf here, and zeros; one whose scores are all -inf (or NaN) a sum of zero (or NaN)
      // (2^-3: the O of eight warps then add up to less than the largest, see loud_sums)
      if constexpr (E4M3) top = __fadd_rn(top, 3.0f);
      const bool none = ref == -INFINITY;
      const float f = none ? 0.0f : exp2f(__fsub_rn(ref, top));
      float total = none ? sum : __fmul_rn(sum, f);
#pragma unroll
      for (int o = 4; o >= 1; o >>= 1) total = __fadd_rn(total, __shfl_xor_sync(0xffffffffu, total, o));
      float acc[P][4] = {};
#pragma unroll
      for (int k = 0; k < WARPS; ++k) {
        const float fk = __shfl_sync(0xffffffffu, f, (lane & 16) + k);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          acc[i][0] = __fadd_rn(acc[i][0], __fmul_rn(v[k][i].x, fk));
          acc[i][1] = __fadd_rn(acc[i][1], __fmul_rn(v[k][i].y, fk));
          acc[i][2] = __fadd_rn(acc[i][2], __fmul_rn(v[k][i].z, fk));
          acc[i][3] = __fadd_rn(acc[i][3], __fmul_rn(v[k][i].w, fk));
        }
      }
      if (hd < nh) {
        const int head = m.g * a.G + m.hc * HEADS + hd;
        if (!m.split_up) {
          const float r = total == 0.0f ? 0.0f : __fdiv_rn(1.0f, total);
          uint16_t* dst = a.out + (int64_t(m.row) * a.Hq + head) * D + 4 * l16;
#pragma unroll
          for (int i = 0; i < P; ++i)
            *reinterpret_cast<uint2*>(dst + 64 * i) = make_uint2(pack_bf2(__fmul_rn(acc[i][0], r), __fmul_rn(acc[i][1], r)),
                                                                 pack_bf2(__fmul_rn(acc[i][2], r), __fmul_rn(acc[i][3], r)));
        } else {
          const int64_t at = (int64_t(m.row) * a.max_split + m.split) * a.Hq + head;
          float* dst = a.part + at * D + 4 * l16;
#pragma unroll
          for (int i = 0; i < P; ++i)
            *reinterpret_cast<float4*>(dst + 64 * i) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
          if (l16 == 0) a.ml[at] = make_float2(top, total);
        }
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(&jread[par]));
        mbar_arrive(smem_u32(&iempty[is]));
      }
      if (jw == 0) {
        // the slots that O came in go back to the copies when every joiner has read them
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&jread[par]), phase, abort_flag, a.err))) return;
        fence_proxy_async_smem();
        if (st >= 0) mbar_arrive(smem_u32(&bars[(WARPS + lane) * STAGES + st]));
      }
    }
  }

  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(CONSUMER_REGS));
  // ---------------- consumers ----------------
  uint64_t* full = bars + warp * STAGES;
  uint64_t* empty = full + WARPS * STAGES;
  uint8_t* ring = smem + C::TILES + warp * STAGES * 2 * C::KT;
  uint8_t* ring_sc = smem + C::SCALES + warp * STAGES * C::SC;
  int taken = 0;
  for (int item = 0;; ++item) {
    const int is = item % ITEMS;
    const int par = item & 1;
    if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(E4M3 ? &qready[is] : &ifull[is]), uint32_t(item / ITEMS) & 1u,
                                           abort_flag, a.err)))
      return;
    const Item m = desc[is];
    if (m.row < 0) return;
    // ---- the query fragments: head g8 of the group in row g8, rows 8 .. 15 empty ----
    const int nh = min(HEADS, a.G - m.hc * HEADS);                // heads of this item
    // element pairs of columns 2 t and 2 t + 8 of a k-step: dims 16 s + 2 t and + 8 (bf16), or, as an e4m3
    // lane holds 4 consecutive dims, 16 s + 4 t and + 2
    uint32_t q[KS][2];
    const uint32_t qb = smem_u32(smem + C::Q + is * HEADS * D * 2);  // [half][8 heads][128 bytes], swizzled
    if constexpr (E4M3) {
#pragma unroll
      for (int s = 0; s < KS; ++s)
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                     : "=r"(q[s][0]), "=r"(q[s][1])
                     : "r"(qb + (s >> 2) * 1024 + g8 * 128 + ((((2 * s + (t4 >> 1)) & 7) ^ g8) << 4) + 8 * (t4 & 1))
                     : "memory");
    } else {
#pragma unroll
      for (int s = 0; s < KS; s += 2) {
        uint32_t r[4];
        const int ch = 2 * s + (lane >> 3);
        ldsm4(r, qb + (ch >> 3) * 1024 + (lane & 7) * 128 + (((ch & 7) ^ (lane & 7)) << 4));
        q[s][0] = r[0]; q[s][1] = r[1];
        q[s + 1][0] = r[2]; q[s + 1][1] = r[3];
      }
    }
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i) q[s][i] = g8 < nh ? q[s][i] : 0u;
    float c[2] = {a.c, a.c};
    if constexpr (E4M3) {
      c[0] = s_qc[is * HEADS + 2 * t4];
      c[1] = s_qc[is * HEADS + 2 * t4 + 1];
    }

    float o[D / 16][4];
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;
    // a reference moves when a maximum is more than `above` over it, to `below` under that
    const float above = E4M3 ? kAbove : -float(32 - __clz(m.t1 - m.t0 - 1));
    const float below = above - (kAbove - kBelow);
    float ref[2] = {-INFINITY, -INFINITY}, sum[2] = {0.0f, 0.0f};  // of heads 2 t4 and 2 t4 + 1
    float quiet = 1.0f;  // e4m3: the smallest of one over this lane's keys' V scales
    int slot = -1;  // the slot of the item's last tile, held back: O passes through it

    for (int tile = m.t0 + warp * TOK; tile < m.t1; tile += C::ROUND) {
      if (slot >= 0 && lane == 0) mbar_arrive(smem_u32(&empty[slot]));  // the tile before has been read
      const int st = taken % STAGES;
      slot = st;
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&full[st]), uint32_t(taken / STAGES) & 1u, abort_flag, a.err)))
        return;
      ++taken;
      uint8_t* kt = ring + st * 2 * C::KT;
      const uint32_t kb = smem_u32(kt), vb = kb + C::KT;
      const int nv = min(TOK, m.t1 - tile);  // keys of the tile
      if (nv < TOK) {
        // rows of V behind the last key: whatever the page holds there (or the slot, where no page was
        // copied) must not meet a weight of zero as a NaN
        for (int i = lane; i < (TOK - nv) * (C::ROW / 16); i += 32)
          *reinterpret_cast<uint4*>(kt + C::KT + chunk<D, E4M3>(nv + i / (C::ROW / 16), i % (C::ROW / 16))) =
              make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();  // before a later copy into the slot
        __syncwarp();
      }

      // ---- S^T = K Q^T: lane has keys 16 b + 8 i + g8, heads 2 t4 and 2 t4 + 1 (x[b][2 i], x[b][2 i + 1]) ----
      float x[NB][4];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[b][i] = 0.0f;
      if constexpr (E4M3) {
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          uint32_t r[4];  // 4 dims of a key in each group of 8 keys
          ldsm4(r, kb + chunk<D, E4M3>(lane, s));
#pragma unroll
          for (int b = 0; b < NB; ++b)
            mma16816<true>(x[b], kv::e4m3x2_to_h2(r[2 * b] & 0xFFFFu), kv::e4m3x2_to_h2(r[2 * b + 1] & 0xFFFFu),
                           kv::e4m3x2_to_h2(r[2 * b] >> 16), kv::e4m3x2_to_h2(r[2 * b + 1] >> 16), q[s][0], q[s][1]);
        }
      } else {
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            uint32_t r[4];
            ldsm4(r, kb + chunk<D, E4M3>(16 * b + (lane >> 4) * 8 + (lane & 7), 2 * s + ((lane >> 3) & 1)));
            mma16816<false>(x[b], r[0], r[2], r[1], r[3], q[s][0], q[s][1]);
          }
      }

      // ---- weights ----
      float inv[NB][2], fac[NB][2];  // e4m3: 2^-e and s / 2^e of each key's V scale s, e its exponent
      float tmax[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int key = 16 * b + 8 * i + g8;
          if constexpr (E4M3) {
            const float2 sc = *reinterpret_cast<const float2*>(ring_sc + st * C::SC + key * 8);  // K's, V's
            const uint32_t u = __float_as_uint(sc.y);
            const float ev = __fsub_rn(__uint_as_float((u >> 23) | 0x4B000000u), 8388735.0f);  // 2^23 + 127
            inv[b][i] = __uint_as_float(0x7F000000u - (u & 0x7F800000u));
            fac[b][i] = __fmul_rn(sc.y, inv[b][i]);  // NaN for a scale of NaN
            // the two factors first: either may be near an end of fp32's range where the score is not
#pragma unroll
            for (int h = 0; h < 2; ++h)
              x[b][2 * i + h] = __fadd_rn(__fmul_rn(x[b][2 * i + h], __fmul_rn(c[h], sc.x)), ev);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) x[b][2 * i + h] = __fmul_rn(x[b][2 * i + h], c[h]);
          }
          if (nv < TOK && key >= nv) {
            x[b][2 * i] = x[b][2 * i + 1] = -INFINITY;
            if constexpr (E4M3) {
              inv[b][i] = 1.0f;  // whatever the scale's place holds
              fac[b][i] = 0.0f;
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) tmax[h] = fmaxf(tmax[h], x[b][2 * i + h]);
        }
      if constexpr (E4M3) {
#pragma unroll
        for (int b = 0; b < NB; ++b) quiet = fminf(quiet, fminf(inv[b][0], inv[b][1]));
      }
      // a head's tile maximum is above its reference's slack (also from -inf) if a lane's is: only then do the
      // lanes exchange them
      if (__any_sync(0xffffffffu, tmax[0] > __fadd_rn(ref[0], above) || tmax[1] > __fadd_rn(ref[1], above))) {
#pragma unroll
        for (int off = 4; off <= 16; off <<= 1)
#pragma unroll
          for (int h = 0; h < 2; ++h) tmax[h] = fmaxf(tmax[h], __shfl_xor_sync(0xffffffffu, tmax[h], off));
        if (tile == m.t0 + warp * TOK) {
          // the item's first tile: nothing to scale yet
#pragma unroll
          for (int h = 0; h < 2; ++h) ref[h] = __fsub_rn(tmax[h], below);
        } else {
          float alpha[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const bool moves = tmax[h] > __fadd_rn(ref[h], above);
            const float next = moves ? __fsub_rn(tmax[h], below) : ref[h];
            alpha[h] = moves ? (ref[h] == -INFINITY ? 0.0f : exp2f(__fsub_rn(ref[h], next))) : 1.0f;
            ref[h] = next;
            sum[h] = __fmul_rn(sum[h], alpha[h]);
          }
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[i][k] = __fmul_rn(o[i][k], alpha[k & 1]);
        }
      }
      // no key with a weight yet: every x is -inf
      const float nref[2] = {ref[0] == -INFINITY ? 0.0f : -ref[0], ref[1] == -INFINITY ? 0.0f : -ref[1]};
      // w[2 b + i]: head g8, keys 16 b + 8 i + 2 t4 and + 1 (the transposed 8 x 8 of the lanes' weights)
      uint32_t w[2 * NB], wl[2 * NB];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float w0 = exp2f(__fadd_rn(x[b][2 * i], nref[0])), w1 = exp2f(__fadd_rn(x[b][2 * i + 1], nref[1]));
          if constexpr (E4M3) {
            sum[0] = __fadd_rn(sum[0], __fmul_rn(w0, inv[b][i]));
            sum[1] = __fadd_rn(sum[1], __fmul_rn(w1, inv[b][i]));
            w[2 * b + i] = transpose8(pack_h2(__fmul_rn(w0, fac[b][i]), __fmul_rn(w1, fac[b][i])));
          } else {
            sum[0] = __fadd_rn(sum[0], w0);
            sum[1] = __fadd_rn(sum[1], w1);
            const uint32_t hi = pack_bf2(w0, w1);
            w[2 * b + i] = transpose8(hi);
            wl[2 * b + i] = transpose8(pack_bf2(__fsub_rn(w0, bf_lo(hi)), __fsub_rn(w1, bf_hi(hi))));
          }
        }

      // ---- O^T += V^T W^T: lane has dims g8 and g8 + 8 (e4m3: 2 g8 and 2 g8 + 1) of 16, heads 2 t4, + 1 ----
      if constexpr (E4M3) {
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          uint32_t r[4];
          ldsm4t(r, vb + chunk<D, E4M3>(lane, s));  // pairs of dims of keys 2 t, 2 t + 1 in each 8-key group
#pragma unroll
          for (int i = 0; i < 4; ++i) r[i] = prmt(r[i], 0x3120);
#pragma unroll
          for (int b = 0; b < NB; ++b)
            mma16816<true>(o[s], kv::e4m3x2_to_h2(r[2 * b] & 0xFFFFu), kv::e4m3x2_to_h2(r[2 * b] >> 16),
                           kv::e4m3x2_to_h2(r[2 * b + 1] & 0xFFFFu), kv::e4m3x2_to_h2(r[2 * b + 1] >> 16), w[2 * b],
                           w[2 * b + 1]);
        }
      } else {
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            uint32_t r[4];
            ldsm4t(r, vb + chunk<D, E4M3>(16 * b + (lane >> 4) * 8 + (lane & 7), 2 * s + ((lane >> 3) & 1)));
            mma16816<false>(o[s], r[0], r[1], r[2], r[3], w[2 * b], w[2 * b + 1]);
            mma16816<false>(o[s], r[0], r[1], r[2], r[3], wl[2 * b], wl[2 * b + 1]);
          }
      }
      __syncwarp();  // every lane has read the slot
    }

    // ---- the joiners take it from here: O passes to them through the last tile's slot ----
#pragma unroll
    for (int off = 4; off <= 16; off <<= 1)
#pragma unroll
      for (int h = 0; h < 2; ++h) sum[h] = __fadd_rn(sum[h], __shfl_xor_sync(0xffffffffu, sum[h], off));
    // the item before last has left its place
    if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&jread[par]), (uint32_t(item / 2) & 1u) ^ 1u, abort_flag, a.err)))
      return;
    if (g8 == 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        s_ref[(par * WARPS + warp) * HEADS + 2 * t4 + h] = ref[h];
        s_sum[(par * WARPS + warp) * HEADS + 2 * t4 + h] = sum[h];
      }
    }
    if (slot >= 0) {
      // [head][dim ^ 8 (head / 2)]: the four lanes of a group fall into different banks
      float* ob = reinterpret_cast<float*>(ring + slot * 2 * C::KT);
      const int sw = 8 * t4;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float* ho = ob + (2 * t4 + j) * D;
          if (E4M3) {
            *reinterpret_cast<float2*>(ho + ((16 * i + 2 * g8) ^ sw)) = make_float2(o[i][j], o[i][j + 2]);
          } else {
            ho[(16 * i + g8) ^ sw] = o[i][j];
            ho[(16 * i + g8 + 8) ^ sw] = o[i][j + 2];
          }
        }
    }
    if constexpr (E4M3) {
      if (__builtin_expect(__any_sync(0xffffffffu, quiet <= kLoud), 0)) {
        const int at = (par * WARPS + warp) * HEADS;
        __syncwarp();
        loud_sums<D>(a, m.row, m.g, m.t0 + warp * TOK, m.t1, smem + C::Q + is * HEADS * D * 2, s_qc + is * HEADS,
                     s_ref + at, s_sum + at, reinterpret_cast<float*>(ring + slot * 2 * C::KT));
      }
    }
    if (lane == 0) s_slot[par * WARPS + warp] = slot;
    fence_proxy_async_smem();  // the slot goes back to the copies through the joiners
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(smem_u32(&jfull[par]));
      mbar_arrive(smem_u32(&iempty[is]));
    }
  }
}

// Joins the ranges of a (row, head): out = (sum of f_s O_s) / (sum of f_s l_s), f_s the factor of range s
// under the largest reference, times 2^-9: less than 2^8 ranges' O then add up to less than the largest, which
// may be at the end of fp32's range. The order is fixed: the f l of 32 ranges at a time by a
// butterfly, these sums in order; the f O of the ranges s, s + 8, ... in order from zero, then the eight sums in
// order.
// Two forms with the same bits: a warp for each 64 dims of a (row, head), the eight sums in its registers, or
// (kWide) a CTA a (row, head) and a warp each sum, which reads all ranges at once but starts more threads.
// Rows of one range were written by decode_kernel.
constexpr int NARROW_WARPS = 4;
constexpr int MOST_WIDE = 256;  // ranges that the wide form can take

// Which form: the wide one pays while its CTAs are few for the ranges that there are to read one after the
// other. Wide against narrow: a bf16 row of 20000 keys over 8 KV heads twice (19 ranges at most, 64 heads) 29.5
// against 31.6 us, 20 e4m3 rows of up to 14000 (28, 560) 39.6 and 43.4, 16 of up to 8000 (16, 448) 19.0 and 20.5,
// 42 of these (16, 1176) 40.8 and 40.6, 40 of up to 5000 (10, 1120) 28.4 and 27.5, 33 of up to 1500 (3, 132)
// 8.0 and 7.5. Tables are often wider than their rows, so more than 16 ranges move the border no further: 64
// e4m3 rows of up to 700 with a table for 131072 (38, 1792) take 17.5 us with the wide form and 16.0 with the
// narrow one.
inline bool wide_join(int64_t heads, int max_split, int sms) {
  return max_split > 4 && heads <= int64_t(sms) * (max_split < 16 ? max_split : 16) / 2;
}

// L consecutive floats of a range's vector, zeros for a range that does not exist.
template <int L>
__device__ __forceinline__ void load_part(float (&v)[L], const float* src, bool there) {
#pragma unroll
  for (int i = 0; i < L; ++i) v[i] = 0.0f;
  if (there) {
    if constexpr (L == 4) {
      const float4 u = __ldcg(reinterpret_cast<const float4*>(src));
      v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    } else {
      const float2 u = __ldcg(reinterpret_cast<const float2*>(src));
      v[0] = u.x; v[1] = u.y;
    }
  }
}

template <int D, bool E4M3, bool kWide>
__global__ void __launch_bounds__(kWide ? MOST_WIDE : 32 * NARROW_WARPS) join_kernel(const Args a) {
  constexpr int L = kWide ? D / 32 : 2;               // dims of a lane
  constexpr int PER = kWide ? 1 : D / 64;             // warps of a (row, head)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t unit = kWide ? blockIdx.x : blockIdx.x * NARROW_WARPS + warp, rh = unit / PER;
  const int row = int(rh / uint32_t(a.Hq)), head = int(rh - uint32_t(row) * uint32_t(a.Hq));
  // the lengths are the call's inputs: there before decode_kernel began
  const int len = row < a.R ? a.lens[row] : 0;
  const int64_t at0 = int64_t(row) * a.max_split * a.Hq + head;
  // thread (narrow: lane) s has range s
  const int mine = kWide ? int(threadIdx.x) : lane;
  pdl_wait();
  pdl_trigger();  // what comes next may start up under this grid
  // on its way beside the length: the workspace has the place whether the row has the range or not
  float2 ml = make_float2(-INFINITY, 0.0f);
  if (row < a.R && mine < a.max_split) ml = __ldcg(a.ml + at0 + int64_t(mine) * a.Hq);
  int n = 0, span;
  if (len > 0 && len <= int64_t(a.max_pages) * a.page) n = ranges_of<Cfg<D, E4M3>>(a, len, span);
  if (n <= 1) return;
  if (mine >= n) ml = make_float2(-INFINITY, 0.0f);
  // O of NV ranges at a time; kWide: of the ranges warp, warp + 8, ..., the first on their way while the factors
  // are made (one bf16 row of 32768 keys 18.0 -> 16.3 us, with 4 at a time 16.9; the narrow form gains nothing)
  constexpr int NV = 8;
  const int64_t step = int64_t(a.Hq) * D;
  const float* base = a.part + at0 * D + (kWide ? 0 : 64 * (unit - rh * PER)) + L * lane;
  float v[NV][L];
  if constexpr (kWide) {
#pragma unroll
    for (int k = 0; k < NV; ++k) load_part(v[k], base + (warp + 8 * k) * step, warp + 8 * k < n);
  }
  float top = ml.x;
  if constexpr (!kWide)
    for (int s = lane + 32; s < n; s += 32) top = fmaxf(top, __ldcg(a.ml + at0 + int64_t(s) * a.Hq).x);
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  __shared__ float s_top[8], s_total[8], s_f[kWide ? MOST_WIDE : 1];
  if constexpr (kWide) {
    if (lane == 0) s_top[warp] = top;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) top = fmaxf(top, s_top[k]);
  }
  static_assert(MOST_WIDE <= 256, "the factors' sum");
  top = __fadd_rn(top, 9.0f);
  // the factor of this thread's range and 32 ranges' sum; a range without a weight has -inf here, and a sum of
  // zero (or NaN: kept)
  float f, total;
  auto factor = [&]() {
    const bool none = ml.x == -INFINITY;
    f = none ? 0.0f : exp2f(__fsub_rn(ml.x, top));
    float sum = none ? ml.y : __fmul_rn(ml.y, f);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, off));
    return sum;
  };
  total = factor();
  if constexpr (kWide) {
    s_f[threadIdx.x] = f;
    if (lane == 0) s_total[warp] = total;
    __syncthreads();
    total = s_total[0];
#pragma unroll
    for (int k = 1; k < 8; ++k) total = __fadd_rn(total, s_total[k]);
    const float r = total == 0.0f ? 0.0f : __fdiv_rn(1.0f, total);
    __shared__ float s_acc[8][D];
    float acc[L];
#pragma unroll
    for (int e = 0; e < L; ++e) acc[e] = 0.0f;
#pragma unroll 1
    for (int s0 = warp; s0 < n; s0 += 8 * NV) {
      if (s0 != warp) {
#pragma unroll
        for (int u = 0; u < NV; ++u) load_part(v[u], base + (s0 + 8 * u) * step, s0 + 8 * u < n);
      }
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        const float fs = s_f[s0 + 8 * u];  // zero behind the last range
#pragma unroll
        for (int e = 0; e < L; ++e) acc[e] = __fadd_rn(acc[e], __fmul_rn(v[u][e], fs));
      }
    }
#pragma unroll
    for (int e = 0; e < L; ++e) s_acc[warp][L * lane + e] = acc[e];
    __syncthreads();
    if (threadIdx.x < D) {
      float v = s_acc[0][threadIdx.x];
#pragma unroll
      for (int k = 1; k < 8; ++k) v = __fadd_rn(v, s_acc[k][threadIdx.x]);
      a.out[int64_t(rh) * D + threadIdx.x] = f_to_bf(__fmul_rn(v, r));
    }
  } else {
    float acc[8][L];
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int e = 0; e < L; ++e) acc[k][e] = 0.0f;
#pragma unroll 1
    for (int s0 = 0; s0 < n; s0 += 8) {
      if (s0 > 0 && s0 % 32 == 0) {
        ml = s0 + lane < n ? __ldcg(a.ml + at0 + int64_t(s0 + lane) * a.Hq) : make_float2(-INFINITY, 0.0f);
        total = __fadd_rn(total, factor());
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) load_part(v[k], base + (s0 + k) * step, s0 + k < n);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float fs = __shfl_sync(0xffffffffu, f, (s0 + k) % 32);
#pragma unroll
        for (int e = 0; e < L; ++e) acc[k][e] = __fadd_rn(acc[k][e], __fmul_rn(v[k][e], fs));
      }
    }
#pragma unroll
    for (int k = 1; k < 8; ++k)
#pragma unroll
      for (int e = 0; e < L; ++e) acc[0][e] = __fadd_rn(acc[0][e], acc[k][e]);
    const float r = total == 0.0f ? 0.0f : __fdiv_rn(1.0f, total);
    reinterpret_cast<uint32_t*>(a.out + int64_t(rh) * D)[32 * (unit - rh * PER) + lane] =
        pack_bf2(__fmul_rn(acc[0][0], r), __fmul_rn(acc[0][1], r));
  }
}

// Ranges that a row can have when its table holds max_len keys.
template <int D, bool E4M3>
inline int max_split(int64_t max_len, int heads) {
  static_assert(SPLIT_ITEMS <= MOST_WIDE, "a thread of the wide join for each range");
  const int most = most_of(heads);
  const int64_t n = (max_len + Cfg<D, E4M3>::MIN_SPAN - 1) / Cfg<D, E4M3>::MIN_SPAN;
  return n < most ? int(n) : most;
}

// Map of vectors [rows][D] in boxes of box_rows whole vectors, for tma_load_vectors.
inline bool vector_map(CUtensorMap* m, const void* base, int D, bool e4m3, int64_t rows, uint32_t box_rows) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (enc == nullptr) return false;
  const int size = e4m3 ? 1 : 2, bytes = D * size, box_bytes = bytes < 128 ? bytes : 128;
  cuuint64_t dims[3] = {cuuint64_t(box_bytes / size), cuuint64_t(rows), 2};
  cuuint64_t strides[2] = {cuuint64_t(bytes), 128};
  cuuint32_t box[3] = {cuuint32_t(box_bytes / size), box_rows, 2};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, bytes == 256 ? 3 : 2,
             const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool E4M3>
static int launch(Args a, const void* k, const void* v, int dev, cudaStream_t s) {
  using C = Cfg<D, E4M3>;
  const int heads = a.Hkv * a.HC;
  a.max_split = max_split<D, E4M3>(int64_t(a.max_pages) * a.page, heads);
  a.part = reinterpret_cast<float*>(a.ml + (int64_t(a.R) * a.max_split * a.Hq + 1) / 2 * 2);
  CUtensorMap tm_k, tm_v, tm_q;
  const int64_t rows = a.n_pages * a.Hkv * a.page;
  a.box = C::TOK == 32 && a.page % 32 == 0 ? 32 : 16;
  a.by_page = kv::Div(a.page);
  a.by_heads = kv::Div(heads);
  a.by_hc = kv::Div(a.HC);
  a.by_most = kv::Div(most_of(heads));
  if (!vector_map(&tm_k, k, D, E4M3, rows, a.box) || !vector_map(&tm_v, v, D, E4M3, rows, a.box) ||
      !vector_map(&tm_q, a.qkv, D, false, int64_t(a.R) * (a.Hq + 2 * a.Hkv), HEADS))
    return MOT_ERR_CUDA;
  if (cudaFuncSetAttribute(decode_kernel<D, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(C::BYTES)) !=
      cudaSuccess)
    return MOT_ERR_CUDA;
  static std::atomic<int> regs{0};
  if (regs.load() == 0) {
    cudaFuncAttributes attr;
    if (cudaFuncGetAttributes(&attr, decode_kernel<D, E4M3>) != cudaSuccess) return MOT_ERR_CUDA;
    regs.store(attr.numRegs);
  }
  if (regs.load() != LAUNCH_REGS) return MOT_ERR_CUDA;
  const int64_t items = int64_t(a.R) * a.max_split * heads;
  const unsigned grid = unsigned(items < sm_count(dev) ? items : sm_count(dev));
  if (launch_dependent(decode_kernel<D, E4M3>, dim3(grid), dim3(THREADS), C::BYTES, s, tm_k, tm_v, tm_q, a) !=
      cudaSuccess)
    return MOT_ERR_CUDA;
  if (a.max_split > 1) {
    const int64_t heads_total = int64_t(a.R) * a.Hq, warps = heads_total * (D / 64);
    const cudaError_t e =
        wide_join(heads_total, a.max_split, sm_count(dev))
            ? launch_dependent(join_kernel<D, E4M3, true>, dim3(unsigned(heads_total)), dim3(MOST_WIDE), 0, s, a)
            : launch_dependent(join_kernel<D, E4M3, false>, dim3(unsigned((warps + NARROW_WARPS - 1) / NARROW_WARPS)),
                               dim3(32 * NARROW_WARPS), 0, s, a);
    if (e != cudaSuccess) return MOT_ERR_CUDA;
  }
  return MOT_OK;
}

}  // namespace decode
}  // namespace mot

using namespace mot;

extern "C" size_t mot_paged_decode_workspace_bytes(int64_t R, int Hq, int Hkv, int D, int max_pages, int page) {
  if (kv::check_shape(Hq, Hkv, D, MOT_KV_BF16, 1, page) != MOT_OK) return 0;
  // with more than 76 (KV head, group of 8 heads) pairs a row is one range, which the joiners wait for: by the times of
  // one row of 2^18 keys, 2^24 take 0.2 s (bf16, 1.5 us a round of 128 at HBM's rate) or 0.4 s (loud e4m3 scales, 5.9 us
  // a round of 256), against the 1 s after which a wait is given up
  if (R < 1 || R > MOT_MAX_TOKENS || max_pages < 1 || int64_t(max_pages) * page > (int64_t(1) << 24)) return 0;
  if (R * (Hq + 2 * Hkv) > (int64_t(1) << 31) - 1) return 0;  // head vectors have 32-bit TMA coordinates
  const int G = Hq / Hkv, heads = Hkv * ((G + decode::HEADS - 1) / decode::HEADS);
  const int64_t n = D == 64 ? decode::max_split<64, false>(int64_t(max_pages) * page, heads)
                            : decode::max_split<128, false>(int64_t(max_pages) * page, heads);
  // a (reference, sum) pair and D floats for each range of each (row, head), unless no row is split
  const int64_t parts = n > 1 ? R * n * Hq : 0;
  return sizeof(PlanHeader) + size_t((parts * 8 + 15) / 16 * 16) + size_t(parts) * D * 4;
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
  if (need == 0) return MOT_ERR_GEOMETRY;
  const float c = scale * 1.4426950408889634f;
  if (!(scale > 0.0f) || !(c <= FLT_MAX)) return MOT_ERR_ARG;
  if (!aligned16(qkv) || !kv::aligned4(table) || !kv::aligned4(lens) || !aligned16(k_cache) || !aligned16(v_cache) ||
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
  a.scales = scales;
  a.k = static_cast<const uint8_t*>(k_cache);
  a.n_pages = n_pages;
  a.R = int(R);
  a.max_pages = max_pages;
  a.page = page;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.HC = (a.G + decode::HEADS - 1) / decode::HEADS;
  a.c = c;
  a.ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + sizeof(PlanHeader));
  a.out = out;
  a.err = &static_cast<PlanHeader*>(ws)->error;
  if (D == 64) return e4m3 ? decode::launch<64, true>(a, k_cache, v_cache, dev, s)
                           : decode::launch<64, false>(a, k_cache, v_cache, dev, s);
  return e4m3 ? decode::launch<128, true>(a, k_cache, v_cache, dev, s)
              : decode::launch<128, false>(a, k_cache, v_cache, dev, s);
}
