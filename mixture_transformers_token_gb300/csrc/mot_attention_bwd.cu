// Gradient of joint attention with respect to its fused QKV rows, on the 5th-generation tensor cores.
//
// Sources: [RFC][BAGEL-7B-MoT][CUDA/ROCm] WS1/WS2 kernel roadmap and integration plan #435 (§1 Motivation item 2, §2 Reference
// hazards: the masks, as in the forward; §3 BAGEL-specific rules: dX passes through the frozen und operators; §3 Numerical
// contract: fixed accumulation order, no atomics).
//
// Per query i and visible key j: P = 2^((S - lse / scale) c) with c = scale log2 e, dP = dout_i . v_j, delta_i = dout_i . out_i,
// dS = P (dP - delta_i); dq_i = scale sum_j dS k_j, dk_j = scale sum_i dS q_i, dv_j = sum_i P dout_i. P is recomputed from S: no
// probability is stored.
//
// dq sums over keys, dk and dv over queries, and neither sum may be cut between CTAs in an order that the schedule sets. So
// there are two kinds of CTAs, each with its sums in tensor memory from the first block to the last, at the price of forming S
// and dP twice: seven products of 128 x 128 x D a block instead of five.
//
//   stats_kernel  -delta and -lse / scale of every row and head, [Hq][T] (reads dout and out once); its first CTA makes the
//                 lists of work.
//   grad_kernel   one CTA an SM, which draws pieces of work until there are none left. First those of dK and dV: (tile of keys, KV
//                 head, share of the blocks). The borders of the sequences' key ranges cut the pack's rows into runs that the same
//                 sequences see, and a tile is 128 rows of a run or what is left of it. So nothing that a sequence holds reaches
//                 the sums of rows that are not its keys, as it would through 0 NaN in a tile of two sequences. Over the sequences
//                 that see these rows, the group's heads and the share's blocks of 128 queries: S' = K Q' and dP' = V dO' (keys in
//                 the rows), P' and dS' as bf16 into tensor memory in the places of S' and dP', dV += P' dO, dK += dS' Q with A
//                 from tensor memory. Each share's sums go to the workspace, and the share that comes last adds them up, in the
//                 order of the shares. Then the pieces of dQ: (128 queries of a sequence, head). Over the blocks of 128 keys, S =
//                 Q K', dP = dO V', dS as bf16 into tensor memory in the place of S, dQ += dS K.
//
// For dK and dV, lse and delta belong to the columns. They are subtracted by the products themselves: one more step of K, whose A
// is ones and whose B holds the value as three bf16 (24 bits), so that no thread reads them from shared memory, which the products
// keep busy.
//
// A block's tiles are copied by TMA (128-byte swizzle) one to three blocks ahead; one warp draws the work and copies, one issues the
// products, and sixteen compute (each thread a quarter of the 128 columns of one row). Rows past a sequence's end inside its last
// block are other sequences' rows: they are zeroed in shared memory where they would be summed over, and masked where they are
// columns.
//
// What bounds it: at D = 128 a block's seven products take 3700 cycles of the tensor cores, which are busy 65% of the time. Tensor
// memory is full (S', dP', dV and dK are 128 columns each), so a block's S' waits for the dV of the block before, which waits for
// its P', and dP' likewise: two chains that alternate, each with the latencies of its barriers. 4096 rows of 28/4 heads of 128 (70%
// of them causal): 343 us, 956 TFLOP/s of the five products that cannot be done without; a pack of twelve sequences of 2900 to 3000
// rows 2.47 ms, one of 37 of up to 700 rows with 8/8 heads of 64 98 us. A wait's instructions and size count, as three kinds of
// warps share the instruction cache: with the limit's code in line at every wait the first took 369 us for 357, the second 2.59 ms
// for 2.50. Measured on the first and not taken:
//   shares in a cluster, added up through its shared memory (20000 of a CTA's 120000 cycles, and a twentieth of the SMs without one);
//   halves of 64 queries with a chain each (products of 64 columns take 48 cycles for 32: 3350 cycles a block for 3120);
//   a warp for each chain's products (394 us for 369); dP of the next block before dQ (2270 cycles for 1975);
//   dQ's S and dP across the border of two pieces (371 for 356 us);
//   every wait but one ahead of P' and dS' in the issuing warp (375 for 369 us).

#include <cuda.h>
#include <cuda_runtime.h>

#include "mot.h"
#include "mot_attention.cuh"
#include "mot_device.cuh"
#include "mot_host.hpp"

namespace mot {
namespace attnb {

using namespace attn;

constexpr int BQ = 128, BK = 128;
constexpr int COMPUTE_WARPS = 16;  // four to a quarter of the rows (tensor memory gives a warp 32 lanes): 32 columns a thread
constexpr int THREADS = 32 * (2 + COMPUTE_WARPS);  // copies, products, P and dS
constexpr uint32_t SUB = 128 * 64 * 2;  // a [128 rows x 64 columns] bf16 swizzled tile

// 128 queries of a sequence: its descriptor and the first of them.
struct alignas(16) Item {
  int q0, k0, nq, nk, nc, i0, pad[2];
};

// Lists in the workspace, made by stats_kernel's first CTA.
struct Work {
  int4* tiles;    // (first row, rows, first and last sequence that may see them), ascending
  int4* parts;    // of dK's and dV's CTAs: (tile, share, shares)
  Item* items;    // of dQ's CTAs
  int32_t* ended; // [tile][Hkv] shares whose sums are there
  int32_t* counts;  // parts, items, the next piece of work to be drawn
  // scratch: changes of the number of sequences that see a row, at each row; borders, a bit a row; the borders in order
  int32_t* change;
  uint32_t* border;
  int32_t* runs;
  int max_tiles, max_items;
};

struct Args {
  const int32_t* seqs;  // [n_seq][5]
  int n_seq, T, Hq, Hkv;
  Work work;
  int most_shares;
  float* sums;          // of each tile's rows [Hkv][most_shares][dV, dK][D / 4][rows][4]: as many in all, however the pack is cut
  float c, scale;
  const float* nlse;    // [Hq][T] -lse / scale
  const float* ndelta;  // [Hq][T] -delta
  uint16_t* dqkv;
  uint32_t* err;
};

// ---------------------------------------------------------------------------
// -delta and -lse / scale
// ---------------------------------------------------------------------------

struct StatsArgs {
  const uint16_t* dout;
  const uint16_t* out;
  const float* lse;
  int T, Hq, Hkv;
  float rscale;
  float* nlse;
  float* ndelta;
  const int32_t* seqs;
  int n_seq;
  int most_shares;
  Work work;
  uint32_t* err;
};

constexpr int STATS_THREADS = 128;

// Query blocks [first, end) of a sequence that see a key of the tile from row `row` on: causal query i sees keys up to nk - nq + i.
__device__ __forceinline__ void query_blocks(const int (&s)[5], int row, int& first, int& end) {
  const int off = s[3] - s[2], j = row - s[1];
  const int i = s[4] < j - off ? s[4] : j - off;
  first = i > 0 ? i / BQ : 0;
  end = (s[2] + BQ - 1) / BQ;
}

// How many CTAs share a tile's blocks, a power of two: as many as give the longest of the sequences that see it about 192 pieces of
// work, if a piece keeps eight blocks. Sums that are cut cost about four blocks a piece to send and to add up. A rule on the tile's
// own sequences and the heads alone, as it sets the order of the sums.
__device__ __forceinline__ int shares_of(int64_t blocks, int keys, int Hkv, int most) {
  const int pieces = (keys + BK - 1) / BK * Hkv;
  int s = 1;
  while (s < most && pieces * s < 192 && blocks >= 16 * s) s *= 2;
  return s;
}

// Sum over the CTA's threads before this one; `total` is the whole sum.
__device__ __forceinline__ int scan_before(int x, int* room, int& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int incl = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  __syncthreads();  // the last use of `room`
  if (lane == 31) room[warp] = incl;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < STATS_THREADS / 32; ++w) {
    if (w < warp) before += room[w];
    total += room[w];
  }
  return before + incl - x;
}

// Shares the tiles out; returns the number of parts. `seq` gives a sequence's descriptor, or false for a bad one.
template <typename Seq>
__device__ int make_parts(const StatsArgs& a, int* room, int tiles, const Seq& seq) {
  const Work& w = a.work;
  __syncthreads();  // the tiles are there
  int parts = 0;
  for (int i0 = 0; i0 < tiles; i0 += STATS_THREADS) {
    const int i = i0 + threadIdx.x, lane = threadIdx.x & 31;
    // query blocks of every `step`-th sequence from `from` on that sees a row, and the most keys of one of them
    auto count = [&](int row, int from, int last, int step, int& blocks, int& keys) {
      int d[5];
      for (int s = from; s <= last; s += step) {
        if (!seq(s, d) || d[1] > row || d[1] + d[3] <= row) continue;
        int first, end;
        query_blocks(d, row, first, end);
        blocks += end > first ? end - first : 0;  // at most T of all sequences
        keys = keys > d[3] ? keys : d[3];
      }
    };
    int4 tile = make_int4(0, 0, 0, -1);
    if (i < tiles) tile = __ldcg(w.tiles + i);
    int blocks = 0, keys = 0;
    const bool wide = tile.w - tile.z >= 32;  // the warp's, a lane a sequence
    if (!wide) count(tile.x, tile.z, tile.w, 1, blocks, keys);
    for (uint32_t left = __ballot_sync(0xffffffffu, wide); left != 0u; left &= left - 1) {
      const int of = __ffs(left) - 1;
      int b = 0, k = 0;
      const int at = __shfl_sync(0xffffffffu, tile.x, of), from = __shfl_sync(0xffffffffu, tile.z, of);
      count(at, from + lane, __shfl_sync(0xffffffffu, tile.w, of), 32, b, k);
      b = int(__reduce_add_sync(0xffffffffu, unsigned(b)));
      k = int(__reduce_max_sync(0xffffffffu, unsigned(k)));
      if (lane == of) blocks = b, keys = k;
    }
    const int shares = i < tiles ? shares_of(blocks * int64_t(a.Hq / a.Hkv), keys, a.Hkv, a.most_shares) : 0;
    int total;
    const int at = parts + scan_before(shares, room, total);
    for (int p = 0; p < shares; ++p) w.parts[at + p] = make_int4(i, p, shares, 0);
    parts += total;
  }
  return parts;
}

// Query ranges that overlap so far that they have more than T rows: there is no work, which would grow with their number.
__device__ __forceinline__ void no_work(const Work& w) {
  if (threadIdx.x == 0) w.counts[0] = w.counts[1] = w.counts[2] = 0;
}

// The lists of work of up to kSortedSeqs sequences, in shared memory. The items come heaviest first: the last run of queries of
// every sequence, then the last but one of every sequence, ...
struct FewRoom {
  int d[kSortedSeqs][5], items[kSortedSeqs], edge[2 * kSortedSeqs], first[2 * kSortedSeqs], sorted[2 * kSortedSeqs];
  int scan[STATS_THREADS / 32];
};
__device__ void make_work_few(const StatsArgs& a, FewRoom& s) {
  const Work& w = a.work;
  const int tid = threadIdx.x;
  bool bad = false;
  int rows = 0;
  if (tid < kSortedSeqs) {
    int d[5] = {0, 0, 0, 0, 0};
    if (tid < a.n_seq) {
#pragma unroll
      for (int i = 0; i < 5; ++i) d[i] = a.seqs[5 * tid + i];
      bad = bad_seq(d, a.T);
      if (bad) d[2] = d[3] = 0;
    }
#pragma unroll
    for (int i = 0; i < 5; ++i) s.d[tid][i] = d[i];
    s.items[tid] = (d[2] + BQ - 1) / BQ;
    rows = d[2];  // at most 2^24 each
  }
  int all_rows;
  scan_before(rows, s.scan, all_rows);
  if (__syncthreads_or(bad ? 1 : 0) != 0 || all_rows > a.T) {
    if (tid == 0) atomicOr(a.err, MOT_DEV_BAD_SEQUENCE);
  }
  if (all_rows > a.T) return no_work(w);
  // the borders of the key ranges, each once, in ascending order
  constexpr int NONE = 0x7FFFFFFF;
  static_assert(2 * kSortedSeqs <= STATS_THREADS, "a thread a border");
  const int edges = 2 * a.n_seq, mine_of = tid >> 1;  // a sequence's first key, and the one behind its last
  const bool edge = tid < edges && s.d[mine_of][3] > 0;
  const int at = !edge ? NONE : s.d[mine_of][1] + (tid & 1 ? s.d[mine_of][3] : 0);
  if (tid < edges) s.edge[tid] = at;
  __syncthreads();
  bool first = edge;
  if (edge) {
#pragma unroll 8
    for (int i = 0; i < edges; ++i) first &= i >= tid || s.edge[i] != at;
  }
  if (tid < edges) s.first[tid] = first ? at : NONE;
  const int n = __syncthreads_count(first ? 1 : 0);
  if (first) {
    int rank = 0;
#pragma unroll 8
    for (int i = 0; i < edges; ++i) rank += s.first[i] < at ? 1 : 0;
    s.sorted[rank] = at;
  }
  __syncthreads();
  // the runs between them that some sequence sees, in tiles
  int lo = a.n_seq, hi = -1, from = 0, to = 0;
  if (tid + 1 < n) {
    from = s.sorted[tid];
    to = s.sorted[tid + 1];
#pragma unroll 4
    for (int i = 0; i < a.n_seq; ++i) {
      const bool sees = s.d[i][1] <= from && s.d[i][1] + s.d[i][3] > from;
      lo = sees && i < lo ? i : lo;
      hi = sees ? i : hi;
    }
  }
  const int mine = hi >= 0 ? (to - from + BK - 1) / BK : 0;
  int tiles;
  const int t0 = scan_before(mine, s.scan, tiles);
  for (int r = 0; r < mine; ++r) {
    const int row = from + r * BK;
    w.tiles[t0 + r] = make_int4(row, to - row < BK ? to - row : BK, lo, hi);
  }
  auto seq = [&](int i, int (&d)[5]) {
#pragma unroll
    for (int k = 0; k < 5; ++k) d[k] = s.d[i][k];
    return d[3] > 0;
  };
  const int parts = make_parts(a, s.scan, tiles, seq);
  const int c = tid & (kSortedSeqs - 1);
  for (int r = tid / kSortedSeqs; r < s.items[c]; r += STATS_THREADS / kSortedSeqs) {
    int before = 0;
#pragma unroll 4
    for (int i = 0; i < a.n_seq; ++i) {
      const int k = s.items[i];
      before += k < r ? k : r;
      before += i < c && k > r ? 1 : 0;
    }
    if (before < w.max_items)
      w.items[before] = {s.d[c][0], s.d[c][1], s.d[c][2], s.d[c][3], s.d[c][4], (s.items[c] - 1 - r) * BQ, {0, 0}};
  }
  int items;  // at most 2^6 2^17
  scan_before(tid < kSortedSeqs ? s.items[tid] : 0, s.scan, items);
  if (tid == 0) {
    w.counts[0] = parts;
    w.counts[1] = items < w.max_items ? items : w.max_items;
    w.counts[2] = 0;
  }
}

// The lists of work of any number of sequences, by one CTA: T / 8 + 4 T bytes to clear and to read, and the descriptors. The items
// come sequence by sequence.
__device__ void make_work(const StatsArgs& a, int* room) {
  const Work& w = a.work;
  const int tid = threadIdx.x, words = (a.T >> 5) + 1;
  for (int i = tid; i <= a.T; i += STATS_THREADS) w.change[i] = 0;
  for (int i = tid; i < words; i += STATS_THREADS) w.border[i] = 0u;
  __syncthreads();
  // every good descriptor's borders and changes; its items; and the rows of all query ranges, at most T if none overlap
  int items = 0;
  int64_t rows = 0;
  bool bad_any = false;
  for (int s0 = 0; s0 < a.n_seq; s0 += STATS_THREADS) {
    const int s = s0 + tid;
    int mine = 0;
    if (s < a.n_seq) {
      const int32_t* d = a.seqs + 5 * int64_t(s);
      if (bad_seq(d, a.T)) {
        bad_any = true;
      } else {
        const int k0 = d[1], k1 = d[1] + d[3];
        atomicAdd(w.change + k0, 1);
        atomicAdd(w.change + k1, -1);
        atomicOr(w.border + (k0 >> 5), 1u << (k0 & 31));
        atomicOr(w.border + (k1 >> 5), 1u << (k1 & 31));
        mine = (d[2] + BQ - 1) / BQ;
        rows += d[2];
      }
    }
    int total;
    const int at = items + scan_before(mine, room, total);
    for (int r = 0; r < mine && at + r < w.max_items; ++r) {  // the last queries of a sequence, which see the most keys, first
      const int32_t* d = a.seqs + 5 * int64_t(s);
      w.items[at + r] = {d[0], d[1], d[2], d[3], d[4], (mine - 1 - r) * BQ, {0, 0}};
    }
    items = items + total < w.max_items ? items + total : w.max_items;  // more only where queries overlap
  }
  {
    int64_t sum = 0;  // rows of all threads, 21 bits at a time: 256 of them fit 32 bits
    for (int part = 0; part < 3; ++part) {
      int total;
      scan_before(int((rows >> (21 * part)) & 0x1FFFFF), room, total);
      sum += int64_t(total) << (21 * part);
    }
    const bool any = __syncthreads_or(bad_any ? 1 : 0) != 0;
    if (tid == 0 && (any || sum > a.T)) atomicOr(a.err, MOT_DEV_BAD_SEQUENCE);
    if (sum > a.T) return no_work(w);
  }
  // the borders in ascending order
  int n = 0;
  for (int w0 = 0; w0 < words; w0 += STATS_THREADS) {
    uint32_t bits = w0 + tid < words ? __ldcg(w.border + w0 + tid) : 0u;
    int total;
    int at = n + scan_before(__popc(bits), room, total);
    for (; bits != 0u; bits &= bits - 1) w.runs[at++] = (w0 + tid) * 32 + __ffs(bits) - 1;
    n += total;
  }
  __syncthreads();
  // the runs that some sequence sees, in tiles
  int seen = 0, tiles = 0;
  for (int i0 = 0; i0 < n; i0 += STATS_THREADS) {
    const int i = i0 + tid;
    const int from = i < n ? w.runs[i] : 0, to = i + 1 < n ? w.runs[i + 1] : from;
    int total;
    const int change = i < n ? __ldcg(w.change + from) : 0;
    const int seers = seen + scan_before(change, room, total) + change;
    seen += total;
    const int mine = i < n && seers > 0 ? (to - from + BK - 1) / BK : 0;
    const int at = tiles + scan_before(mine, room, total);
    if (i < n) w.change[from] = at;  // read above, by this thread alone: now the first tile from this border on
    for (int r = 0; r < mine; ++r) {
      const int row = from + r * BK;
      w.tiles[at + r] = make_int4(row, to - row < BK ? to - row : BK, a.n_seq, -1);
    }
    tiles += total;
  }
  __syncthreads();
  // the first and the last sequence of each tile: a thread a sequence, or the warp for one of many tiles, a lane a tile
  for (int s0 = 0; s0 < a.n_seq; s0 += STATS_THREADS) {
    const int s = s0 + tid, lane = tid & 31;
    int lo = 0, hi = 0;
    if (s < a.n_seq) {
      const int32_t* d = a.seqs + 5 * int64_t(s);
      if (!bad_seq(d, a.T)) lo = __ldcg(w.change + d[1]), hi = __ldcg(w.change + d[1] + d[3]);  // both are borders
    }
    const bool wide = hi - lo >= 32;
    for (int i = lo; i < (wide ? lo : hi); ++i) {
      atomicMin(&w.tiles[i].z, s);
      atomicMax(&w.tiles[i].w, s);
    }
    for (uint32_t left = __ballot_sync(0xffffffffu, wide); left != 0u; left &= left - 1) {
      const int of = __ffs(left) - 1, end = __shfl_sync(0xffffffffu, hi, of);
      for (int i = __shfl_sync(0xffffffffu, lo, of) + lane; i < end; i += 32) {
        atomicMin(&w.tiles[i].z, s - lane + of);
        atomicMax(&w.tiles[i].w, s - lane + of);
      }
    }
  }
  auto seq = [&](int s, int (&d)[5]) {
    for (int k = 0; k < 5; ++k) d[k] = a.seqs[5 * int64_t(s) + k];
    return !bad_seq(d, a.T);
  };
  const int parts = make_parts(a, room, tiles, seq);
  if (tid == 0) {
    w.counts[0] = parts;
    w.counts[1] = items;
    w.counts[2] = 0;
  }
}

// A CTA takes STATS_ROWS rows and 32 heads; D / 8 lanes a row and head, the sums through shared memory into rows of [Hq][T]. (14 us
// for 4096 rows of 28 heads of 128, cold; 32 rows a CTA left it 129 CTAs and took 51 us, 8 rows took 4 us more on shorter rows.)
constexpr int STATS_ROWS = 4;

template <int D>
__global__ void __launch_bounds__(STATS_THREADS) stats_kernel(const StatsArgs a) {
  constexpr int LANES = D / 8, GROUPS = STATS_THREADS / LANES;
  __shared__ union {
    float sums[32][STATS_ROWS + 1];
    FewRoom few;
    int scan[STATS_THREADS / 32];
  } room;
  pdl_trigger();
  if (blockIdx.y == 0)
    for (int64_t i = int64_t(blockIdx.x) * STATS_THREADS + threadIdx.x; i < int64_t(a.work.max_tiles) * a.Hkv;
         i += int64_t(gridDim.x) * STATS_THREADS)
      a.work.ended[i] = 0;
  if (blockIdx.x == 0) {
    if (blockIdx.y != 0) return;
    if (a.n_seq <= kSortedSeqs) make_work_few(a, room.few);
    else make_work(a, room.scan);
    return;
  }
  const int sub = threadIdx.x % LANES, grp = threadIdx.x / LANES;
  const int row0 = int(blockIdx.x - 1) * STATS_ROWS, h0 = int(blockIdx.y) * 32;
  const int nh = a.Hq - h0 < 32 ? a.Hq - h0 : 32;
  constexpr int BATCH = D == 128 ? 8 : 4;  // rows and heads whose loads are under way at once (one after the other: 18 us)
  static_assert(STATS_ROWS * 32 % (BATCH * GROUPS) == 0, "whole batches");
#pragma unroll 1
  for (int i0 = grp; i0 < STATS_ROWS * 32; i0 += BATCH * GROUPS) {
    uint4 xs[BATCH], ys[BATCH];
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int r = (i0 + u * GROUPS) >> 5, h = (i0 + u * GROUPS) & 31;
      xs[u] = ys[u] = make_uint4(0u, 0u, 0u, 0u);
      if (row0 + r < a.T && h < nh) {
        const int64_t off = (int64_t(row0 + r) * a.Hq + h0 + h) * D + 8 * sub;
        xs[u] = __ldg(reinterpret_cast<const uint4*>(a.dout + off));
        ys[u] = __ldg(reinterpret_cast<const uint4*>(a.out + off));
      }
    }
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const uint4 x = xs[u], y = ys[u];
      float s = __fadd_rn(__fmul_rn(bf_lo(x.x), bf_lo(y.x)), __fmul_rn(bf_hi(x.x), bf_hi(y.x)));
      s = __fadd_rn(s, __fadd_rn(__fmul_rn(bf_lo(x.y), bf_lo(y.y)), __fmul_rn(bf_hi(x.y), bf_hi(y.y))));
      s = __fadd_rn(s, __fadd_rn(__fmul_rn(bf_lo(x.z), bf_lo(y.z)), __fmul_rn(bf_hi(x.z), bf_hi(y.z))));
      s = __fadd_rn(s, __fadd_rn(__fmul_rn(bf_lo(x.w), bf_lo(y.w)), __fmul_rn(bf_hi(x.w), bf_hi(y.w))));
#pragma unroll
      for (int off = LANES / 2; off >= 1; off >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, off));
      if (sub == 0) room.sums[(i0 + u * GROUPS) & 31][(i0 + u * GROUPS) >> 5] = s;
    }
  }
  __syncthreads();
  const int h = threadIdx.x / STATS_ROWS, r = threadIdx.x % STATS_ROWS;
  static_assert(32 * STATS_ROWS == STATS_THREADS, "a thread a row and head");
  if (row0 + r < a.T && h < nh) {
    const int64_t at = int64_t(h0 + h) * a.T + row0 + r;
    a.ndelta[at] = -room.sums[h][r];
    a.nlse[at] = -__fmul_rn(a.lse[at], a.rscale);
  }
}

// ---------------------------------------------------------------------------
// pieces of both kernels
// ---------------------------------------------------------------------------

// The sequences that see a tile's rows, in order; used by a whole warp, the descriptors read one a lane.
struct SeqIter {
  const int32_t* seqs;
  int T, row, last, lane, base;
  uint32_t mask = 0;
  int d[5];
  __device__ SeqIter(const Args& a, const int4& tile, int lane_)
      : seqs(a.seqs), T(a.T), row(tile.x), last(tile.w), lane(lane_), base(tile.z - 32) {}
  __device__ bool next(int (&s)[5]) {
    while (mask == 0) {
      base += 32;
      if (base > last) return false;
      bool in = base + lane <= last;
      if (in) {
#pragma unroll
        for (int i = 0; i < 5; ++i) d[i] = seqs[5 * int64_t(base + lane) + i];
        in = !bad_seq(d, T) && d[1] <= row && d[1] + d[3] > row;  // all of a tile's rows or none
      }
      mask = __ballot_sync(0xffffffffu, in);
    }
    const int l = __ffs(mask) - 1;
    mask &= mask - 1;
#pragma unroll
    for (int i = 0; i < 5; ++i) s[i] = __shfl_sync(0xffffffffu, d[i], l);
    return true;
  }
};

// A tile's blocks are shared out in turn, counted over the sequences that see it, the group's heads and the query blocks, so that the
// shares (a power of two) differ by one block. (By query block plus head, short sequences left most of sixteen shares without any.)
// How many of the n blocks from the `at`-th on a share has.
__device__ __forceinline__ int blocks_of_share(int share, int at, int n, int shares) {
  const int skip = (share - at) & (shares - 1);
  return n > skip ? (n - 1 - skip) / shares + 1 : 0;
}

// Zeroes rows [from, 128) of `tiles` swizzled [128 x 64] tiles that follow one another (a row is 128 consecutive bytes).
__device__ __forceinline__ void zero_rows(uint8_t* tile, int tiles, int from, int lane) {
  for (int b = 0; b < tiles; ++b)
    for (int i = from * 8 + lane; i < 128 * 8; i += 32) *reinterpret_cast<uint4*>(tile + b * SUB + i * 16) = make_uint4(0, 0, 0, 0);
}

// mbar_drain that costs no reading of the clock (400 ns) where the phase is over.
__device__ __forceinline__ void drained(uint32_t bar, uint32_t parity) {
  if (!mbar_try_wait(bar, parity)) mbar_drain(bar, parity);
}

template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* m, int x, int y, uint32_t bar) {
#pragma unroll
  for (int b = 0; b < D / 64; ++b) tma_load_2d(dst + b * SUB, m, x + 64 * b, y, bar);
}

// Shared-memory descriptors (smem_desc_sw128, smem_desc_mn_sw128 with halves SUB apart) by their low words: the steps inside a
// tile are added to these, so that one thread forms an operand in one addition. Formed anew for every product, descriptors took
// the issuing thread 77 cycles a product, longer than the 64 that the product takes.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t addr) { return ((addr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_low_mn(uint32_t addr) { return ((addr & 0x3FFFFu) >> 4) | ((SUB >> 4) << 16); }
__device__ __forceinline__ uint64_t desc_of(uint32_t low) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(low), "r"(kDescHigh));
  return d;
}

// D[128 x 128] = A B' of two row-major [128][DK] tiles (desc_low of each).
template <int DK>
__device__ __forceinline__ void product_nt(uint32_t on, uint32_t d, uint32_t a, uint32_t b) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, 128);
#pragma unroll
  for (int kk = 0; kk < DK / 16; ++kk) {
    const uint32_t at = ((kk / 4) * SUB + (kk % 4) * 32) >> 4;
    mma_bf16_on(on, d, desc_of(a + at), desc_of(b + at), idesc, kk > 0);
  }
}

// A [128][16] operand of one step of K without a swizzle: 8 rows of 16 bytes (8 of the 16 values) are 128 consecutive bytes, the
// other 8 values of the rows follow them, then the next 8 rows.
__device__ __forceinline__ uint32_t step_offset(int row) { return uint32_t(row >> 3) * 256 + uint32_t(row & 7) * 16; }
__device__ __forceinline__ uint64_t desc_step(uint32_t addr) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};"
      : "=l"(d)
      : "r"(((addr & 0x3FFFFu) >> 4) | ((128u >> 4) << 16)), "r"((256u >> 4) | (1u << 14)));
  return d;
}
// x as the sum of three bf16 (24 bits), in an operand's first values
__device__ __forceinline__ uint4 in_three(float x) {
  const float hi = bf_round(x), mid = bf_round(__fsub_rn(x, hi)), lo = __fsub_rn(__fsub_rn(x, hi), mid);
  return make_uint4(cvt_bf2(hi, mid), cvt_bf2(lo, 0.0f), 0u, 0u);
}

// D[128 x DN] += A B of a bf16 [128 x 128] A in tensor memory (every 32 of its columns, 16 words, where the 32 fp32 values were
// that they come from) and a row-major [128][DN] tile (its desc_low_mn).
template <int DN>
__device__ __forceinline__ void product_ta(uint32_t on, uint32_t d, uint32_t a_tmem, uint32_t b, bool accumulate) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, DN) | kIdescBMnMajor;
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    mma_bf16_ta_on(on, d, a_tmem + (kk / 2) * 32 + (kk % 2) * 8, desc_of(b + ((kk * 2048) >> 4)), idesc, accumulate || kk > 0);
}

// Writes PIECES 16-byte pieces of each lane's row, rows `stride` values apart from `to` on, of which the first `rows` are written.
// PIECES lanes exchange theirs first, so that they write pieces that lie side by side: 32 rows at once, 16 bytes each, held the
// load and store unit for 3500 cycles a tile, and the products' warp with it.
template <int PIECES>
__device__ __forceinline__ void write_rows(uint16_t* to, int64_t stride, int rows, int lane, uint4 (&p)[PIECES]) {
#pragma unroll
  for (int bit = 1; bit < PIECES; bit <<= 1) {
    const bool upper = (lane & bit) != 0;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      if (i & bit) continue;
      uint4 send = upper ? p[i] : p[i + bit];
      send.x = __shfl_xor_sync(0xffffffffu, send.x, bit);
      send.y = __shfl_xor_sync(0xffffffffu, send.y, bit);
      send.z = __shfl_xor_sync(0xffffffffu, send.z, bit);
      send.w = __shfl_xor_sync(0xffffffffu, send.w, bit);
      if (upper) p[i] = send;
      else p[i + bit] = send;
    }
  }
#pragma unroll
  for (int k = 0; k < PIECES; ++k) {  // piece lane % PIECES of row PIECES (lane / PIECES) + k
    const int row = lane / PIECES * PIECES + k;
    if (row < rows) *reinterpret_cast<uint4*>(to + row * stride + lane % PIECES * 8) = p[k];
  }
}

__device__ __forceinline__ void ld_columns(uint32_t taddr, float (&v)[32]) { tmem_ld32(taddr, v); }
__device__ __forceinline__ void ld_columns(uint32_t taddr, float (&v)[16]) { tmem_ld16(taddr, v); }

// The CTA's next piece of work: a number that the copying warp draws and hands to the others, one ahead of them.
struct Drawn {
  int4 info[2];  // of the two rings' places: what the work is
  int4 more[2];
  int share[2];
  int4 sent[2];  // of every other piece whose sums were sent: tile and KV head, shares, first row, rows
};

// Warps that wait for a piece of work: those that issue products and those that compute.
constexpr int TAKERS = 1 + COMPUTE_WARPS;

// Whether a wait that began at t0 (0: now) may go on: its beginning, or GIVE_UP after the limit or another warp's timeout. Out of
// line: in line at every wait it filled the instruction cache that three kinds of warps share.
constexpr uint64_t GIVE_UP = ~uint64_t(0);
__device__ __noinline__ uint64_t still_waiting(uint64_t t0, volatile uint32_t* abort_flag, uint32_t* err) {
  if (*abort_flag) return GIVE_UP;
  const uint64_t now = global_timer_ns();
  if (t0 == 0) return now;
  if (now - t0 <= kWaitLimitNs) return t0;
  *abort_flag = 1u;
  if (err != nullptr) atomicOr(err, MOT_DEV_TIMEOUT);
  return GIVE_UP;
}

// A wait by a whole warp.
struct Waits {
  volatile uint32_t* abort_flag;
  uint32_t* err;
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t phase) const {
    const uint32_t at = smem_u32(bar);
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t i = 1; !__all_sync(0xffffffffu, mbar_try_wait(at, phase & 1u)); ++i) {
      if (__builtin_expect((i & 255u) == 0, 0)) {
        t0 = still_waiting(t0, abort_flag, err);
        if (__any_sync(0xffffffffu, t0 == GIVE_UP)) return false;
      }
    }
    return true;
  }
};

// Both phases' barriers and what the CTA's warps share lie behind the larger layout.
constexpr uint32_t kSharedBytes = 896;

// ---------------------------------------------------------------------------
// dK and dV
// ---------------------------------------------------------------------------

template <int D>
struct KvLayout {
  static constexpr int STAGES = D == 128 ? 2 : 4;
  static constexpr uint32_t TILE = 128 * D * 2;
  static constexpr uint32_t STEP = 128 * 16 * 2;                  // an operand of one step of K
  static constexpr uint32_t K = 0, V = TILE;
  static constexpr uint32_t QD = 2 * TILE;                        // STAGES of (Q, dO)
  static constexpr uint32_t ONES = QD + STAGES * 2 * TILE;        // [128][16]: ones in columns 0 to 2
  static constexpr uint32_t STATS = ONES + STEP;                  // STAGES of [128][16] -lse / scale and of -delta, in three
  static constexpr uint32_t EDGES = STATS + STAGES * 2 * STEP;    // STAGES of the block's edges, see the copies
  static constexpr uint32_t BYTES = EDGES + STAGES * 16;
  static constexpr uint32_t S = 0, DP = 128, DV = 256, DK = 384;  // tensor memory
};

struct KvBars {
  uint64_t k_full, v_full, k_free, v_free;  // the tile's K and V; every product of the tile that reads them is done
  uint64_t raw;                             // a tile that is zeroed in part before it is full
  uint64_t q_full[4], q_empty[4], do_full[4], do_empty[4];  // a block's tiles and their stats; their products are done
  uint64_t edges[4];                        // a block's edges are there
  uint64_t s_full, dp_full, p_full, ds_full, dv_done, dk_done, drain, meet;
  uint64_t drawn[2], taken[2];
};

// A share's sums of a tile and KV head.
template <int D>
__device__ __forceinline__ float* sums_of(const Args& a, int row0, int rows, int g, int share) {
  return a.sums + ((int64_t(row0) * a.Hkv + int64_t(rows) * g) * a.most_shares + int64_t(rows) * share) * (2 * D);
}
// Four fp32 of a row: 32 rows of a warp are 512 consecutive bytes.
template <int D>
__device__ __forceinline__ float4* sums_at(float* sums, int rows, int m, int piece, int row) {
  return reinterpret_cast<float4*>(sums) + (m * (D / 4) + piece) * rows + row;
}

// The thread's row of dV and dK as bf16, its quarter of the columns: the sums of the shares in order, BATCH of them read at once (of
// one: from tensor memory).
template <int D, int BATCH>
__device__ __forceinline__ void add_shares(float* sums, int shares, uint32_t at, bool any, int part, int row, int row0, int rows,
                                           int g, const Args& a) {
  using L = KvLayout<D>;
  const int64_t N = int64_t(a.Hq + 2 * a.Hkv) * D;
  const int lane = row & 31, base = row - lane;  // the warp's first row
#pragma unroll 1
  for (int m = 0; m < 2; ++m)
#pragma unroll 1
    for (int c0 = part * (D / 4); c0 < (part + 1) * (D / 4); c0 += 16) {
      __syncwarp();
      float v[16] = {};
      if constexpr (BATCH == 1) {
        if (any) tmem_ld16(at + (m ? L::DK : L::DV) + c0, v);
      } else {
        const float4* from = sums_at<D>(sums, rows, m, c0 / 4, row < rows ? row : rows - 1);  // rows past the last read that
#pragma unroll 1
        for (int p0 = 0; p0 < shares; p0 += BATCH) {
          float4 u[BATCH][4];
#pragma unroll
          for (int p = 0; p < BATCH; ++p)
#pragma unroll
            for (int q = 0; q < 4; ++q) u[p][q] = __ldcg(from + (int64_t(p0 + p) * (D / 2) + q) * rows);
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int p = 0; p < BATCH; ++p) {
              const bool start = p == 0 && p0 == 0;
              v[4 * q] = start ? u[p][q].x : __fadd_rn(v[4 * q], u[p][q].x);
              v[4 * q + 1] = start ? u[p][q].y : __fadd_rn(v[4 * q + 1], u[p][q].y);
              v[4 * q + 2] = start ? u[p][q].z : __fadd_rn(v[4 * q + 2], u[p][q].z);
              v[4 * q + 3] = start ? u[p][q].w : __fadd_rn(v[4 * q + 3], u[p][q].w);
            }
        }
      }
      const float f = m ? a.scale : 1.0f;
      uint4 o[2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        o[k] = make_uint4(cvt_bf2(__fmul_rn(v[8 * k], f), __fmul_rn(v[8 * k + 1], f)),
                          cvt_bf2(__fmul_rn(v[8 * k + 2], f), __fmul_rn(v[8 * k + 3], f)),
                          cvt_bf2(__fmul_rn(v[8 * k + 4], f), __fmul_rn(v[8 * k + 5], f)),
                          cvt_bf2(__fmul_rn(v[8 * k + 6], f), __fmul_rn(v[8 * k + 7], f)));
      write_rows<2>(a.dqkv + (row0 + base) * N + (a.Hq + (m ? 0 : a.Hkv) + g) * D + c0, N, rows - base, lane, o);
    }
  __syncwarp();
}

// Pieces of work [0, n_work) by this and the other CTAs, until they are drawn. Returns the first drawn number past them, to the
// copying warp.
template <int D>
__device__ __forceinline__ int dkv_phase(const CUtensorMap& tm_qkv, const CUtensorMap& tm_do, const Args& a, uint8_t* smem,
                                         KvBars& B, Drawn& drawn, volatile int* ended, uint32_t tmem, int n_work,
                                         const Waits& wait) {
  using L = KvLayout<D>;
  constexpr int STAGES = L::STAGES;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = a.Hq / a.Hkv;
  int past = n_work;
  if (warp == 0) {
    // ---------------- work and copies ----------------
    bool ok = true;
    int t = 0, raws = 0, n = 0;  // blocks, blocks zeroed in part, pieces of work so far
    for (;; ++n) {
      int w = 0;
      if (lane == 0) w = atomicAdd(a.work.counts + 2, 1);
      w = __shfl_sync(0xffffffffu, w, 0);
      if (!(ok = wait(&B.taken[n & 1], (n >> 1) + 1))) break;
      if (w >= n_work) {
        past = w;
        if (lane == 0) {
          drawn.info[n & 1] = make_int4(-1, 0, 0, 0);
          mbar_arrive(smem_u32(&B.drawn[n & 1]));
        }
        break;
      }
      const int g = w % a.Hkv;
      const int4 part = __ldcg(a.work.parts + w / a.Hkv);
      const int share = part.y, shares = part.z;
      const int4 tile = __ldcg(a.work.tiles + part.x);
      const int row0 = tile.x;
      SeqIter count(a, tile, lane);
      int s[5], blocks = 0, at = 0;  // at: blocks of the sequences before, mod shares
      while (count.next(s)) {
        int first, end;
        query_blocks(s, row0, first, end);
        const int all = end > first ? (end - first) * G : 0;
        blocks += blocks_of_share(share, at, all, shares);
        at = (at + all) & (shares - 1);
      }
      if (lane == 0) {
        drawn.info[n & 1] = make_int4(blocks, part.x * a.Hkv + g, shares, 0);
        drawn.share[n & 1] = share;
        drawn.more[n & 1] = tile;
        mbar_arrive(smem_u32(&B.drawn[n & 1]));
      }
      // K and V: the tile before has been read
      if (!(ok = wait(&B.k_free, n + 1))) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(smem_u32(&B.k_full), L::TILE);
        load_tile<D>(smem_u32(smem + L::K), &tm_qkv, (a.Hq + g) * D, row0, smem_u32(&B.k_full));
      }
      if (!(ok = wait(&B.v_free, n + 1))) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(smem_u32(&B.v_full), L::TILE);
        load_tile<D>(smem_u32(smem + L::V), &tm_qkv, (a.Hq + a.Hkv + g) * D, row0, smem_u32(&B.v_full));
      }
      SeqIter it(a, tile, lane);
      at = 0;
      while (ok && it.next(s)) {
        int first, end;
        query_blocks(s, row0, first, end);
        for (int hh = 0; hh < G && ok; ++hh) {
          const int h = g * G + hh;
          const int skip = (share - at) & (shares - 1);
          at = (at + (end > first ? end - first : 0)) & (shares - 1);
          for (int b = first + skip; b < end; b += shares, ++t) {
            const int st = t % STAGES, y = s[0] + b * BQ, have = s[2] - b * BQ < BQ ? s[2] - b * BQ : BQ;
            // dO before Q: its place is free when dV is done, Q's when dK is, and S' wants Q first
#pragma unroll
            for (int m = 1; m >= 0 && ok; --m) {
              const float* from = (m ? a.ndelta : a.nlse) + int64_t(h) * a.T + y;
              float v[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) v[i] = lane + 32 * i < have ? __ldcg(from + lane + 32 * i) : 0.0f;
              if (!(ok = wait(m ? &B.do_empty[st] : &B.q_empty[st], t / STAGES + 1))) break;
              uint8_t* tile_at = smem + L::QD + (st * 2 + m) * L::TILE;
              uint64_t* full = m ? &B.do_full[st] : &B.q_full[st];
              uint64_t* bar = have == BQ ? full : &B.raw;
              if (lane == 0) {
                mbar_arrive_expect_tx(smem_u32(bar), L::TILE);
                load_tile<D>(smem_u32(tile_at), m ? &tm_do : &tm_qkv, h * D, y, smem_u32(bar));
              }
#pragma unroll
              for (int i = 0; i < 4; ++i)
                *reinterpret_cast<uint4*>(smem + L::STATS + (st * 2 + m) * L::STEP + step_offset(lane + 32 * i)) = in_three(v[i]);
              fence_proxy_async_smem();
              // column c of the block sees key row r if min(x, y + r) <= c < z
              if (m == 0 && lane == 0)
                *reinterpret_cast<int4*>(smem + L::EDGES + st * 16) =
                    make_int4(s[4] - b * BQ, row0 - s[1] - (s[3] - s[2]) - b * BQ, have, 0);
              __syncwarp();
              if (lane == 0) {
                if (m == 0) mbar_arrive(smem_u32(&B.edges[st]));
                mbar_arrive(smem_u32(full));
              }
              if (have < BQ) {
                if (!(ok = wait(bar, raws))) break;
                ++raws;
                zero_rows(tile_at, D / 64, have, lane);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(full));
              }
            }
            if (!ok) break;
          }
        }
      }
      if (!ok) break;
    }
    // every copy has landed before shared memory has another use (after a timeout: as far as one more limit shows)
    if (lane == 0) {
      if (n > 0) drained(smem_u32(&B.k_full), uint32_t(n - 1) & 1u), drained(smem_u32(&B.v_full), uint32_t(n - 1) & 1u);
      for (int j = t - STAGES > 0 ? t - STAGES : 0; j < t; ++j)
        drained(smem_u32(&B.q_full[j % STAGES]), uint32_t(j / STAGES) & 1u),
            drained(smem_u32(&B.do_full[j % STAGES]), uint32_t(j / STAGES) & 1u);
      if (!ok) {
        drained(smem_u32(&B.k_full), uint32_t(n) & 1u);
        drained(smem_u32(&B.raw), uint32_t(raws) & 1u);
        drained(smem_u32(&B.q_full[t % STAGES]), uint32_t(t / STAGES) & 1u);
        drained(smem_u32(&B.do_full[t % STAGES]), uint32_t(t / STAGES) & 1u);
      }
    }
  } else if (warp == 1) {
    // ---------------- products ----------------
    const uint32_t on = elect_one();
    const uint32_t ks = desc_low(smem_u32(smem + L::K)), vs = desc_low(smem_u32(smem + L::V));
    const uint64_t ones = desc_step(smem_u32(smem + L::ONES));
    auto tiles = [&](int t) { return smem_u32(smem + L::QD + t % STAGES * 2 * L::TILE); };
    auto form_s = [&](int t) {
      if (!wait(&B.q_full[t % STAGES], t / STAGES)) return false;
      if (t > 0 && !wait(&B.dv_done, t - 1)) return false;  // P' of the block before has been read
      tc_fence_after();
      product_nt<D>(on, tmem + L::S, ks, desc_low(tiles(t)));
      mma_bf16_on(on, tmem + L::S, ones, desc_step(smem_u32(smem + L::STATS + t % STAGES * 2 * L::STEP)), idesc_bf16_f32(128, 128), 1);
      mma_commit_on(on, smem_u32(&B.s_full));
      return true;
    };
    auto form_dp = [&](int t) {
      if (!wait(&B.do_full[t % STAGES], t / STAGES)) return false;
      if (t > 0 && !wait(&B.dk_done, t - 1)) return false;  // dS' of the block before has been read
      tc_fence_after();
      product_nt<D>(on, tmem + L::DP, vs, desc_low(tiles(t) + L::TILE));
      mma_bf16_on(on, tmem + L::DP, ones, desc_step(smem_u32(smem + L::STATS + (t % STAGES * 2 + 1) * L::STEP)),
                  idesc_bf16_f32(128, 128), 1);
      mma_commit_on(on, smem_u32(&B.dp_full));
      return true;
    };
    bool ok = true;
    int t = 0;  // blocks so far
    for (int n = 0; ok; ++n) {
      if (!(ok = wait(&B.drawn[n & 1], n >> 1))) break;
      const int blocks = drawn.info[n & 1].x;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&B.taken[n & 1]));
      if (blocks < 0) break;
      if (!(ok = wait(&B.k_full, n))) break;
      const int from = t, to = t + blocks;
      if (blocks > 0 && !(ok = form_s(t))) break;
      if (blocks <= 1) mma_commit_on(on, smem_u32(&B.k_free));
      if (!(ok = wait(&B.v_full, n))) break;
      if (blocks > 0 && !(ok = form_dp(t))) break;
      if (blocks <= 1) mma_commit_on(on, smem_u32(&B.v_free));
      // S' of the next block as soon as P' of this one has been read, so that the warps that compute go from dS' to the next P'
      for (; t < to; ++t) {
        if (!(ok = wait(&B.p_full, t))) break;
        tc_fence_after();
        product_ta<D>(on, tmem + L::DV, tmem + L::S, desc_low_mn(tiles(t) + L::TILE), t > from);
        mma_commit_on(on, smem_u32(&B.dv_done));
        mma_commit_on(on, smem_u32(&B.do_empty[t % STAGES]));
        if (t + 1 < to && !(ok = form_s(t + 1))) break;
        if (t + 2 == to) mma_commit_on(on, smem_u32(&B.k_free));
        if (!(ok = wait(&B.ds_full, t))) break;
        tc_fence_after();
        product_ta<D>(on, tmem + L::DK, tmem + L::DP, desc_low_mn(tiles(t)), t > from);
        mma_commit_on(on, smem_u32(&B.dk_done));
        mma_commit_on(on, smem_u32(&B.q_empty[t % STAGES]));
        if (t + 1 < to && !(ok = form_dp(t + 1))) break;
        if (t + 2 == to) mma_commit_on(on, smem_u32(&B.v_free));
      }
    }
    // every product issued is done before tensor memory has another use
    mma_commit_on(on, smem_u32(&B.drain));
    drained(smem_u32(&B.drain), 0);
  } else {
    // ---------------- P' and dS': key row 32 (warp % 4) + lane, queries [32 part, 32 part + 32) of the block ----------------
    const int part = (warp - 2) >> 2, quarter = warp & 3, row = quarter * 32 + lane, cb = 32 * part;
    const uint32_t at = tmem + (uint32_t(quarter * 32) << 16);
    const unsigned long long c2 = f2_pack(a.c, a.c);
    // A share's sums are sent when its blocks are done, and said to be there after the next piece's first block: by then they have
    // arrived (a fence at once took 3000 cycles). The share that comes last adds them up.
    int sent = -1, met = 0;  // the place of what was sent and not yet said to be there
    auto meet = [&]() {  // of the warps that compute; like every wait it gives up
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&B.meet));
      return wait(&B.meet, met++);
    };
    auto publish = [&]() {
      if (sent < 0) return true;
      __threadfence();
      if (!meet()) return false;  // all warps' sums are there, and *ended of the piece before has been read
      if (warp == 2 && lane == 0) {
        *ended = atomicAdd(a.work.ended + drawn.sent[sent].x, 1);
        __threadfence();
      }
      if (!meet()) return false;
      const int4 s = drawn.sent[sent];
      if (*ended == s.y - 1) {
        __threadfence();
        const int g = s.x % a.Hkv;
        float* sums = sums_of<D>(a, s.z, s.w, g, 0);
        if (s.y >= 4) add_shares<D, 4>(sums, s.y, at, true, part, row, s.z, s.w, g, a);
        else add_shares<D, 2>(sums, s.y, at, true, part, row, s.z, s.w, g, a);
      }
      sent = -1;
      return true;
    };
    bool ok = true;
    int t = 0;  // blocks so far
    for (int n = 0; ok; ++n) {
      if (!(ok = wait(&B.drawn[n & 1], n >> 1))) break;
      const int4 info = drawn.info[n & 1], tile = drawn.more[n & 1];
      const int share = drawn.share[n & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&B.taken[n & 1]));
      if (info.x < 0) break;
      for (const int to = t + info.x; t < to; ++t) {
        const int st = t % STAGES;
        if (!(ok = wait(&B.edges[st], t / STAGES))) break;
        const int4 edge = *reinterpret_cast<const int4*>(smem + L::EDGES + st * 16);
        // columns [lo, hi) of this thread's 32 are visible; rows past the tile see none
        const int hi = row < tile.y ? edge.z - cb : 0, lo = (edge.x < edge.y + row ? edge.x : edge.y + row) - cb;
        const bool masked = __any_sync(0xffffffffu, lo > 0 || hi < 32);
        if (!(ok = wait(&B.s_full, t))) break;
        tc_fence_after();
        float x[32];
        tmem_ld32(at + L::S + cb, x);
        if (masked) {
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] = c >= lo && c < hi ? x[c] : -INFINITY;
        }
        uint32_t pk[16];
#pragma unroll
        for (int c = 0; c < 32; c += 2) {  // S' - lse / scale came from the products
          float u0, u1;
          f2_unpack(f2_mul(f2_pack(x[c], x[c + 1]), c2), u0, u1);
          x[c] = ex2(u0);
          x[c + 1] = ex2(u1);
          pk[c / 2] = cvt_bf2(x[c], x[c + 1]);
        }
        tmem_st16_words(at + L::S + cb, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&B.p_full));
        if (!(ok = wait(&B.dp_full, t))) break;
        tc_fence_after();
        float y[32];
        tmem_ld32(at + L::DP + cb, y);
        if (masked) {
#pragma unroll
          for (int c = 0; c < 32; ++c) y[c] = c >= lo && c < hi ? y[c] : 0.0f;
        }
#pragma unroll
        for (int c = 0; c < 32; c += 2) {  // and dP' - delta
          float u0, u1;
          f2_unpack(f2_mul(f2_pack(y[c], y[c + 1]), f2_pack(x[c], x[c + 1])), u0, u1);
          pk[c / 2] = cvt_bf2(u0, u1);
        }
        tmem_st16_words(at + L::DP + cb, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&B.ds_full));
        if (!(ok = publish())) break;
      }
      if (!ok) break;
      // The last dK is done, and with it all before it. (The next tile's dV and dK are formed after these warps' next P' and dS'.)
      const bool any = info.x > 0;
      if (any && !(ok = wait(&B.dk_done, t - 1))) break;
      tc_fence_after();
      if (info.z == 1) {
        add_shares<D, 1>(nullptr, 1, at, any, part, row, tile.x, tile.y, info.y % a.Hkv, a);
      } else {
        if (!(ok = publish())) break;  // the piece before's, where this one had no block
        float* to = sums_of<D>(a, tile.x, tile.y, info.y % a.Hkv, share);
#pragma unroll 1
        for (int m = 0; m < 2; ++m) {
          float v[D / 4] = {};
          if (any) ld_columns(at + (m ? L::DK : L::DV) + part * (D / 4), v);
          if (row < tile.y) {
            float4* put = sums_at<D>(to, tile.y, m, part * (D / 16), row);
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
              __stcg(put + i * tile.y, make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
          }
        }
        sent = n & 1;
        if (warp == 2 && lane == 0) drawn.sent[sent] = make_int4(info.y, info.z, tile.x, tile.y);
      }
      tc_fence_before();  // dV and dK have been read: the next P' and dS' say so
    }
    if (ok) publish();
  }
  return past;
}

// ---------------------------------------------------------------------------
// dQ
// ---------------------------------------------------------------------------

template <int D>
struct QLayout {
  static constexpr int K_STAGES = D == 128 ? 3 : 4, V_STAGES = D == 128 ? 2 : 3;
  static constexpr uint32_t TILE = 128 * D * 2;
  static constexpr uint32_t Q = 0, DO = TILE, K = 2 * TILE, V = K + K_STAGES * TILE, BYTES = V + V_STAGES * TILE;
  static constexpr uint32_t S = 0, DP = 256, DQ = 384;  // tensor memory: S of block t at 128 (t % 2)
};

struct QBars {
  uint64_t q_full, q_free;  // the item's Q and dO; every product of the item that reads them is done
  uint64_t raw;             // a K block that is zeroed in part before it is full
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[2], dp_full, ds_full, dq_done, drain;
  uint64_t drawn[2], taken[2];
};

// Items [0, n_work), the first of this CTA's drawn already.
template <int D>
__device__ __forceinline__ void dq_phase(const CUtensorMap& tm_qkv, const CUtensorMap& tm_do, const Args& a, uint8_t* smem,
                                         QBars& B, Drawn& drawn, uint32_t tmem, int first, int n_before, int n_work,
                                         const Waits& wait) {
  using L = QLayout<D>;
  constexpr int K_STAGES = L::K_STAGES, V_STAGES = L::V_STAGES;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = a.Hq / a.Hkv;
  // an item's blocks of keys: all that its last query sees
  auto blocks_of = [](const int4& sq, int nc, int i0) {
    const int i1 = i0 + BQ < sq.z ? i0 + BQ : sq.z;
    return ((i1 > nc ? sq.w : sq.w - sq.z + i1) + BK - 1) / BK;
  };

  if (warp == 0) {
    // ---------------- work and copies ----------------
    bool ok = true;
    int kt = 0, vt = 0, raws = 0, n = 0;  // K and V blocks, blocks zeroed in part, items so far
    for (;; ++n) {
      int w = first;
      if (n > 0) {
        if (lane == 0) w = atomicAdd(a.work.counts + 2, 1);
        w = __shfl_sync(0xffffffffu, w, 0);
      }
      w -= n_before;
      if (!(ok = wait(&B.taken[n & 1], (n >> 1) + 1))) break;
      if (w >= n_work) {
        if (lane == 0) {
          drawn.info[n & 1] = make_int4(0, 0, -1, 0);
          drawn.more[n & 1] = make_int4(0, 0, 0, 0);
          mbar_arrive(smem_u32(&B.drawn[n & 1]));
        }
        break;
      }
      const int4* from = reinterpret_cast<const int4*>(a.work.items + w / a.Hq);
      const int4 sq = __ldcg(from), it = __ldcg(from + 1);  // q0, k0, nq, nk; n_causal, first query
      const int h = w % a.Hq, g = h / G, blocks = blocks_of(sq, it.x, it.y);
      if (lane == 0) {
        drawn.info[n & 1] = sq;
        drawn.more[n & 1] = make_int4(it.x, it.y, h, 0);
        mbar_arrive(smem_u32(&B.drawn[n & 1]));
      }
      if (!(ok = wait(&B.q_free, n + 1))) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(smem_u32(&B.q_full), 2 * L::TILE);
        load_tile<D>(smem_u32(smem + L::Q), &tm_qkv, h * D, sq.x + it.y, smem_u32(&B.q_full));
        load_tile<D>(smem_u32(smem + L::DO), &tm_do, h * D, sq.x + it.y, smem_u32(&B.q_full));
      }
      for (int t = 0; t < blocks; ++t) {
        const int ks = kt % K_STAGES, vs = vt % V_STAGES, y = sq.y + t * BK, have = sq.w - t * BK < BK ? sq.w - t * BK : BK;
        if (!(ok = wait(&B.k_empty[ks], kt / K_STAGES + 1))) break;
        uint8_t* k = smem + L::K + ks * L::TILE;
        uint64_t* bar = have == BK ? &B.k_full[ks] : &B.raw;
        if (lane == 0) {
          mbar_arrive_expect_tx(smem_u32(bar), L::TILE);
          load_tile<D>(smem_u32(k), &tm_qkv, (a.Hq + g) * D, y, smem_u32(bar));
        }
        ++kt;
        if (!(ok = wait(&B.v_empty[vs], vt / V_STAGES + 1))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(smem_u32(&B.v_full[vs]), L::TILE);
          load_tile<D>(smem_u32(smem + L::V + vs * L::TILE), &tm_qkv, (a.Hq + a.Hkv + g) * D, y, smem_u32(&B.v_full[vs]));
        }
        ++vt;
        if (have < BK) {  // the last block: its rows past the sequence's keys are summed over in dS K
          if (!(ok = wait(bar, raws))) break;
          ++raws;
          zero_rows(k, D / 64, have, lane);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&B.k_full[ks]));
        }
      }
      if (!ok) break;
    }
    // every copy has landed before the CTA can exit (after a timeout: as far as one more limit shows)
    if (lane == 0) {
      const int items = n + (ok ? 0 : 1);
      if (items > 0) drained(smem_u32(&B.q_full), uint32_t(items - 1) & 1u);
      for (int j = kt - K_STAGES > 0 ? kt - K_STAGES : 0; j < kt; ++j)
        drained(smem_u32(&B.k_full[j % K_STAGES]), uint32_t(j / K_STAGES) & 1u);
      for (int j = vt - V_STAGES > 0 ? vt - V_STAGES : 0; j < vt; ++j)
        drained(smem_u32(&B.v_full[j % V_STAGES]), uint32_t(j / V_STAGES) & 1u);
      if (!ok) drained(smem_u32(&B.raw), uint32_t(raws) & 1u);
    }
  } else if (warp == 1) {
    // ---------------- products: per block dQ += dS K, dP of the next block, S of the one after it ----------------
    const uint32_t on = elect_one();
    const uint32_t q = desc_low(smem_u32(smem + L::Q)), dy = desc_low(smem_u32(smem + L::DO));
    auto form_s = [&](int u) {
      const int ks = u % K_STAGES;
      if (!wait(&B.k_full[ks], u / K_STAGES)) return false;
      tc_fence_after();
      product_nt<D>(on, tmem + L::S + 128 * (u & 1), q, desc_low(smem_u32(smem + L::K + ks * L::TILE)));
      mma_commit_on(on, smem_u32(&B.s_full[u & 1]));
      return true;
    };
    auto form_dp = [&](int u) {
      const int vs = u % V_STAGES;
      if (!wait(&B.v_full[vs], u / V_STAGES)) return false;
      tc_fence_after();
      product_nt<D>(on, tmem + L::DP, dy, desc_low(smem_u32(smem + L::V + vs * L::TILE)));
      mma_commit_on(on, smem_u32(&B.dp_full));
      mma_commit_on(on, smem_u32(&B.v_empty[vs]));
      return true;
    };
    bool ok = true;
    int u = 0;  // blocks so far
    for (int n = 0; ok; ++n) {
      if (!(ok = wait(&B.drawn[n & 1], n >> 1))) break;
      const int4 sq = drawn.info[n & 1], it = drawn.more[n & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&B.taken[n & 1]));
      if (sq.z < 0) break;
      const int from = u, to = u + blocks_of(sq, it.x, it.y);
      if (!(ok = wait(&B.q_full, n) && form_s(u) && form_dp(u) && (u + 1 >= to || form_s(u + 1)))) break;
      if (u + 1 == to) mma_commit_on(on, smem_u32(&B.q_free));
      for (; u < to; ++u) {
        const int ks = u % K_STAGES;
        if (!(ok = wait(&B.ds_full, u))) break;  // S and dP of the block have been read, dS is written
        tc_fence_after();
        product_ta<D>(on, tmem + L::DQ, tmem + L::S + 128 * (u & 1), desc_low_mn(smem_u32(smem + L::K + ks * L::TILE)), u > from);
        mma_commit_on(on, smem_u32(&B.dq_done));
        mma_commit_on(on, smem_u32(&B.k_empty[ks]));
        if (u + 1 < to && !(ok = form_dp(u + 1))) break;
        if (u + 2 == to) mma_commit_on(on, smem_u32(&B.q_free));
        // dS has been read: S of the block after the next comes into its place. (Waited for at every block, before the next dQ
        // is issued: a barrier two phases ahead looks like one that is not there yet.)
        if (!(ok = wait(&B.dq_done, u))) break;
        if (u + 2 < to && !(ok = form_s(u + 2))) break;
      }
    }
    mma_commit_on(on, smem_u32(&B.drain));
    drained(smem_u32(&B.drain), 0);
  } else {
    // ---------------- dS: query row 32 (warp % 4) + lane, keys [32 part, 32 part + 32) of the block ----------------
    const int part = (warp - 2) >> 2, quarter = warp & 3, row = quarter * 32 + lane, cb = 32 * part;
    const uint32_t at = tmem + (uint32_t(quarter * 32) << 16);
    const unsigned long long c2 = f2_pack(a.c, a.c);
    const int64_t N = int64_t(a.Hq + 2 * a.Hkv) * D;
    int4 next_sq, next_it;
    float next_nl = 0.0f, next_nd = 0.0f;
    // item n and its row's values, which are on their way while the item before is written
    auto fetch = [&](int n) {
      if (!wait(&B.drawn[n & 1], n >> 1)) return false;
      next_sq = drawn.info[n & 1];
      next_it = drawn.more[n & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&B.taken[n & 1]));
      if (next_sq.z >= 0 && next_it.y + row < next_sq.z) {  // past the last item there is no more
        const int64_t stat = int64_t(next_it.z) * a.T + next_sq.x + next_it.y + row;
        next_nl = __ldcg(a.nlse + stat);
        next_nd = __ldcg(a.ndelta + stat);
      }
      return true;
    };
    bool ok = fetch(0);
    int u = 0;  // blocks so far
    for (int n = 1; ok && next_sq.z >= 0; ++n) {
      const int4 sq = next_sq, it = next_it;
      const int i = it.y + row, h = it.z;
      const bool valid = i < sq.z;
      const int lim = !valid ? 0 : i < it.x ? sq.w - sq.z + i + 1 : sq.w;  // keys [0, lim) are visible
      const float nl = valid ? next_nl : 0.0f, nd = valid ? next_nd : 0.0f;
      const unsigned long long nl2 = f2_pack(nl, nl), nd2 = f2_pack(nd, nd);
      const int from = u;
      for (const int to = u + blocks_of(sq, it.x, it.y); u < to; ++u) {
        const int hi = lim - (u - from) * BK - cb;  // columns [0, hi) of this thread's 32 are visible
        const bool masked = __any_sync(0xffffffffu, hi < 32);
        if (!(ok = wait(&B.s_full[u & 1], u >> 1))) break;
        tc_fence_after();
        float x[32];
        tmem_ld32(at + L::S + 128 * (u & 1) + cb, x);
        if (masked) {
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] = c < hi ? x[c] : -INFINITY;
        }
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          float u0, u1;
          f2_unpack(f2_mul(f2_add(f2_pack(x[c], x[c + 1]), nl2), c2), u0, u1);
          x[c] = ex2(u0);
          x[c + 1] = ex2(u1);
          asm volatile("" : "+f"(x[c]), "+f"(x[c + 1]));  // now, not after the wait for dP
        }
        if (!(ok = wait(&B.dp_full, u))) break;
        tc_fence_after();
        uint32_t pk[16];
        float y[32];
        tmem_ld32(at + L::DP + cb, y);
        if (masked) {
#pragma unroll
          for (int c = 0; c < 32; ++c) y[c] = c < hi ? y[c] : 0.0f;
        }
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          float u0, u1;
          f2_unpack(f2_mul(f2_add(f2_pack(y[c], y[c + 1]), nd2), f2_pack(x[c], x[c + 1])), u0, u1);
          pk[c / 2] = cvt_bf2(u0, u1);
        }
        tmem_st16_words(at + L::S + 128 * (u & 1) + cb, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&B.ds_full));
      }
      if (!ok) break;
      // the item's last dQ is done: dP of its last block, which these warps have read, came after the dQ before it
      if (!(ok = fetch(n) && wait(&B.dq_done, u - 1))) break;
      tc_fence_after();
      float v[D / 4];
      ld_columns(at + L::DQ + part * (D / 4), v);
      tc_fence_before();  // dQ has been read: the next item's first dS says so
      uint4 o[D / 32];
#pragma unroll
      for (int k = 0; k < D / 32; ++k)
        o[k] = make_uint4(cvt_bf2(__fmul_rn(v[8 * k], a.scale), __fmul_rn(v[8 * k + 1], a.scale)),
                          cvt_bf2(__fmul_rn(v[8 * k + 2], a.scale), __fmul_rn(v[8 * k + 3], a.scale)),
                          cvt_bf2(__fmul_rn(v[8 * k + 4], a.scale), __fmul_rn(v[8 * k + 5], a.scale)),
                          cvt_bf2(__fmul_rn(v[8 * k + 6], a.scale), __fmul_rn(v[8 * k + 7], a.scale)));
      const int r0 = it.y + quarter * 32;  // the warp's first query
      write_rows<D / 32>(a.dqkv + (sq.x + r0) * N + h * D + part * (D / 4), N, sq.z - r0, lane, o);
    }
  }
}

// What a CTA's warps share beside the tiles.
struct Shared {
  KvBars kv;
  QBars q;
  Drawn drawn[2];  // one for each phase
  uint32_t tmem, abort_flag;
  int ended, first;
};
static_assert(sizeof(Shared) <= kSharedBytes, "room behind the tiles");

template <int D>
constexpr uint32_t kTileBytes = (KvLayout<D>::BYTES > QLayout<D>::BYTES ? KvLayout<D>::BYTES : QLayout<D>::BYTES);

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    grad_kernel(const __grid_constant__ CUtensorMap tm_qkv, const __grid_constant__ CUtensorMap tm_do,
                const __grid_constant__ Args a) {
  using L = KvLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Shared& sh = *reinterpret_cast<Shared*>(smem + kTileBytes<D>);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    auto init = [](uint64_t& bar, int count) { mbar_init(smem_u32(&bar), uint32_t(count)); };
    for (uint64_t* b : {&sh.kv.k_full, &sh.kv.v_full, &sh.kv.k_free, &sh.kv.v_free, &sh.kv.raw, &sh.kv.s_full, &sh.kv.dp_full,
                        &sh.kv.dv_done, &sh.kv.dk_done, &sh.kv.drain, &sh.q.q_full, &sh.q.q_free, &sh.q.raw, &sh.q.s_full[0],
                        &sh.q.s_full[1], &sh.q.dp_full, &sh.q.dq_done, &sh.q.drain})
      init(*b, 1);
    for (uint64_t* b : {&sh.kv.p_full, &sh.kv.ds_full, &sh.kv.meet, &sh.q.ds_full}) init(*b, COMPUTE_WARPS);
    for (int i = 0; i < 4; ++i) {
      for (uint64_t* b : {&sh.kv.q_full[i], &sh.kv.do_full[i]}) init(*b, 2);  // the tile, and its stats
      for (uint64_t* b : {&sh.kv.q_empty[i], &sh.kv.do_empty[i], &sh.kv.edges[i], &sh.q.k_full[i], &sh.q.k_empty[i],
                          &sh.q.v_full[i], &sh.q.v_empty[i]})
        init(*b, 1);
    }
    for (int i = 0; i < 2; ++i) {
      init(sh.kv.drawn[i], 1);
      init(sh.q.drawn[i], 1);
      init(sh.kv.taken[i], TAKERS);
      init(sh.q.taken[i], TAKERS);
    }
    sh.abort_flag = 0u;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  for (int i = threadIdx.x; i < int((2 * L::STAGES + 1) * L::STEP / 16); i += THREADS)  // only the stats' first values change
    *reinterpret_cast<uint4*>(smem + L::ONES + i * 16) =
        i < int(L::STEP / 16) && (i & 8) == 0 ? make_uint4(0x3F803F80u, 0x3F80u, 0u, 0u) : make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  if (warp == 1) {
    tmem_alloc(smem_u32(&sh.tmem), 512);
    tmem_relinquish();
  }
  pdl_wait();  // stats_kernel
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const Waits wait{&sh.abort_flag, a.err};
  const int n_kv = __ldcg(a.work.counts) * a.Hkv, n_q = __ldcg(a.work.counts + 1) * a.Hq;
  const int first = dkv_phase<D>(tm_qkv, tm_do, a, smem, sh.kv, sh.drawn[0], &sh.ended, tmem, n_kv, wait);
  tc_fence_before();
  fence_proxy_async_smem();  // what was written to the tiles comes before the second phase's copies
  __syncthreads();           // every product and copy of the first phase is done
  tc_fence_after();
  if (*const_cast<volatile uint32_t*>(&sh.abort_flag) == 0u)
    dq_phase<D>(tm_qkv, tm_do, a, smem, sh.q, sh.drawn[1], tmem, first, n_kv, n_q, wait);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

inline bool shape_ok(int64_t T, int Hq, int Hkv, int D, int n_seq) {
  return T >= 1 && T <= MOT_MAX_TOKENS && (D == 64 || D == 128) && Hq >= 1 && Hkv >= 1 && Hq <= 1024 && Hkv <= 1024 &&
         Hq % Hkv == 0 && n_seq >= 1 && n_seq <= MOT_MAX_TOKENS;
}

// The most CTAs that share a tile. One or two KV heads make few pieces, so that shares pay where a tile has blocks enough: 2000 causal
// rows of 16/1 heads of 128 take 96 us, with four 136. Small groups have few blocks a tile, and cut sums cost about four blocks a
// piece. With the caps of large groups for all (16, 8 and 4 shares for 1, 2 and more KV heads) heads of 128 take, in us, with a
// group of one 2000 rows of 1/1 heads 46.8 for 43.7, 12 sequences of up to 3000 of 8/8 740 for 712 and 64 of 500 of 4/4 150 for
// 151; of two 8000 rows of 2/1 146 for 133; of three 12 of up to 3000 of 12/4 1079 for 1050, but 2000 and 8000 rows of 3/1 54.9 for
// 65.2 and 168 for 182 and 4000 of 6/2 105 for 107.
inline int most_shares(int Hq, int Hkv) {
  const int G = Hq / Hkv;
  return G >= 4 ? (Hkv == 1 ? 16 : Hkv == 2 ? 8 : 4) : G >= 2 ? 2 : 1;
}

constexpr int64_t kMostWork = 1 << 30;  // pieces of work: drawn as 32-bit numbers, some past the last

// The workspace after its header, in bytes.
struct Room {
  int64_t nlse, ndelta, tiles, parts, items, counts, ended, change, border, runs, sums, end, ctas;
  int max_tiles, max_items;
  Room(int64_t T, int Hq, int Hkv, int D, int64_t n_seq) {
    const int64_t most = most_shares(Hq, Hkv);
    auto up = [](int64_t n) { return (n + 15) / 16 * 16; };
    const int64_t borders = 2 * n_seq < T + 1 ? 2 * n_seq : T + 1, blocks = (T + 127) / 128;
    max_tiles = int(blocks + borders < T ? blocks + borders : T);  // a run adds at most one short tile
    max_items = int(blocks + n_seq < T ? blocks + n_seq : T);
    nlse = 0;
    ndelta = nlse + up(T * Hq * 4);
    tiles = ndelta + up(T * Hq * 4);
    parts = tiles + int64_t(max_tiles) * 16;
    items = parts + int64_t(max_tiles) * most * 16;
    counts = items + int64_t(max_items) * 32;
    ended = counts + 16;
    change = ended + up(int64_t(max_tiles) * Hkv * 4);
    border = change + up((T + 1) * 4);
    runs = border + up((T / 32 + 1) * 4);
    sums = runs + up(borders * 4);
    end = sums + (most > 1 ? T * Hkv * most * (2 * D * 4) : 0);
    ctas = int64_t(max_tiles) * Hkv * most + int64_t(max_items) * Hq;
  }
};

// `most`: at least as many as there are pieces of work.
template <int D>
static int launch(const uint16_t* dout, const uint16_t* qkv, const uint16_t* out, const float* lse, const Args& a, int64_t most,
                  int sms, cudaStream_t s) {
  CUtensorMap tm_qkv, tm_do;
  const uint64_t N = uint64_t(a.Hq + 2 * a.Hkv) * D;
  if (!make_tmap_bf16(&tm_qkv, qkv, N, uint64_t(a.T), 64, 128) ||
      !make_tmap_bf16(&tm_do, dout, uint64_t(a.Hq) * D, uint64_t(a.T), 64, 128))
    return MOT_ERR_CUDA;
  constexpr int bytes = 1024 + int(kTileBytes<D>) + int(kSharedBytes);
  static_assert(bytes > 114 * 1024, "one CTA an SM: two would compete for tensor memory");
  static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
  if (cudaFuncSetAttribute(grad_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return MOT_ERR_CUDA;
  StatsArgs st{};
  st.dout = dout;
  st.out = out;
  st.lse = lse;
  st.T = a.T;
  st.Hq = a.Hq;
  st.Hkv = a.Hkv;
  st.rscale = 1.0f / a.scale;
  st.nlse = const_cast<float*>(a.nlse);
  st.ndelta = const_cast<float*>(a.ndelta);
  st.seqs = a.seqs;
  st.n_seq = a.n_seq;
  st.work = a.work;
  st.most_shares = a.most_shares;
  st.err = a.err;
  stats_kernel<D><<<dim3(unsigned((a.T + STATS_ROWS - 1) / STATS_ROWS + 1), unsigned((a.Hq + 31) / 32)), STATS_THREADS, 0, s>>>(st);
  if (cudaGetLastError() != cudaSuccess) return MOT_ERR_CUDA;
  if (launch_dependent(grad_kernel<D>, dim3(unsigned(most < sms ? most : sms)), dim3(THREADS), size_t(bytes), s, tm_qkv, tm_do, a) !=
      cudaSuccess)
    return MOT_ERR_CUDA;
  return MOT_OK;
}

}  // namespace attnb
}  // namespace mot

using namespace mot;

extern "C" size_t mot_joint_attention_backward_workspace_bytes(int64_t T, int Hq, int Hkv, int D, int n_seq) {
  if (!attnb::shape_ok(T, Hq, Hkv, D, n_seq)) return 0;
  const attnb::Room room(T, Hq, Hkv, D, n_seq);
  return room.ctas <= attnb::kMostWork ? sizeof(PlanHeader) + size_t(room.end) : 0;
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
  const attnb::Room room(T, Hq, Hkv, D, n_seq);
  if (room.ctas > attnb::kMostWork) return MOT_ERR_GEOMETRY;
  if (ws_bytes < mot_joint_attention_backward_workspace_bytes(T, Hq, Hkv, D, n_seq)) return MOT_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const void* ptrs[] = {dout, qkv, out, lse, seqs, ws, dqkv};
  int dev = -1;
  const int st = check_device(s, ptrs, 7, &dev);
  if (st != MOT_OK) return st;
  DeviceGuard guard(dev);
  uint8_t* base = static_cast<uint8_t*>(ws) + sizeof(PlanHeader);
  attnb::Args a{};
  a.seqs = seqs;
  a.n_seq = n_seq;
  a.T = int(T);
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.c = c;
  a.scale = scale;
  a.nlse = reinterpret_cast<float*>(base + room.nlse);
  a.ndelta = reinterpret_cast<float*>(base + room.ndelta);
  a.work.tiles = reinterpret_cast<int4*>(base + room.tiles);
  a.work.parts = reinterpret_cast<int4*>(base + room.parts);
  a.work.items = reinterpret_cast<attnb::Item*>(base + room.items);
  a.work.counts = reinterpret_cast<int32_t*>(base + room.counts);
  a.work.ended = reinterpret_cast<int32_t*>(base + room.ended);
  a.most_shares = attnb::most_shares(Hq, Hkv);
  a.sums = reinterpret_cast<float*>(base + room.sums);
  a.work.change = reinterpret_cast<int32_t*>(base + room.change);
  a.work.border = reinterpret_cast<uint32_t*>(base + room.border);
  a.work.runs = reinterpret_cast<int32_t*>(base + room.runs);
  a.work.max_tiles = room.max_tiles;
  a.work.max_items = room.max_items;
  a.dqkv = dqkv;
  a.err = &static_cast<PlanHeader*>(ws)->error;
  if (D == 64) return attnb::launch<64>(dout, qkv, out, lse, a, room.ctas, sm_count(dev), s);
  return attnb::launch<128>(dout, qkv, out, lse, a, room.ctas, sm_count(dev), s);
}
