// What joint attention's forward and backward kernels share: the check of a sequence's descriptor (q_start, k_start, nq, nk,
// n_causal), the map from a CTA index to its work item, and the arithmetic of a pair of scores.
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

// The work items of a sequence are its runs of ROWS query rows; item r counts from the
// end (r = 0 is the last run, which sees the most keys). The grid visits items heaviest
// first with the heads fastest: all heads of item 0 of every sequence, then item 1 of every
// sequence, ... (for up to 64 sequences; beyond that, sequence by sequence), so the in-order
// block dispatch balances the uneven causal work. CTA u takes head u % Hq of item u / Hq.
// Returns false past the last item; a bad descriptor contributes none.
constexpr int kSortedSeqs = 64;

template <int ROWS>
__device__ __forceinline__ int seq_items(const int32_t* seqs, int T, int s) {
  const int32_t* d = seqs + 5 * s;
  return bad_seq(d, T) ? 0 : (d[2] + ROWS - 1) / ROWS;
}

// Finds the item of index k; called by a whole warp, every lane returns the same answer.
// The lanes fetch the descriptors in parallel (one sequence per lane and round of 32), so the
// lookup costs a few memory round trips, not one per sequence.
template <int ROWS>
__device__ bool find_item(const int32_t* seqs, int n_seq, int T, int k, int lane, int4& sq, int& nc, int& i0) {
  int found_s = -1, r = -1;
  if (n_seq <= kSortedSeqs) {
    // items of sequences lane and lane + 32; round rr takes every sequence with more than rr
    // items, in sequence order
    const int it0 = lane < n_seq ? seq_items<ROWS>(seqs, T, lane) : 0;
    const int it1 = lane + 32 < n_seq ? seq_items<ROWS>(seqs, T, lane + 32) : 0;
    int most = it0 > it1 ? it0 : it1;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
      const int o = __shfl_xor_sync(0xffffffffu, most, off);
      most = o > most ? o : most;
    }
    int acc = 0;
    for (int rr = 0; rr < most; ++rr) {
      const uint32_t m0 = __ballot_sync(0xffffffffu, it0 > rr), m1 = __ballot_sync(0xffffffffu, it1 > rr);
      const int c0 = __popc(m0), c1 = __popc(m1);
      if (k < acc + c0 + c1) {
        const int t = k - acc;  // the t-th sequence (from 0) taking part in this round
        found_s = t < c0 ? int(__fns(m0, 0, t + 1)) : 32 + int(__fns(m1, 0, t - c0 + 1));
        r = rr;
        break;
      }
      acc += c0 + c1;
    }
    if (found_s < 0) return false;
  } else {
    // sequence by sequence: a warp-wide running count over rounds of 32 sequences
    int acc = 0;
    for (int s0 = 0; s0 < n_seq && found_s < 0; s0 += 32) {
      const int s = s0 + lane;
      const int nt = s < n_seq ? seq_items<ROWS>(seqs, T, s) : 0;
      int incl = nt;  // inclusive prefix sum over the lanes
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, k < acc + incl && k >= acc + incl - nt);
      if (hit != 0u) {
        const int l = __ffs(hit) - 1;
        found_s = s0 + l;
        r = k - acc - (__shfl_sync(0xffffffffu, incl, l) - __shfl_sync(0xffffffffu, nt, l));
      }
      acc += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (found_s < 0) return false;
  }
  const int32_t* d = seqs + 5 * found_s;
  sq = make_int4(d[0], d[1], d[2], d[3]);
  nc = d[4];
  i0 = (seq_items<ROWS>(seqs, T, found_s) - 1 - r) * ROWS;
  return true;
}

// CTA 0 checks every descriptor, that the query ranges do not overlap (their rows sum to
// at most T) and that the grid covers every item; a failure sets MOT_DEV_BAD_SEQUENCE. Called
// by a whole warp, one sequence per lane and round.
template <int ROWS>
__device__ void check_sequences(const int32_t* seqs, int n_seq, int T, int Hq, int64_t grid, uint32_t* err, int lane) {
  int64_t tiles = 0, rows = 0;
  bool bad = false;
  for (int s = lane; s < n_seq; s += 32) {
    const int32_t* d = seqs + 5 * s;
    if (bad_seq(d, T)) {
      bad = true;
      continue;
    }
    tiles += (d[2] + ROWS - 1) / ROWS;
    rows += d[2];
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    tiles += __shfl_xor_sync(0xffffffffu, tiles, off);
    rows += __shfl_xor_sync(0xffffffffu, rows, off);
  }
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0 && (bad || rows > T || tiles * Hq > grid)) atomicOr(err, MOT_DEV_BAD_SEQUENCE);
}

}  // namespace attn
}  // namespace mot
