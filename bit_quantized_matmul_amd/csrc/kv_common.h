// The paged 8-bit cache and the rotation of positions, as their kernels share them.
#pragma once

#include "lowp_types.h"

namespace bqm {

constexpr int kPage = 64;                 // tokens of a page, the block of one scale a head
constexpr int kMaxKvDim = 256;

// Columns of a head in the cache: dim padded to a size that kernels are built for.
inline int kv_padded_dim(int dim) { return dim <= 128 ? (dim + 31) / 32 * 32 : (dim + 63) / 64 * 64; }

// Ragged sequences: rows [offsets[s], offsets[s + 1]) are the newest tokens of sequence s, of
// which the cache holds lens[s] with them; without offsets row s is sequence s's one.
struct KvBatch {
  const int32_t *offsets, *lens, *pages;  // pages [seqs, width], rows `stride` apart
  int64_t stride;
  int seqs, tokens, width, count;         // count: pages of the cache
};

struct KvSeq {
  int s, lo, n, len;
  __device__ __forceinline__ int first() const { return len - n; }     // position of row lo; may be negative
};

__device__ __forceinline__ KvSeq kv_seq(const KvBatch &B, int s) {
  KvSeq q{s, s, 1, max(0, B.lens[s])};
  if (B.offsets) {
    q.lo = min(max(0, B.offsets[s]), B.tokens);
    q.n = max(0, min(B.offsets[s + 1], B.tokens) - q.lo);
  }
  return q;
}

// Positions that the sequence's row of the table has pages for.
__device__ __forceinline__ int kv_limit(const KvBatch &B, const KvSeq &q) { return min(q.len, B.width * kPage); }

// The page of positions 64 i .. 64 i + 63, -1 where the table names none of the cache's.
__device__ __forceinline__ int kv_page(const KvBatch &B, const KvSeq &q, int i) {
  const int p = B.pages[q.s * B.stride + i];
  return (unsigned)p < (unsigned)B.count ? p : -1;
}

// Which workgroups a sequence has: those from offset * mul / div + add * (its number) on.  The map is such that
// the next sequence's begin behind all that this one can need, so a workgroup finds its own in a few steps and not by
// adding up what the sequences before it have; the ones that nobody needs end.
struct KvMap {
  int mul, div, add;
  int64_t groups;
};

// Places of sequences that need at most `most` a row, and at most n mul / div rounded up and `add` - 1 more of n rows:
// whichever of the two maps takes fewer.
inline KvMap kv_map(int tokens, int seqs, int most, int mul, int div, int add) {
  const int64_t rows = (int64_t)tokens * most, runs = (int64_t)tokens * mul / div + (int64_t)seqs * add;
  return rows <= runs ? KvMap{most, 1, 0, rows} : KvMap{mul, div, add, runs};
}

// The sequence of workgroup `bid` and its place there, below jobs(seq); false where there is none.  Every wave
// searches for itself, 64 sequences at a time.  (4096 sequences of one row: attention 52 us, append 28; with the sums of all
// sequences before it 131 and 89, and without offsets 44 and 23.)
template <typename F>
__device__ __forceinline__ bool kv_find(const KvBatch &B, const KvMap &M, int bid, F jobs, KvSeq *q, int *job) {
  if (!B.offsets) {                                                      // offset s is s, and most of the first map
    const int s = bid / M.mul;
    if (s >= B.seqs) return false;
    *q = kv_seq(B, s);
    *job = bid - s * M.mul;
    return *job < jobs(*q);
  }
  const int lane = threadIdx.x & 63;
  const auto begin = [&](int s, int offset) { return (int)((int64_t)offset * M.mul / M.div) + M.add * s; };
  int s0 = 0, n = B.seqs;
  while (n > 64) {
    const int step = (n + 63) / 64, s = s0 + lane * step;
    const bool before = s < s0 + n && begin(s, min(max(0, B.offsets[min(s, B.seqs - 1)]), B.tokens)) <= bid;
    const int at = __popcll(__ballot(before)) - 1;
    if (at < 0) return false;
    n = min(step, n - at * step);
    s0 += at * step;
    if (n <= 0) return false;                                            // offsets out of order
  }
  const bool in = lane < n;
  const KvSeq own = in ? kv_seq(B, s0 + lane) : KvSeq{0, 0, 0, 0};
  const int first = begin(s0 + lane, own.lo);
  const int at = __popcll(__ballot(in && first <= bid)) - 1;
  if (at < 0) return false;
  *q = KvSeq{s0 + at, __builtin_amdgcn_readlane(own.lo, at), __builtin_amdgcn_readlane(own.n, at),
             __builtin_amdgcn_readlane(own.len, at)};
  *job = bid - __builtin_amdgcn_readlane(first, at);
  return *job >= 0 && *job < jobs(*q);
}

// ------------------------------------------------------------------ rotation
//
// Turns a position: f / (2 pi), for f radians.
__device__ __forceinline__ double turns_of(double f) { return f * 0.15915494309189535; }

// cos and sin of p times f turns.  The angle is formed and quarter turns are taken off it in 64 bits (in 32, position
// 2^20 would leave a radian 0.06 off): the nearest whole number of them is what 1.5 x 2^52 added to it leaves in its
// lower bits.  What is left, at most an eighth, is rounded once; the series' first terms left out are below 2^-28.
// So cos and sin are nearly what rounding from 64 bits gives: of 18 million turned keys 13 to 22 become another code than
// exact ones would, and 22 to 29 with cos and sin rounded from 64 bits.
__device__ __forceinline__ void turn(int p, double f, float scale, float sign, float *c, float *s) {
  constexpr double kWhole = 0x1.8p52;
  const double t = (double)p * f, z = fma(4.0, t, kWhole);
  const float x = (float)(fma(-0.25, z - kWhole, t) * 6.283185307179586);
  const float x2 = x * x;
  const float sn = fmaf(x * x2, fmaf(x2, fmaf(x2, fmaf(x2, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), x);
  const float cs = fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, -1.0f / 3628800, 1.0f / 40320), -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
  const int q = (int)(__double_as_longlong(z) & 3);                      // quarter turns, modulo 4
  const float a = q & 1 ? sn : cs, b = q & 1 ? cs : sn;
  const float ss = scale * sign;
  *c = (q + 1) & 2 ? -scale * a : scale * a;
  *s = q & 2 ? -ss * b : ss * b;
}

struct Rope {
  const int32_t *positions;
  const double *freqs;                    // [rotary / 2]
  int rotary, interleaved;
  float mscale, sign;
};

// A unit is 2 N columns of a head: N from c1 on and N from c2 on.  The first rotary / (2 N)
// are N pairs each, the rest follow in order.
template <int N>
__device__ __forceinline__ bool unit_columns(const Rope &R, int u, int *c1, int *c2) {
  const int turned = R.rotary / (2 * N);
  if (u < turned && !R.interleaved) {
    *c1 = u * N;
    *c2 = R.rotary / 2 + u * N;
  } else {                                                               // also where c1 >= rotary
    *c1 = u * 2 * N;
    *c2 = *c1 + N;
  }
  return u < turned;
}

// cs: (cos, sin) of the unit's N pairs
template <int N>
__device__ __forceinline__ void unit_turn(const Rope &R, const float2 *cs, float (&a)[N], float (&b)[N]) {
  if (N == 1 || !R.interleaved) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float x = a[i], y = b[i];
      a[i] = fmaf(x, cs[i].x, -(y * cs[i].y));
      b[i] = fmaf(x, cs[i].y, y * cs[i].x);
    }
  } else if constexpr (N > 1) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      float x = a[2 * i], y = a[2 * i + 1];
      a[2 * i] = fmaf(x, cs[i].x, -(y * cs[i].y));
      a[2 * i + 1] = fmaf(x, cs[i].y, y * cs[i].x);
      x = b[2 * i], y = b[2 * i + 1];
      b[2 * i] = fmaf(x, cs[N / 2 + i].x, -(y * cs[N / 2 + i].y));
      b[2 * i + 1] = fmaf(x, cs[N / 2 + i].y, y * cs[N / 2 + i].x);
    }
  }
}

}  // namespace bqm
