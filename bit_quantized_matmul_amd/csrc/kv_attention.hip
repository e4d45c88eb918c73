// Attention over the paged 8-bit cache: few rows a sequence, the launches, and the join of parts.
//
//   o[t, h] = sum_j p_j v_j,   p = softmax_j(scale q[t, h] . k_j),   position - window < j <= position
//
// One pass over the pages with the running maximum m and sum l of the softmax: a page with a larger
// maximum scales what was summed before by exp(m - m').  Codes become fp16 in registers, where they are
// exact; a page's two scales are applied to its scores and to its sum of values in fp32, so pages whose scales
// are far apart cost no bits.
#include "kv_attention.h"

#include <algorithm>

namespace bqm {
namespace attn {
namespace {

// ------------------------------------------------------------------ few rows
//
// The cache is read once and bounds the time.  A tile is 16 queries of one key head: the rows of a
// sequence times the heads that share the key head.  A workgroup takes `chunk` pages of a tile, its waves
// every NW-th of them, straight into registers: a wave's loads of the next page's keys are on their way
// while it weighs this page's scores, and its loads of the next values while it multiplies the next keys.
// One token of 131072 positions, 8 key heads of 128: 52 us, 5.1 TB/s; 64 of up to 8192: 106 us, 4.5 TB/s.
template <typename T, int kDp, int NW>
__global__ __launch_bounds__(64 * NW) void kv_stream_kernel(AttnArgs A, bool qvec, const T *__restrict__ q,
                                                            T *__restrict__ out) {
  // Probabilities are two fp16 terms for every type: one, of 11 bits, leaves errors like half a step of an fp16 result, and the kernel
  // waits for memory (one token of 131072: the same; 64 of up to 8192: 116 us with one term, 117 with two).
  constexpr int kTerms = kTermsOf<T>, kPTerms = 2, kWide = kDp / 64, kSteps = kDp / 32, kCols = kDp / 16;
  constexpr bool kOdd = kDp % 64 != 0;    // a last half chunk of 32 columns
  KvSeq s;
  int job;
  const int rep = A.rep;
  if (!kv_find(A.B, A.M, blockIdx.x, [rep](const KvSeq &x) { return (int)(((int64_t)x.n * rep + 15) / 16); }, &s, &job)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4, kh = blockIdx.y;
  const int last_c = min(s.n * rep, job * 16 + 16) - 1;
  const int c = min(job * 16 + col, last_c), i = c / rep, h = kh * rep + (c - i * rep);
  const int64_t row = s.lo + i;
  const int pos = s.first() + i;
  const int first = s.first() + job * 16 / rep, last = s.first() + last_c / rep;
  int p0, p1;
  pages_of(A, s, first, last, &p0, &p1);
  p0 += (int)blockIdx.z * A.chunk;
  p1 = min(p1, p0 + A.chunk);
  const bool live = job * 16 + col <= last_c;

  __shared__ float sm[NW][16], sl[NW][16];
  __shared__ __align__(16) float so[NW][16][kDp + 4];
  const int64_t at = (row * A.heads + h) * A.splits + blockIdx.z;
  if (p0 >= p1) {                                                        // no page: rows without positions, parts past the last
    if (A.splits > 1) {
      if (threadIdx.x < 16 && live) A.ml[at] = float2{-INFINITY, 0.0f};
    } else if (live) {
      for (int d = threadIdx.x >> 4; d < A.dim; d += 4 * NW) out[(row * A.heads + h) * A.dim + d] = from_f32<T>(0.0f);
    }
    return;
  }
  const int lo = A.window ? max(0, pos - A.window + 1) : 0, hi = min(pos + 1, kv_limit(A.B, s));

  // codes of one page: keys, token 16 (r >> 2) + 4 t + (r & 3) as row r of tile t, and values
  i32x4 kw[4][kWide ? kWide : 1], vw[kCols];
  i32x2 ko[4];
  float ks = 0.0f, vs = 0.0f;
  const int64_t row0 = 16 * (col >> 2) + (col & 3);
  auto load_k = [&](int page) {
    const uint8_t *p = A.kc + ((int64_t)page * A.kv_heads + kh) * (kPage * kDp) + row0 * kDp;
    ks = A.ks[(int64_t)page * A.kv_heads + kh];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int w = 0; w < kWide; ++w) kw[t][w] = *reinterpret_cast<const i32x4 *>(p + t * 4 * kDp + w * 64 + g * 16);
      if constexpr (kOdd) ko[t] = *reinterpret_cast<const i32x2 *>(p + t * 4 * kDp + kWide * 64 + g * 8);
    }
  };
  auto load_v = [&](int page) {
    const uint8_t *p = A.vc + ((int64_t)page * A.kv_heads + kh) * (kPage * kDp) + col * kPage + g * 16;
    vs = A.vs[(int64_t)page * A.kv_heads + kh];
#pragma unroll
    for (int d = 0; d < kCols; ++d) vw[d] = *reinterpret_cast<const i32x4 *>(p + d * 16 * kPage);
  };
  auto page_at = [&](int pi) { return pi < p1 ? __builtin_amdgcn_readfirstlane(kv_page(A.B, s, pi)) : -1; };
  int pi = p0 + wave;
  int page = page_at(pi), next = page_at(pi + NW);
  if (page >= 0) {
    load_k(page);
    load_v(page);
  }

  // queries, a power of two apart so that the largest of a row is at most 2^15
  f16x8 qf[kSteps][kTerms];
  float mul;                                                             // of q, without the page's
  int qe;
  {
    float v[kSteps][8];
    const T *qr = q + row * A.qt + h * A.qh;
    uint32_t top = 0;
#pragma unroll
    for (int w = 0; w < kSteps; ++w) {
      const int cc = w < 2 * kWide ? (w / 2) * 64 + g * 16 + (w & 1) * 8 : kWide * 64 + g * 8;
      load_q8(qr, cc, A.dim, qvec, v[w]);
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[w][j]) & 0x7FFFFFFFu);
    }
    top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
    const float a = __uint_as_float(top);
    qe = top && top < 0x7F800000u ? __builtin_amdgcn_frexp_expf(a) - 15 : 0;
    mul = top < 0x7F800000u ? fabsf(A.scale) : __builtin_nanf("");       // a row that is not finite is NaN
    const float sign = A.scale < 0.0f ? -1.0f : 1.0f;
#pragma unroll
    for (int w = 0; w < kSteps; ++w) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[w][j] = sign * ldexpf(v[w][j], -qe);
      to_terms<kTerms>(v[w], qf[w]);
    }
  }

  f32x4_t o[kCols] = {};
  float m = -INFINITY, l = 0.0f;
  for (; pi < p1; pi += NW) {
    const int after = page_at(pi + 2 * NW);
    f32x4_t x[4] = {};
    const float k_scale = ks;
    if (page >= 0) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int w = 0; w < kSteps; ++w) {
          f16x8 a;
          if (w < 2 * kWide) a = widen(kw[t][w / 2][2 * (w & 1)], kw[t][w / 2][2 * (w & 1) + 1]);
          else a = widen(ko[t][0], ko[t][1]);
#pragma unroll
          for (int z = 0; z < kTerms; ++z) x[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, qf[w][z], x[t], 0, 0, 0);
        }
    }
    if (next >= 0) load_k(next);
    if (page >= 0) {
      // scores are x times f >= 0
      const float f = ldexpf(mul * __builtin_amdgcn_frexp_mantf(k_scale), __builtin_amdgcn_frexp_expf(k_scale) + qe);
      const int j0 = pi * kPage + g * 16;
      const bool whole = pi * kPage + kPage <= min(first + 1, kv_limit(A.B, s)) && (!A.window || pi * kPage > last - A.window);
      uint32_t see = 0xFFFFu;
      if (!whole) {                                                      // bit 4 t + r: token j0 + 4 t + r
        const int a = min(max(lo - j0, 0), 16), b = min(max(hi - j0, 0), 16);
        see = ((1u << b) - 1u) & ~((1u << a) - 1u);
      }
      float top = -INFINITY;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) top = fmaxf(top, whole || (see >> (4 * t + r) & 1) ? x[t][r] : -INFINITY);
      top = rows_max(top);
      const float most = top > -INFINITY ? top * f : -INFINITY, m1 = fmaxf(m, most);
      if (__ballot(m1 > m)) {
        const float alpha = m1 > -INFINITY ? __builtin_amdgcn_exp2f(m - m1) : 0.0f;
        l *= alpha;
#pragma unroll
        for (int d = 0; d < kCols; ++d) o[d] *= alpha;
        m = m1;
      }
      // exponents are taken from the page's largest score on: past 2^24 a score's own steps in fp32 are larger than 2^15, the
      // largest probability, has room for in fp16
      const float lead = most > -INFINITY ? (most - m) + kUp : -INFINITY;
      f16x8 p[2][kPTerms];
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        float e[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const float v = __builtin_amdgcn_exp2f(fmaf(x[2 * a + r / 4][r % 4] - top, f, lead));
          e[r] = whole || (see >> (8 * a + r) & 1) ? v : 0.0f;
        }
        to_terms<kPTerms>(e, p[a]);
        l = add_terms<kPTerms>(p[a], l);
      }
      // of a row that sees none of the page's positions 0, and not what may be no number
      const float v_scale = top > -INFINITY ? vs * 0x1p-15f : 0.0f;
      if (!whole) {
        // what some row does not see may be NaN, and 0 times it would be too: such codes are taken out, and
        // the sums of the rows that do see them made NaN
        bool bad = false;
#pragma unroll
        for (int d = 0; d < kCols; ++d)
#pragma unroll
          for (int w = 0; w < 4; ++w) bad |= has_nan(vw[d][w]);
        if (__builtin_expect(__ballot(bad) != 0, 0)) {
          f16x8 sees[2];
#pragma unroll
          for (int r = 0; r < 16; ++r) sees[r / 8][r % 8] = (_Float16)(see >> r & 1 ? 1.0f : 0.0f);
#pragma unroll
          for (int d = 0; d < kCols; ++d) {
            f32x4_t n = {};
#pragma unroll
            for (int a = 0; a < 2; ++a)
              n = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen(nan_ones(vw[d][2 * a]), nan_ones(vw[d][2 * a + 1])), sees[a], n, 0, 0, 0);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              if (n[w] != 0.0f) o[d][w] = __builtin_nanf("");
              vw[d][w] = without_nan(vw[d][w]);
            }
          }
        }
      }
#pragma unroll
      for (int d = 0; d < kCols; ++d) {
        f32x4_t part = {};
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          const f16x8 v = widen(vw[d][2 * a], vw[d][2 * a + 1]);
#pragma unroll
          for (int z = 0; z < kPTerms; ++z) part = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, p[a][z], part, 0, 0, 0);
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) o[d][w] = fmaf(part[w], v_scale, o[d][w]);
      }
    }
    if (next >= 0) load_v(next);
    page = next;
    next = after;
  }
  l = rows_sum(l);

  // the waves' sums join in LDS
  if (g == 0) {
    sm[wave][col] = m;
    sl[wave][col] = l * 0x1p-15f;
  }
#pragma unroll
  for (int d = 0; d < kCols; ++d) *reinterpret_cast<f32x4_t *>(&so[wave][col][d * 16 + g * 4]) = o[d];
  __syncthreads();
  // 4 NW threads a query
  const int qc = threadIdx.x / (4 * NW), part = threadIdx.x % (4 * NW);
  const int c2 = job * 16 + qc;
  if (c2 > last_c) return;
  const int i2 = c2 / rep, h2 = kh * rep + (c2 - i2 * rep);
  const int64_t head = (int64_t)(s.lo + i2) * A.heads + h2;
  float top = -INFINITY, sum = 0.0f, w[NW];
#pragma unroll
  for (int v = 0; v < NW; ++v) top = fmaxf(top, sm[v][qc]);
#pragma unroll
  for (int v = 0; v < NW; ++v) {
    w[v] = top > -INFINITY ? __builtin_amdgcn_exp2f(sm[v][qc] - top) : sl[v][qc];   // no maximum: 0, or NaN
    sum = fmaf(sl[v][qc], w[v], sum);
  }
  if (A.splits > 1 && part == 0) A.ml[head * A.splits + blockIdx.z] = float2{top, sum};
  const float by = sum != 0.0f ? 1.0f / sum : 0.0f;
  for (int d = part; d < kDp; d += 4 * NW) {
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < NW; ++k) v = fmaf(so[k][qc][d], w[k], v);
    if (A.splits > 1) A.part[(head * A.splits + blockIdx.z) * kDp + d] = v;
    else if (d < A.dim) out[head * A.dim + d] = from_sum<T>(v * by);
  }
}

// ------------------------------------------------------------------ parts
//
// kThreads a row and head: they first weigh the parts, then sum them, four columns a thread and kRows
// parts at a time.  A wave takes up to 16 parts, a workgroup more (us, a wave and a workgroup: 32 heads of 64 parts
// 6.2 and 4.8; 64 rows of 32 heads, 4 parts 4.8 and 5.6).  What bounds it is one trip to memory after the other, so
// the parts are asked for before their weights are known (5.9 -> 4.8 and 4.9 -> 4.8; 9 sequences of 12 heads 4.2 -> 3.6).
constexpr int kMaxParts = 2048, kFewParts = 16;

template <typename T, int kDp, int kThreads>
__global__ __launch_bounds__(256) void kv_join_kernel(AttnArgs A, T *__restrict__ out) {
  constexpr int kLanes = kDp / 4, kRows = kThreads / kLanes, kEach = 256 / kThreads, kWavesEach = kThreads / 64;
  constexpr int kParts = kThreads == 64 ? kFewParts : kMaxParts;
  constexpr int kFirst = kThreads == 64 ? (kFewParts + kRows - 1) / kRows : 8;
  __shared__ float w[kEach][kParts], red[2][4];
  __shared__ f32x4_t sums[kEach][kRows][kLanes];
  const int row = blockIdx.x, e = threadIdx.x / kThreads, x = threadIdx.x % kThreads;
  const int h = blockIdx.y * kEach + e, wave = threadIdx.x >> 6, first = e * kWavesEach;
  const int64_t head = (int64_t)row * A.heads + min(h, A.heads - 1);
  const float2 *ml = A.ml + head * A.splits;
  const int d = x % kLanes, r = x / kLanes;
  const f32x4_t *p = reinterpret_cast<const f32x4_t *>(A.part + head * A.splits * kDp) + d;
  // everything goes out at once, before it is known which parts there are: what was not written is not used
  f32x4_t v[kFirst];
#pragma unroll
  for (int i = 0; i < kFirst; ++i) v[i] = p[(int64_t)min(r + i * kRows, A.splits - 1) * kLanes];
  const float2 mine = ml[min(x, A.splits - 1)];
  if (A.B.offsets && (row < A.B.offsets[0] || row >= A.B.offsets[A.B.seqs])) return;     // a row of no sequence
  float top = mine.x, sum = 0.0f;
  for (int z = x + kThreads; z < A.splits; z += kThreads) top = fmaxf(top, ml[z].x);
  top = wave_max(top);
  if constexpr (kWavesEach > 1) {
    if ((threadIdx.x & 63) == 0) red[0][wave] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWavesEach; ++i) top = fmaxf(top, red[0][first + i]);
  }
  for (int z = x; z < A.splits; z += kThreads) {
    const float2 m = z == x ? mine : ml[z];
    // nothing was seen (the part may not be written: marked by -1), or no maximum anywhere: NaN.  A weight that is too small
    // for fp32 stays 0: what is NaN in such a part was attended to as well.
    const float f = m.y == 0.0f ? -1.0f : top > -INFINITY ? __builtin_amdgcn_exp2f(m.x - top) : m.y;
    w[e][z] = f;
    sum = f < 0.0f ? sum : fmaf(m.y, f, sum);
  }
  sum = group_sum<64>(sum);
  if ((threadIdx.x & 63) == 0) red[1][wave] = sum;
  __syncthreads();
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kWavesEach; ++i) sum += red[1][first + i];
  if (r < kRows) {
    f32x4_t acc = {};
    const auto add = [&](int z, f32x4_t part) {
      const float f = w[e][z];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = f < 0.0f ? acc[i] : fmaf(part[i], f, acc[i]);
    };
#pragma unroll
    for (int i = 0; i < kFirst; ++i)
      if (r + i * kRows < A.splits) add(r + i * kRows, v[i]);
#pragma unroll 4
    for (int z = r + kFirst * kRows; z < A.splits; z += kRows) add(z, p[(int64_t)z * kLanes]);
    sums[e][r][d] = acc;
  }
  __syncthreads();
  if (x >= kLanes || h >= A.heads) return;
  const float by = sum != 0.0f ? 1.0f / sum : 0.0f;
  f32x4_t acc = sums[e][0][d];
#pragma unroll
  for (int k = 1; k < kRows; ++k) acc += sums[e][k][d];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (d * 4 + i < A.dim) out[head * A.dim + d * 4 + i] = from_sum<T>(acc[i] * by);
}

// ------------------------------------------------------------------ dispatch

struct Plan {
  bool many;                              // tiles of 128 queries
  KvMap map;
  int chunk, splits;
};

int64_t above(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tiles of 128 queries where a sequence has many in the mean and there is work for them, in pages times key heads
// times 32 queries.  How many depends on how many waves the tile's registers leave (16 bits up to 128 columns two or more a SIMD,
// fp32 one from 96 columns on, all one past 128) and on fp32's two terms, which cost the tiles more: they are bound by arithmetic,
// the others by memory.  us in tiles of 16 / 128 queries, 8 key heads; sequences x rows of positions, 32 heads:
//                16 bits, 128 columns   192            256            fp32, 64       128            192            256
//   1 x 64 of 8192         56 / 41      66 / 76        110 / 114      34 / 35        58 / 74        90 / 95        113 / 207
//   64 x 8 of 2048        100 / 65      136 / 192      209 / 326      58 / 68        102 / 191      164 / 262      209 / 561
//   64 x 16 of 2048       170 / 126     239 / 290      375 / 485      88 / 135       171 / 291      288 / 398      372 / 799
//   128 x 20 of 300       126 / 52      157 / 119      357 / 184      67 / 50        131 / 109      279 / 151      393 / 335
//   16 x 32 of 4096       177 / 99      253 / 209      384 / 365      96 / 97        182 / 211      295 / 291      386 / 658
//   64 x 64 of 512        177 / 74      219 / 163      479 / 267      102 / 76       182 / 158      384 / 226      520 / 546
//   1 x 512 of 8192       241 / 104     289 / 223      561 / 350      141 / 109      252 / 222      454 / 302      584 / 789
//   4 x 2048 of 4096     1274 / 498    1471 / 1111    2881 / 1877     737 / 528     1306 / 1166    2416 / 1601    2943 / 4530
//   8 heads: 16 x 256 of 1024
//                          75 / 55      92 / 110       190 / 165      44 / 52        79 / 104       150 / 145      196 / 314
// fp32 of 256 columns, whose queries and sums are 256 registers, stays in tiles of 16 (there is no other kernel of it).
struct ManyRule {
  int queries;                            // more than these a sequence
  int64_t work;                           // and no less than this
};
bool takes_many(int dtype, int dim, int64_t queries, int64_t runs, int kv_heads, int width) {
  const int dp = kv_padded_dim(dim);
  if (dtype == BQM_F32 && dp > kMostTileF32) return false;
  const ManyRule r = dp > 128 ? ManyRule{64, 12000} : dtype == BQM_F32 ? ManyRule{128, 24000} : ManyRule{16, 6000};
  return queries > r.queries * runs && above(queries, 32 * runs) * runs * kv_heads * width >= r.work;
}

// Pages a workgroup takes.  Tiles of 16: one workgroup a CU where all sequences are as long as the table is wide, but 4
// pages at least (one a wave), all of up to 8, and 32 at most, so that sequences of unlike length share the CUs (us with
// 4 / 8 / 16 / 32 pages: one sequence of 512 10.4 / 9.1 / 9.0 / 9.0, of 8192 11.8 / 13.0 / 16.2 / 23.4, of 131072 96 / 75 / 64
// / 58; 4 of 4096 16.4 / 14.8 / 18.0 / 25.2; 16 of 8192 69 / 59 / 50 / 48; 64 of up to 8192 110 with 32, 121 with 128).  The
// parts of all workgroups are bounded too.  Tiles of 128: two workgroups a CU, 8 pages at least (us with 8 / 16 / 32 / 64
// pages: 128 rows of 8192 50 / 59 / 65 / 110, 512 145 / 119 / 106 / 160).
Plan plan(int dtype, int tokens, int seqs, int heads, int kv_heads, int dim, int width, int window) {
  constexpr int64_t kMostGroups = 4096;
  const int rep = heads / kv_heads;
  const int64_t runs = seqs < tokens ? seqs : tokens, queries = (int64_t)tokens * rep;
  Plan p;
  p.many = takes_many(dtype, dim, queries, runs, kv_heads, width);
  const int of = p.many ? 128 : 16;
  p.map = kv_map(tokens, seqs, (rep + of - 1) / of, rep, of, 1);
  const int64_t groups = p.map.groups * kv_heads, work = groups * width;
  int64_t chunk;
  if (p.many) {
    chunk = groups >= 512 ? width : above(work, 512);
    if (chunk < 8) chunk = 8;
  } else {
    chunk = above(work, 256);
    chunk = width <= 8 ? width : chunk < 4 ? 4 : chunk > 32 ? 32 : chunk;
    if (chunk < above(work, kMostGroups)) chunk = above(work, kMostGroups);
  }
  if (chunk < above(width, kMaxParts)) chunk = above(width, kMaxParts);
  p.splits = (int)above(width, chunk);
  // a window: the pages that a tile's rows can see, in no more parts
  const int64_t most = ((int64_t)window + of) / kPage + 2;
  if (window && most < width) {
    if (chunk > above(most, p.splits)) chunk = above(most, p.splits);
    if (chunk < 4) chunk = 4;
    p.splits = (int)above(most, chunk);
  }
  p.chunk = (int)chunk;
  return p;
}

template <typename T, int kDp>
hipError_t start(const AttnArgs &A, const Plan &p, bool vec, const T *q, T *out, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (p.many) {
    e = launch_tiles(A, vec, q, std::is_same_v<T, float> ? BQM_F32 : std::is_same_v<T, __bf16> ? BQM_BF16 : BQM_F16, out, s);
  } else {
    kv_stream_kernel<T, kDp, 4><<<dim3((unsigned)A.M.groups, A.kv_heads, A.splits), 256, 0, s>>>(A, vec, q, out);
    e = hipGetLastError();
  }
  if (e != hipSuccess || A.splits == 1) return e;
  if (A.splits <= kFewParts) kv_join_kernel<T, kDp, 64><<<dim3(A.B.tokens, (A.heads + 3) / 4), 256, 0, s>>>(A, out);
  else kv_join_kernel<T, kDp, 256><<<dim3(A.B.tokens, A.heads), 256, 0, s>>>(A, out);
  return hipGetLastError();
}

template <typename T>
hipError_t run(const AttnArgs &A, const Plan &p, const void *q, void *out, hipStream_t s) {
  const int64_t unit = 16 / (int)sizeof(T);
  const bool vec = ((uintptr_t)q & 15u) == 0 && A.qt % unit == 0 && A.qh % unit == 0;
  switch (kv_padded_dim(A.dim)) {
    case 32: return start<T, 32>(A, p, vec, (const T *)q, (T *)out, s);
    case 64: return start<T, 64>(A, p, vec, (const T *)q, (T *)out, s);
    case 96: return start<T, 96>(A, p, vec, (const T *)q, (T *)out, s);
    case 128: return start<T, 128>(A, p, vec, (const T *)q, (T *)out, s);
    case 192: return start<T, 192>(A, p, vec, (const T *)q, (T *)out, s);
    default: return start<T, 256>(A, p, vec, (const T *)q, (T *)out, s);
  }
}

}  // namespace
}  // namespace attn

using namespace attn;

int64_t kv_attention_scratch(int tokens, int seqs, int heads, int kv_heads, int dim, int width) {
  int splits = 1;                         // the workspace is asked for without the type
  for (int dtype : {BQM_F32, BQM_BF16}) splits = std::max(splits, plan(dtype, tokens, seqs, heads, kv_heads, dim, width, 0).splits);
  return splits > 1 ? (int64_t)tokens * heads * splits * (kv_padded_dim(dim) * 4 + 8) : 0;
}

hipError_t launch_kv_attention(const KvBatch &B, const void *q, int dtype, int heads, int dim, int64_t qt, int64_t qh,
                               const uint8_t *kc, const uint8_t *vc, const float *ks, const float *vs, int kv_heads,
                               float scale, int window, void *out, void *scratch, hipStream_t s) {
  // position - window stays in 32 bits: positions are above -2^24, and no cache holds 2^31 - 2^25
  constexpr int kMostWindow = 0x7FFFFFFF - (1 << 25);
  window = window < kMostWindow ? window : kMostWindow;
  const Plan p = plan(dtype, B.tokens, B.seqs, heads, kv_heads, dim, B.width, window);
  float *part = (float *)scratch;
  float2 *ml = (float2 *)(part + (p.splits > 1 ? (int64_t)B.tokens * heads * p.splits * kv_padded_dim(dim) : 0));
  const AttnArgs A{B, p.map, heads, kv_heads, heads / kv_heads, dim, window, qt, qh, scale * 1.44269504f, kc, vc, ks, vs, p.chunk, p.splits, part, ml};
  if (dtype == BQM_F32) return run<float>(A, p, q, out, s);
  if (dtype == BQM_BF16) return run<__bf16>(A, p, q, out, s);
  return run<_Float16>(A, p, q, out, s);
}

}  // namespace bqm
