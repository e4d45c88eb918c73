// Appending keys and values to the paged 8-bit cache.
//
// A page holds 64 tokens of every head: keys as E4M3 codes [64, dp] and values as codes [dp, 64], each
// with one scale a head.  Values lie with their tokens side by side because the attention's second product
// sums over tokens: its loads are 16 tokens of one column.
//
// Scales are powers of two: a floating point code loses nothing by that but the smallest numbers, and when
// a later token is larger than the page's scale reaches, the earlier codes become
// E4M3(code * earlier scale / scale) exactly, but for what falls below the smallest normal code.
// scale = the smallest power of two, 2^-126 at least, with |value| <= 448 scale over the page's tokens.
//
// An element that is infinite or NaN becomes the NaN code and has no part in the scale, so that a
// token that overflowed spoils its own attention and not its neighbours'.
//
// A workgroup takes the tokens of one page and head; so no two write to the same scale.  17900 tokens of 8 heads of 128: 32 to 36
// us, 3.1 TB/s and more, where HBM would take 23.  Bound by neither: the vector unit is busy 39% of the time (1285
// instructions a wave for 64 tokens, 480 of them angles), and a page's phases - loads, angles, the reduction and its barrier,
// codes, stores - follow each other with nothing of the next page under way but what the other waves (four a SIMD) do.
// Single tokens of 64 sequences 6.7 us, of one 5.6, by the chain from lengths to pages to scales.  Sharing the
// angles among heads (a workgroup for 2, 4 or 8 of them) took as long or longer: its registers leave fewer waves.
//
// Rows that do not start on 16 bytes, and rotary % 16 or dim % 8 other than 0, are loaded an element at a time: 17900 tokens of
// 8 x 128 66 us (30 aligned), of 8 x 80 with 40 turned 49, of 4 x 26 10.  fp32 rows 38 us.  256 columns leave one or two waves a
// SIMD: 66 us, the same rate.
#include "kv_common.h"

namespace bqm {
namespace {

constexpr int kAppendThreads = 256;

struct AppendArgs {
  KvBatch B;
  KvMap M;
  Rope R;
  int heads, dim;
  int64_t kt, kh, vt, vh;                 // strides of tokens and heads
  uint8_t *kc, *vc;                       // [count, heads, 64, dp], [count, heads, dp, 64]
  float *ks, *vs;                         // [count, heads]
};

constexpr uint32_t kInf = 0x7F800000u;

// |v| as an integer: ordered as the values are, infinities and NaN above all others
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The smallest power of two >= 2^-126 that amax (finite, >= 0) is at most 448 times of: 448 = 1.75 x 2^8.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u);      // biased exponent
  return __uint_as_float((uint32_t)max(e, 1) << 23);
}

// Four codes of v times inv (at most 448 by the choice of the scale), and, where `odd` says that there may be
// some, NaN for what is not finite.
__device__ __forceinline__ uint32_t quad(float a, float b, float c, float d, float inv, bool odd) {
  uint32_t w = e4m3_quad(a * inv, b * inv, c * inv, d * inv);
  if (__builtin_expect(odd, 0)) {
    const float v[4] = {a, b, c, d};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (magnitude(v[i]) >= kInf) w = (w & ~(0xFFu << (8 * i))) | (0x7Fu << (8 * i));
  }
  return w;
}

// The codes of a word times f (a power of two, at most 1), where `keep` has no bits.
__device__ __forceinline__ uint32_t rescaled(uint32_t w, float f, uint32_t keep) {
  const int i = (int)w;
  const uint32_t n = e4m3_quad(__builtin_amdgcn_cvt_f32_fp8(i, 0) * f, __builtin_amdgcn_cvt_f32_fp8(i, 1) * f,
                               __builtin_amdgcn_cvt_f32_fp8(i, 2) * f, __builtin_amdgcn_cvt_f32_fp8(i, 3) * f);
  return (n & ~keep) | (w & keep);
}

// N elements as they are in memory.
template <typename T, int N>
struct Raw {
  typedef T Vec __attribute__((ext_vector_type(N), aligned(16)));
  Vec v;
};
template <typename T>
struct Raw<T, 1> {
  T v;
};

// A 4 x 4 transposition of bytes between four neighbouring lanes: lane r gets byte r of each.  Even lanes take
// bytes 0 and 2 of their own and of lane ^ 1, odd ones 1 and 3; then lanes 0 and 1 the lower halves of their own
// and of lane ^ 2, lanes 2 and 3 the upper.
__device__ __forceinline__ uint32_t turn_bytes(uint32_t w, int r) {
  const uint32_t near = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, 0xB1, 0xF, 0xF, false);
  w = __builtin_amdgcn_perm(near, w, r & 1 ? 0x03070105u : 0x06020400u);
  const uint32_t far = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, 0x4E, 0xF, 0xF, false);
  return __builtin_amdgcn_perm(far, w, r & 2 ? 0x03020706u : 0x05040100u);
}

// A thread's item is a unit of a token's row, the tokens of a group of four in four neighbouring lanes: their
// values' codes are turned around between these lanes, so that LDS takes four tokens at a time.
template <typename T, int N, int kDp>
__global__ __launch_bounds__(kAppendThreads) void kv_append_kernel(AppendArgs A, const T *__restrict__ k,
                                                                   const T *__restrict__ v) {
  constexpr int kUnits = kDp / (2 * N), kItems = kPage * kUnits;
  constexpr int kEach = (kItems + kAppendThreads - 1) / kAppendThreads;
  constexpr int kRow = kPage + 4;         // LDS bytes of a column's tokens
  __shared__ __align__(16) uint8_t turned_v[kDp * kRow];
  __shared__ uint32_t red[2][kAppendThreads / 64];

  KvSeq q;
  int job;
  const KvBatch &B = A.B;
  const auto pages_of = [&](const KvSeq &x) {
    const int first = max(0, x.first()), end = kv_limit(B, x);
    return end > first ? (end - 1) / kPage - first / kPage + 1 : 0;
  };
  if (!kv_find(B, A.M, blockIdx.x, pages_of, &q, &job)) return;
  const int first = max(0, q.first()), end = kv_limit(B, q);
  const int pi = first / kPage + job, page = kv_page(B, q, pi);
  // the page's new tokens: slots [a, b), rows from `row` on
  const int a = max(first - pi * kPage, 0), b = min(end - pi * kPage, kPage);
  const int row = q.lo + pi * kPage + a - q.first();
  const int h = blockIdx.y, n = b - a, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const auto token_unit = [&](int e, int *t, int *u) {
    const int i = e * kAppendThreads + threadIdx.x, four = i / 4;
    *u = four % kUnits;
    *t = four / kUnits * 4 + i % 4;
  };

  float x[kEach][2][N];
  Raw<T, N> y[kEach][2];
  const auto load = [&](const T *p, int c) {
    Raw<T, N> o{};
    if (c < A.dim) o = *reinterpret_cast<const Raw<T, N> *>(p + c);
    return o;
  };
  const auto values = [](const Raw<T, N> &r, float (&o)[N]) {
    if constexpr (N == 1) {
      o[0] = to_f32(r.v);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) o[j] = to_f32(r.v[j]);
    }
  };
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    int t, u, c1, c2;
    token_unit(e, &t, &u);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      y[e][s] = Raw<T, N>{};
#pragma unroll
      for (int j = 0; j < N; ++j) x[e][s][j] = 0.0f;
    }
    if (t >= n) continue;
    unit_columns<N>(A.R, u, &c1, &c2);
    const T *kr = k + (row + t) * A.kt + h * A.kh, *vr = v + (row + t) * A.vt + h * A.vh;
    values(load(kr, c1), x[e][0]);
    values(load(kr, c2), x[e][1]);
    y[e][0] = load(vr, c1);
    y[e][1] = load(vr, c2);
  }
  if (page < 0) return;                                                  // looked up while they are on their way
  const int64_t ph = (int64_t)page * A.heads + h;
  const float old_k = A.ks[ph], old_v = A.vs[ph];
  uint32_t top[2] = {0, 0};
  const auto largest = [](const float (&p)[N], uint32_t m) {
#pragma unroll
    for (int i = 0; i < N; ++i) m = max(m, magnitude(p[i]));
    return m;
  };
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    int t, u, c1, c2;
    token_unit(e, &t, &u);
    if (unit_columns<N>(A.R, u, &c1, &c2) && t < n) {
      const int p = A.R.positions[row + t];
      float2 cs[N];
#pragma unroll
      for (int j = 0; j < N; ++j) turn(p, turns_of(A.R.freqs[u * N + j]), A.R.mscale, A.R.sign, &cs[j].x, &cs[j].y);
      unit_turn<N>(A.R, cs, x[e][0], x[e][1]);
    }
    top[0] = largest(x[e][1], largest(x[e][0], top[0]));
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float f[N];
      values(y[e][s], f);
      top[1] = largest(f, top[1]);
    }
  }
  const bool odd_k = top[0] >= kInf, odd_v = top[1] >= kInf;
  if (__builtin_expect(odd_k || odd_v, 0)) {                             // once more, of the finite ones
    top[0] = top[1] = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        float f[N];
        values(y[e][s], f);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const uint32_t mk = magnitude(x[e][s][i]), mv = magnitude(f[i]);
          top[0] = mk < kInf ? max(top[0], mk) : top[0];
          top[1] = mv < kInf ? max(top[1], mv) : top[1];
        }
      }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float m = wave_max(__uint_as_float(top[i]));
    if (lane == 0) red[i][wave] = __float_as_uint(m);
  }
  __syncthreads();
  float need[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float m = 0.0f;
#pragma unroll
    for (int w = 0; w < kAppendThreads / 64; ++w) m = fmaxf(m, __uint_as_float(red[i][w]));
    need[i] = scale_for(m);
  }
  const float sk = a ? fmaxf(old_k, need[0]) : need[0], sv = a ? fmaxf(old_v, need[1]) : need[1];
  uint8_t *kp = A.kc + ph * kPage * kDp, *vp = A.vc + ph * kPage * kDp;
  if (threadIdx.x == 0) {
    A.ks[ph] = sk;
    A.vs[ph] = sv;
  }
  // codes that were there before
  if (a && sk != old_k) {
    uint32_t *w = reinterpret_cast<uint32_t *>(kp);
    for (int i = threadIdx.x; i < a * kDp / 4; i += kAppendThreads) w[i] = rescaled(w[i], old_k / sk, 0);
  }
  if (a && sv != old_v) {
    uint32_t *w = reinterpret_cast<uint32_t *>(vp);
    for (int i = threadIdx.x; i < A.dim * (kPage / 4); i += kAppendThreads) {
      const int t = i % (kPage / 4) * 4;
      if (t < a) w[i] = rescaled(w[i], old_v / sv, a - t >= 4 ? 0u : 0xFFFFFFFFu << (8 * (a - t)));
    }
  }
  const float ik = 1.0f / sk, iv = 1.0f / sv;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    int t, u, c1, c2;
    token_unit(e, &t, &u);
    unit_columns<N>(A.R, u, &c1, &c2);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int c = s ? c2 : c1, r = threadIdx.x & 3;
      uint8_t *to = kp + (a + t) * kDp + c;
      float f[N];
      values(y[e][s], f);
      if constexpr (N == 1) {
        if (t >= n) continue;
        *to = (uint8_t)quad(x[e][s][0], 0.0f, 0.0f, 0.0f, ik, odd_k);
        turned_v[c * kRow + t] = (uint8_t)quad(f[0], 0.0f, 0.0f, 0.0f, iv, odd_v);
      } else {
        uint32_t w[2], z[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          w[j] = quad(x[e][s][4 * j], x[e][s][4 * j + 1], x[e][s][4 * j + 2], x[e][s][4 * j + 3], ik, odd_k);
          z[j] = turn_bytes(quad(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3], iv, odd_v), r);
          if (kItems % kAppendThreads == 0 || t < kPage)
            *reinterpret_cast<uint32_t *>(turned_v + (c + 4 * j + r) * kRow + t - r) = z[j];
        }
        if (t < n) *reinterpret_cast<u32x2_t *>(to) = u32x2_t{w[0], w[1]};
      }
    }
  }
  __syncthreads();
  // a column's tokens: the page's, or four a thread where the slots are aligned to that, or one
  if (n == kPage) {
    for (int i = threadIdx.x; i < A.dim * 4; i += kAppendThreads) {
      const uint32_t *from = reinterpret_cast<const uint32_t *>(turned_v + i / 4 * kRow + i % 4 * 16);
      *reinterpret_cast<u32x4_t *>(vp + i * 16) = u32x4_t{from[0], from[1], from[2], from[3]};
    }
  } else if (((a | n) & 3) == 0) {
    const int words = n / 4;
    for (int i = threadIdx.x; i < A.dim * words; i += kAppendThreads) {
      const int c = i / words, t = (i - c * words) * 4;
      *reinterpret_cast<uint32_t *>(vp + c * kPage + a + t) = *reinterpret_cast<const uint32_t *>(turned_v + c * kRow + t);
    }
  } else {
    for (int i = threadIdx.x; i < A.dim * n; i += kAppendThreads) {
      const int c = i / n, t = i - c * n;
      vp[c * kPage + a + t] = turned_v[c * kRow + t];
    }
  }
}

template <typename T, int N, int kDp>
hipError_t start(const AppendArgs &A, const T *k, const T *v, hipStream_t s) {
  const dim3 grid((unsigned)A.M.groups, (unsigned)A.heads);
  kv_append_kernel<T, N, kDp><<<grid, kAppendThreads, 0, s>>>(A, k, v);
  return hipGetLastError();
}

template <typename T, int N>
hipError_t by_dim(const AppendArgs &A, const T *k, const T *v, hipStream_t s) {
  switch (kv_padded_dim(A.dim)) {
    case 32: return start<T, N, 32>(A, k, v, s);
    case 64: return start<T, N, 64>(A, k, v, s);
    case 96: return start<T, N, 96>(A, k, v, s);
    case 128: return start<T, N, 128>(A, k, v, s);
    case 192: return start<T, N, 192>(A, k, v, s);
    default: return start<T, N, 256>(A, k, v, s);
  }
}

template <typename T>
hipError_t run(const AppendArgs &A, const void *k, const void *v, hipStream_t s) {
  const int64_t unit = 16 / (int)sizeof(T);
  const bool vec = A.R.rotary % 16 == 0 && A.dim % 8 == 0 && (((uintptr_t)k | (uintptr_t)v) & 15u) == 0 &&
                   A.kt % unit == 0 && A.kh % unit == 0 && A.vt % unit == 0 && A.vh % unit == 0;
  if (vec) return by_dim<T, 8>(A, (const T *)k, (const T *)v, s);
  return by_dim<T, 1>(A, (const T *)k, (const T *)v, s);
}

}  // namespace

namespace {
// n new tokens touch (n + 62) / 64 + 1 pages at most, which is n / 64 + 2 or less, and no more than n.
KvMap append_map(int tokens, int seqs) { return kv_map(tokens, seqs, 1, 1, kPage, 2); }
}  // namespace

int64_t kv_append_jobs(int tokens, int seqs) { return append_map(tokens, seqs).groups; }

hipError_t launch_kv_append(const KvBatch &B, const void *k, const void *v, int dtype, int heads, int dim, int64_t kt,
                            int64_t kh, int64_t vt, int64_t vh, const int32_t *positions, const double *freqs, int rotary,
                            bool interleaved, float mscale, uint8_t *kc, uint8_t *vc, float *ks, float *vs, hipStream_t s) {
  const AppendArgs A{B, append_map(B.tokens, B.seqs), {positions, freqs, rotary, interleaved, mscale, 1.0f}, heads, dim, kt, kh, vt, vh, kc, vc, ks, vs};
  if (dtype == BQM_F32) return run<float>(A, k, v, s);
  if (dtype == BQM_BF16) return run<__bf16>(A, k, v, s);
  return run<_Float16>(A, k, v, s);
}

}  // namespace bqm
