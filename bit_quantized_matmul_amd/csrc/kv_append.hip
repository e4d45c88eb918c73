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
// A workgroup takes the tokens of one page and head; so no two write to the same scale.
#include "kv_common.h"

namespace bqm {
namespace {

constexpr int kAppendThreads = 256;

struct AppendArgs {
  KvBatch B;
  Rope R;
  int heads, dim;
  int64_t kt, kh, vt, vh;                 // strides of tokens and heads
  uint8_t *kc, *vc;                       // [count, heads, 64, dp], [count, heads, dp, 64]
  float *ks, *vs;                         // [count, heads]
};

__device__ __forceinline__ bool finite(float v) { return (__float_as_uint(v) & 0x7FFFFFFFu) < 0x7F800000u; }

// The smallest power of two >= 2^-126 that amax (finite, >= 0) is at most 448 times of: 448 = 1.75 x 2^8.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u);      // biased exponent
  return __uint_as_float((uint32_t)max(e, 1) << 23);
}

// Four codes of v times inv, NaN for what is not finite.
__device__ __forceinline__ uint32_t quad(float a, float b, float c, float d, float inv) {
  const float v[4] = {a, b, c, d};
  float q[4];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    q[i] = __builtin_amdgcn_fmed3f(v[i] * inv, -448.0f, 448.0f);
    bad |= !finite(v[i]);
  }
  uint32_t w = e4m3_quad(q[0], q[1], q[2], q[3]);
  if (__builtin_expect(bad, 0)) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!finite(v[i])) w = (w & ~(0xFFu << (8 * i))) | (0x7Fu << (8 * i));
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
  if (!kv_find(B, blockIdx.x, 1, pages_of, &q, &job)) return;
  const int first = max(0, q.first()), end = kv_limit(B, q);
  const int pi = first / kPage + job, page = kv_page(B, q, pi);
  if (page < 0) return;
  // the page's new tokens: slots [a, b), rows from `row` on
  const int a = max(first - pi * kPage, 0), b = min(end - pi * kPage, kPage);
  const int row = q.lo + pi * kPage + a - q.first();
  const int h = blockIdx.y, n = b - a;
  const int64_t ph = (int64_t)page * A.heads + h;

  float x[kEach][2][N], y[kEach][2][N];
  uint32_t top[2] = {0, 0};
  const auto largest = [](const float (&p)[N], uint32_t m) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t u = __float_as_uint(p[i]) & 0x7FFFFFFFu;
      m = u < 0x7F800000u && u > m ? u : m;
    }
    return m;
  };
  const auto load = [&](const T *p, int c, float (&o)[N]) {
    if constexpr (N == 1) o[0] = c < A.dim ? to_f32(p[c]) : 0.0f;
    else if (c < A.dim) load_vec<N>(p + c, o);
  };
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = e * kAppendThreads + threadIdx.x, t = i / kUnits, u = i % kUnits;
#pragma unroll
    for (int j = 0; j < N; ++j) x[e][0][j] = x[e][1][j] = y[e][0][j] = y[e][1][j] = 0.0f;
    if (t >= n) continue;
    int c1, c2;
    const bool turned = unit_columns<N>(A.R, u, &c1, &c2);
    const T *kr = k + (row + t) * A.kt + h * A.kh, *vr = v + (row + t) * A.vt + h * A.vh;
    load(kr, c1, x[e][0]);
    load(kr, c2, x[e][1]);
    load(vr, c1, y[e][0]);
    load(vr, c2, y[e][1]);
    if (turned) {
      const int p = A.R.positions[row + t];
      float2 cs[N];
#pragma unroll
      for (int j = 0; j < N; ++j) turn(p, A.R.freqs[u * N + j], A.R.mscale, A.R.sign, &cs[j].x, &cs[j].y);
      unit_turn<N>(A.R, cs, x[e][0], x[e][1]);
    }
    top[0] = largest(x[e][1], largest(x[e][0], top[0]));
    top[1] = largest(y[e][1], largest(y[e][0], top[1]));
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float m = wave_max(__uint_as_float(top[i]));
    if (lane == 0) red[i][wave] = __float_as_uint(m);
  }
  const float old_k = A.ks[ph], old_v = A.vs[ph];
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
    const int i = e * kAppendThreads + threadIdx.x, t = i / kUnits, u = i % kUnits;
    if (t >= n) continue;
    int c[2];
    unit_columns<N>(A.R, u, &c[0], &c[1]);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint8_t *to = kp + (a + t) * kDp + c[s];
      if constexpr (N == 1) {
        *to = (uint8_t)quad(x[e][s][0], 0.0f, 0.0f, 0.0f, ik);
        turned_v[c[s] * kRow + t] = (uint8_t)quad(y[e][s][0], 0.0f, 0.0f, 0.0f, iv);
      } else {
        uint32_t w[2], z[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          w[j] = quad(x[e][s][4 * j], x[e][s][4 * j + 1], x[e][s][4 * j + 2], x[e][s][4 * j + 3], ik);
          z[j] = quad(y[e][s][4 * j], y[e][s][4 * j + 1], y[e][s][4 * j + 2], y[e][s][4 * j + 3], iv);
        }
        *reinterpret_cast<u32x2_t *>(to) = u32x2_t{w[0], w[1]};
#pragma unroll
        for (int j = 0; j < N; ++j) turned_v[(c[s] + j) * kRow + t] = (uint8_t)(z[j / 4] >> (8 * (j % 4)));
      }
    }
  }
  __syncthreads();
  // a column's tokens, four a thread where the page's slots are aligned to that
  if (((a | n) & 3) == 0) {
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
  const dim3 grid((unsigned)kv_append_jobs(A.B.tokens, A.B.seqs), (unsigned)A.heads);
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

// Pages that `tokens` new tokens of `seqs` sequences can touch at most: a run of n touches
// (n + 62) / 64 + 1 of them, and no more than n.
int64_t kv_append_jobs(int tokens, int seqs) {
  const int64_t runs = seqs < tokens ? seqs : tokens, most = tokens / kPage + 2 * runs;
  return most < tokens ? most : tokens;
}

hipError_t launch_kv_append(const KvBatch &B, const void *k, const void *v, int dtype, int heads, int dim, int64_t kt,
                            int64_t kh, int64_t vt, int64_t vh, const int32_t *positions, const double *freqs, int rotary,
                            bool interleaved, float mscale, uint8_t *kc, uint8_t *vc, float *ks, float *vs, hipStream_t s) {
  const AppendArgs A{B, {positions, freqs, rotary, interleaved, mscale, 1.0f}, heads, dim, kt, kh, vt, vh, kc, vc, ks, vs};
  if (dtype == BQM_F32) return run<float>(A, k, v, s);
  if (dtype == BQM_BF16) return run<__bf16>(A, k, v, s);
  return run<_Float16>(A, k, v, s);
}

}  // namespace bqm
