// The choice of a token's experts, as routing and the expert layer of few tokens share it.
//
// Logits are compared as they are; equal ones go to the lower expert; NaN counts as -inf, which
// is never chosen, and +inf as the largest fp32 value.
#pragma once

#include "lowp_types.h"

namespace bqm {
namespace {

constexpr int kMaxExperts = 1024, kMaxTop = 32;
constexpr float kHuge = 3.4028234663852886e38f;

// Reductions over 16 consecutive lanes (DPP row rotations) or the wave (then swaps of rows).
template <int CTRL>
__device__ __forceinline__ int row_move(int v) {
  return __builtin_amdgcn_update_dpp(v, v, CTRL, 0xF, 0xF, false);
}

template <int LANES, typename F>
__device__ __forceinline__ int lanes_reduce(int v, F op) {
  v = op(v, row_move<0x121>(v));                               // row_ror 1, 2, 4, 8
  v = op(v, row_move<0x122>(v));
  v = op(v, row_move<0x124>(v));
  v = op(v, row_move<0x128>(v));
  if constexpr (LANES == 64) {
    auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);     // rows 0, 0, 2, 2 and 1, 1, 3, 3
    v = op((int)s[0], (int)s[1]);
    s = __builtin_amdgcn_permlane32_swap(v, v, false, false);          // the lower half twice, the upper twice
    v = op((int)s[0], (int)s[1]);
  }
  return v;
}

template <int LANES>
__device__ __forceinline__ float lanes_max(float v) {
  return __int_as_float(lanes_reduce<LANES>(__float_as_int(v), [](int a, int b) {
    return __float_as_int(fmaxf(__int_as_float(a), __int_as_float(b)));
  }));
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  return __int_as_float(lanes_reduce<LANES>(__float_as_int(v), [](int a, int b) {
    return __float_as_int(__int_as_float(a) + __int_as_float(b));
  }));
}

template <int LANES>
__device__ __forceinline__ int lanes_min(int v) {
  return lanes_reduce<LANES>(v, [](int a, int b) { return min(a, b); });
}

// Sorts N = 4, 8 or 16 keys, largest first: Batcher's odd-even merge sort.
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t (&k)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int h = p; h >= 1; h /= 2)
#pragma unroll
      for (int j = h % p; j + h < N; j += 2 * h)
#pragma unroll
        for (int i = 0; i < h; ++i)
          if (i + j + h < N && (i + j) / (2 * p) == (i + j + h) / (2 * p)) {
            const uint32_t x = k[i + j], y = k[i + j + h];
            k[i + j] = x > y ? x : y;
            k[i + j + h] = x > y ? y : x;
          }
}

// A lane's logits of one token, and the search for the largest of all lanes'.
// 32-bit logits: the largest of the lane's, then of the lanes', then the lowest index
// that has it.
template <typename T, int LANES, int kPer>
struct Logits {
  struct Pick {
    float w = -INFINITY;
    int at = -1;
  };
  float v[kPer];
  int lane;

  __device__ __forceinline__ void load(const T *x, int experts, int l) {
    lane = l;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane + LANES * i;
      const float a = e < experts ? to_f32(x[e]) : -INFINITY;
      v[i] = a != a ? -INFINITY : fminf(a, kHuge);
    }
  }
  __device__ __forceinline__ float value(int i) const { return v[i]; }
  static __device__ __forceinline__ float logit(Pick p) { return p.w; }
  static __device__ __forceinline__ int expert(Pick p) { return p.w > -INFINITY ? p.at : -1; }
  // the largest left, which leaves (-inf if there is none)
  __device__ __forceinline__ Pick next() {
    float b = -INFINITY;
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (v[i] > b) {
        b = v[i];
        at = lane + LANES * i;
      }
    const float w = lanes_max<LANES>(b);
    const int got = lanes_min<LANES>(b == w ? at : 0x7FFFFFFF);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (got == lane + LANES * i) v[i] = -INFINITY;
    return {w, got};
  }
};

// 16-bit logits: a key of the ordered bits over the inverted index, 0 for NaN and -inf, so
// that one integer maximum finds value and lowest index.  The lane sorts its keys once and
// offers its first (16384 tokens of 256: 14.0 us with the search above, 10.8 us so).
template <typename T, int LANES, int kPer>
struct Keys {
  using Pick = uint32_t;
  uint32_t k[kPer];

  __device__ __forceinline__ void load(const T *x, int experts, int lane) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane + LANES * i;
      uint32_t h = 0;
      if (e < experts) {
        const float f = to_f32(x[e]);
        uint32_t b = __builtin_bit_cast(uint16_t, x[e]);
        b = b == 0x8000u ? 0u : b;                             // -0 is 0
        h = f > -INFINITY ? ((b & 0x8000u) ? ~b & 0xFFFFu : b | 0x8000u) << 16 | (0xFFFFu - (uint32_t)e) : 0u;
      }
      k[i] = h;
    }
    sort_keys(k);
  }
  static __device__ __forceinline__ int expert(Pick key) { return key ? (int)(0xFFFFu - (key & 0xFFFFu)) : -1; }
  static __device__ __forceinline__ float logit(Pick key) {
    if (key == 0) return -INFINITY;
    const uint32_t u = key >> 16;
    const uint16_t b = (uint16_t)((u & 0x8000u) ? u & 0x7FFFu : ~u);
    return fminf(to_f32(__builtin_bit_cast(T, b)), kHuge);
  }
  __device__ __forceinline__ float value(int i) const { return logit(k[i]); }
  __device__ __forceinline__ Pick next() {
    const uint32_t w = (uint32_t)lanes_reduce<LANES>((int)k[0], [](int a, int b) {
      return (uint32_t)a > (uint32_t)b ? a : b;
    });
    const bool mine = k[0] == w;
#pragma unroll
    for (int i = 0; i + 1 < kPer; ++i) k[i] = mine ? k[i + 1] : k[i];
    k[kPer - 1] = mine ? 0u : k[kPer - 1];
    return w;
  }
};

template <int LANES, int kPer> struct Keys<float, LANES, kPer> : Logits<float, LANES, kPer> {};

// LANES lanes choose one token's experts; lane l of them holds experts l, l + LANES, ... of row x.
// done(j, id, weight) for every choice j, by some lane.
template <typename T, int LANES, int kPer, typename F>
__device__ __forceinline__ void choose_experts(const T *row, int experts, int top, int renorm, F done) {
  const int lane = threadIdx.x & (LANES - 1);
  Keys<T, LANES, kPer> x;
  x.load(row, experts, lane);
  float ref = 0.0f, total = 0.0f;                              // the largest logit; the sum of exp(l - ref)
  if (!renorm) {
    float best = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPer; ++i) best = fmaxf(best, x.value(i));
    best = lanes_max<LANES>(best);
    ref = best > -INFINITY ? best : 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) total += expf(x.value(i) - ref);
    total = lanes_sum<LANES>(total);
  }
  using K = Keys<T, LANES, kPer>;
  typename K::Pick first{}, mine[2] = {};                      // the largest; the choices lane and lane + LANES
  for (int j = 0; j < top; ++j) {
    const typename K::Pick p = x.next();
    if (j == 0) first = p;
    if (j == lane) mine[0] = p;
    if (j == lane + LANES) mine[1] = p;
  }
  const float most = K::logit(first);
  ref = most > -INFINITY ? most : 0.0f;
  float e[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) e[h] = K::expert(mine[h]) >= 0 ? expf(K::logit(mine[h]) - ref) : 0.0f;
  if (renorm) total = lanes_sum<LANES>(e[0] + e[1]);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = lane + h * LANES, id = K::expert(mine[h]);
    if (j < top) done(j, id, id >= 0 ? e[h] / total : 0.0f);
  }
}

}  // namespace
}  // namespace bqm
