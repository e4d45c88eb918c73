// What the attention's kernels share: operands in the matrix cores' registers, the softmax of a page.
//
// A wave multiplies a page of 64 tokens.  Scores are the products K Q^T, keys the instruction's A operand and
// queries its B operand, so a lane holds some tokens' scores of one query; the second product is V^T P^T
// with values as A and the probabilities as B operand, whose lanes hold some tokens of one query again.
// Which token is which row of the first product is free, so it is chosen that a lane's scores are
// the tokens that it holds as B operand, and the probabilities stay in their lanes.
#pragma once

#include <type_traits>

#include "kv_common.h"

namespace bqm {
namespace attn {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

struct AttnArgs {
  KvBatch B;
  KvMap M;                                // tiles to sequences
  int heads, kv_heads, rep, dim, window;  // rep: heads / kv_heads
  int64_t qt, qh;                         // strides of q's tokens and heads
  float scale;                            // times log2(e)
  const uint8_t *kc, *vc;
  const float *ks, *vs;
  int chunk, splits;                      // pages a workgroup takes, and workgroups of a tile
  float *part;                            // [tokens, heads, splits, dp], with splits > 1
  float2 *ml;                             // [tokens, heads, splits]: maximum, sum
};

// Probabilities are 2^15 times themselves in fp16, so that what falls below its normal numbers is below 2^-29.
constexpr float kUp = 15.0f;

// Eight codes as fp16: exact.
__device__ __forceinline__ f16x8 widen(int lo, int hi) {
  f16x8 h;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(i ? hi : lo, 1.0f, false);
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(i ? hi : lo, 1.0f, true);
    h[4 * i] = a[0];
    h[4 * i + 1] = a[1];
    h[4 * i + 2] = b[0];
    h[4 * i + 3] = b[1];
  }
  return h;
}

// v as kTerms fp16 numbers: rounded, or with what the first leaves (22 bits in all).
template <int kTerms>
__device__ __forceinline__ void to_terms(const float (&v)[8], f16x8 (&t)[kTerms]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const f16x2 h = __builtin_convertvector(f32x2{v[i], v[i + 1]}, f16x2);
    t[0][i] = h[0];
    t[0][i + 1] = h[1];
    if constexpr (kTerms == 2) {
      const f16x2 l = __builtin_convertvector(f32x2{v[i] - (float)h[0], v[i + 1] - (float)h[1]}, f16x2);
      t[1][i] = l[0];
      t[1][i + 1] = l[1];
    }
  }
}

// 16-bit q are exact in one term, a power of two apart; fp32 take two.
template <typename T> constexpr int kTermsOf = sizeof(T) == 2 ? 1 : 2;

// 8 columns of a row of q from c on, zeros past dim
template <typename T>
__device__ __forceinline__ void load_q8(const T *p, int c, int dim, bool vec, float (&v)[8]) {
  if (vec && c + 8 <= dim) {
    load_vec<8>(p + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = to_f32(p[min(c + i, dim - 1)]);
      v[i] = c + i < dim ? x : 0.0f;
    }
  }
}

// The larger of the two halves' v, and their sum: swapped between registers.
__device__ __forceinline__ float halves_max(float v) {
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float halves_sum(float v) {
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}
// The same of the four rows of 16 lanes.
__device__ __forceinline__ float rows_max(float v) {
  const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return halves_max(fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1])));
}
__device__ __forceinline__ float rows_sum(float v) {
  const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return halves_sum(__uint_as_float(s[0]) + __uint_as_float(s[1]));
}

// l + the sum of probabilities as they were rounded: what the second product weighs with.
template <int kTerms>
__device__ __forceinline__ float add_terms(const f16x8 (&t)[kTerms], float l) {
#pragma unroll
  for (int z = 0; z < kTerms; ++z)
#pragma unroll
    for (int i = 0; i < 8; i += 2) l = __builtin_amdgcn_fdot2(f16x2{t[z][i], t[z][i + 1]}, f16x2{(_Float16)1.0f, (_Float16)1.0f}, l, false);
  return l;
}

// True where some byte is a NaN code.
__device__ __forceinline__ bool has_nan(int w) { return (((w & 0x7F7F7F7F) + 0x01010101) & (int)0x80808080) != 0; }

// The bytes of w that are NaN codes as 0x38, E4M3's 1, and the others 0.
__device__ __forceinline__ int nan_ones(int w) {
  const uint32_t n = ((((uint32_t)w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7;      // 1 a byte
  return (int)(n * 0x38u);
}
__device__ __forceinline__ int without_nan(int w) {
  const uint32_t n = ((((uint32_t)w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7;
  return w & (int)~(n * 0xFFu);
}

// The pages that a tile's rows, positions first .. last, see: [p0, p1).
__device__ __forceinline__ void pages_of(const AttnArgs &A, const KvSeq &s, int first, int last, int *p0, int *p1) {
  const int end = min(last + 1, kv_limit(A.B, s));
  const int begin = A.window ? max(0, first - A.window + 1) : 0;
  *p0 = begin / kPage;
  *p1 = end > begin ? (end - 1) / kPage + 1 : *p0;
}

// Tiles of 128 queries (kv_attention_tile.hip): fp32 heads up to kMostTileF32 columns, padded.
constexpr int kMostTileF32 = 192;
hipError_t launch_tiles(const AttnArgs &A, bool vec, const void *q, int dtype, void *out, hipStream_t s);

}  // namespace attn
}  // namespace bqm
