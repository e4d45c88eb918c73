// Element types of the 8-bit float and mixture-of-experts operators: the
// 16- and 32-bit types of their inputs and results, and E4M3 codes.
#pragma once

#include "bqm_common.h"

namespace bqm {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

inline int elem_size(int dtype) { return dtype == BQM_F32 ? 4 : 2; }
inline bool known_dtype(int dtype) { return dtype == BQM_F32 || dtype == BQM_BF16 || dtype == BQM_F16; }

// fp32 value of an element, and the element nearest to an fp32 value (half to even)
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__bf16 v) { return (float)v; }
__device__ __forceinline__ float to_f32(_Float16 v) { return (float)v; }
template <typename T> __device__ __forceinline__ T from_f32(float v) { return (T)v; }

// N consecutive elements as fp32, with 16-byte loads: p is aligned to 16 bytes.
template <int N>
__device__ __forceinline__ void load_vec(const float *p, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const f32x4_t a = *reinterpret_cast<const f32x4_t *>(p + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[i + j] = a[j];
  }
}
template <int N, typename T>
__device__ __forceinline__ void load_vec(const T *p, float (&v)[N]) {
  typedef T tx8 __attribute__((ext_vector_type(8)));
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    const tx8 a = *reinterpret_cast<const tx8 *>(p + i);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i + j] = to_f32(a[j]);
  }
}

// The E4M3 codes of four values (half to even), |value| <= 448.
__device__ __forceinline__ uint32_t e4m3_quad(float a, float b, float c, float d) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true);
}

// The sum of `v` over the lanes up to this one, by moves between lanes' registers: within
// rows of 16, then a row's last lane to the row after it, then lane 31 to the upper half.  (A grouped
// product of 52792 rows, 192 columns, 3472 results: 225 us, with shuffles through LDS 242.)
__device__ __forceinline__ int wave_prefix(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);      // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);      // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);      // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);      // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);      // row_bcast:15
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);      // row_bcast:31
  return v;
}

}  // namespace bqm
