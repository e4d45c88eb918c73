// E4M3 codes with one fp32 scale a block of 128.
//
// Activations: a block is 128 consecutive columns of one token.  With
// a = max |v| over the block, s = max(RN(a / 448), 2^-126) (1 for a block of
// zeros) and q = E4M3(clamp(RN(v / s), -448, 448)): the largest entry lands on
// the type's largest value, and no quotient is formed with a subnormal scale.
// A block with a NaN or an infinity has a NaN scale and NaN codes, so that every
// product that reads it is NaN instead of a plausible number.  Rows are padded
// with code 0 to whole blocks, so the products need no case for a short last
// block; scales are stored [block][token], which is how the products read them:
// one block's scales of neighbouring tokens at a time.
// With SwiGLU, v = g / (1 + exp(-g)) * u from rows [g | u].
//
// Weights: a block is 128 x 128, the same formula.
#include "lowp_types.h"

namespace bqm {
namespace {

constexpr int kBlk = 128;
constexpr float kE4M3Max = 448.0f;

// max over 16 consecutive lanes; NaN if any is NaN
__device__ __forceinline__ float max16_nan(float a) {
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) {
    const float b = __shfl_xor(a, o, 16);
    a = (a > b || a != a) ? a : b;
  }
  return a;
}

__device__ __forceinline__ float block_scale(float a) {
  if (!(a <= 3.4028234663852886e38f)) return __builtin_nanf("");
  return a > 0.0f ? fmaxf(__fdiv_rn(a, kE4M3Max), 1.17549435e-38f) : 1.0f;
}

// The codes of 8 values of a block with scale s.  RN(v / s) without a division an
// element: with y = RN(1 / s) and q = v y, one step q + (v - q s) y is the correctly
// rounded quotient (Markstein), as long as the remainder v - q s is no subnormal; tiny
// scales divide.
__device__ __forceinline__ u32x2_t codes8(const float (&v)[8], float s) {
  if (s != s) return u32x2_t{0x7F7F7F7Fu, 0x7F7F7F7Fu};
  const bool tiny = s < 0x1p-60f;
  const float y = __fdiv_rn(1.0f, s);
  float c[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float q = v[j] * y;
    c[j] = fmaf(fmaf(-q, s, v[j]), y, q);
  }
  if (tiny) {
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = __fdiv_rn(v[j], s);
  }
  u32x2_t p;
#pragma unroll
  for (int j = 0; j < 8; ++j) c[j] = __builtin_amdgcn_fmed3f(c[j], -kE4M3Max, kE4M3Max);
#pragma unroll
  for (int h = 0; h < 2; ++h) p[h] = e4m3_pair(c[4 * h], c[4 * h + 1]) | e4m3_pair(c[4 * h + 2], c[4 * h + 3]) << 16;
  return p;
}

// 8 elements from column c of a row of k, zeros past it
template <typename T, bool kVec>
__device__ __forceinline__ void load8(const T *row, int c, int k, float (&v)[8]) {
  if (kVec && c + 8 <= k) {
    load_vec<8>(row + c, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j < k ? to_f32(row[c + j]) : 0.0f;
  }
}

// g / d for d = 1 + exp(-g): the reciprocal refined once, then the quotient, within
// 0.51 units; past 2^100 (g < -69) and for NaN the plain division.
__device__ __forceinline__ float silu_mul(float g, float u) {
  const float d = 1.0f + expf(-g);
  float r = __builtin_amdgcn_rcpf(d);
  r = fmaf(fmaf(-d, r, 1.0f), r, r);
  float q = g * r;
  q = fmaf(fmaf(-q, d, g), r, q);
  if (!(d < 0x1p100f) || !(fabsf(g) < 0x1p100f)) q = g / d;
  return q * u;
}

// 16 lanes hold a block; a workgroup of 256 takes `rows` tokens x 16 / rows blocks.
template <typename T, bool kVec, bool kSwiglu>
__global__ __launch_bounds__(256) void fp8_quant_kernel(const T *__restrict__ x, int m, int k, int64_t stride,
                                                        int rows, uint8_t *__restrict__ q,
                                                        float *__restrict__ scale) {
  const int kb = (k + kBlk - 1) / kBlk;
  const int grp = threadIdx.x >> 4, sub = threadIdx.x & 15;
  // neighbouring workgroups take neighbouring blocks of the same rows: rows are often
  // a multiple of 8 KiB apart, and one column of many of them lies in few memory channels
  // (2048 x 14336 with SwiGLU 47 us with neighbouring rows)
  const int per = 16 / rows, across = (kb + per - 1) / per;
  const int row = (int)(blockIdx.x / across) * rows + grp % rows;
  const int b = (int)(blockIdx.x % across) * per + grp / rows;
  if (row >= m || b >= kb) return;                 // whole 16-lane groups leave together
  const T *xr = x + (int64_t)row * stride;
  const int c = b * kBlk + sub * 8;
  float v[8];
  load8<T, kVec>(xr, c, k, v);
  if constexpr (kSwiglu) {
    float u[8];
    if (kVec) {
      load8<T, kVec>(xr + k, c, k, u);
    } else {
      load8<T, false>(xr + k, c, k, u);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = silu_mul(v[j], u[j]);
  }
  float a = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float w = fabsf(v[j]);
    a = (a > w || a != a) ? a : w;
  }
  const float s = block_scale(max16_nan(a));
  *reinterpret_cast<u32x2_t *>(q + ((int64_t)row * kb + b) * kBlk + sub * 8) = codes8(v, s);
  if (sub == 0) scale[(int64_t)b * m + row] = s;
}

// One workgroup of 256 per 128 x 128 block: 16 lanes a row, 8 rows each.
template <typename T>
__global__ __launch_bounds__(256) void fp8_pack_kernel(const T *__restrict__ w, int rows, int cols,
                                                       uint8_t *__restrict__ q, float *__restrict__ scale) {
  const int kb = (cols + kBlk - 1) / kBlk, nb = (rows + kBlk - 1) / kBlk;
  const int b = blockIdx.x % kb, rb = blockIdx.x / kb;
  const int64_t e = blockIdx.y;
  const int grp = threadIdx.x >> 4, sub = threadIdx.x & 15;
  const T *we = w + e * rows * (int64_t)cols;
  const int c = b * kBlk + sub * 8;
  float v[8][8];
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = rb * kBlk + i * 16 + grp;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[i][j] = r < rows && c + j < cols ? to_f32(we[(int64_t)r * cols + c + j]) : 0.0f;
      const float x = fabsf(v[i][j]);
      a = (a > x || a != a) ? a : x;
    }
  }
  a = max16_nan(a);
  __shared__ float red[16];
  if (sub == 0) red[grp] = a;
  __syncthreads();
  a = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) a = (a > red[i] || a != a) ? a : red[i];
  const float s = block_scale(a);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = rb * kBlk + i * 16 + grp;
    if (r < rows)
      *reinterpret_cast<u32x2_t *>(q + ((e * rows + r) * kb + b) * kBlk + sub * 8) = codes8(v[i], s);
  }
  if (threadIdx.x == 0) scale[(e * nb + rb) * kb + b] = s;
}

template <typename T>
hipError_t quant_t(const T *x, int m, int k, int64_t stride, bool swiglu, uint8_t *q, float *scale, hipStream_t s) {
  const int kb = (k + kBlk - 1) / kBlk;
  const int rows = m >= 16 ? 16 : 1;
  const unsigned grid = (unsigned)((m + rows - 1) / rows) * (unsigned)((kb + 16 / rows - 1) / (16 / rows));
  // 16-byte loads where every row (and, with SwiGLU, its second half) starts on 16 bytes
  const int per = 16 / (int)sizeof(T);
  const bool vec = ((uintptr_t)x & 15u) == 0 && (m == 1 || stride % per == 0) && (!swiglu || k % per == 0);
  if (swiglu) {
    if (vec) fp8_quant_kernel<T, true, true><<<grid, 256, 0, s>>>(x, m, k, stride, rows, q, scale);
    else fp8_quant_kernel<T, false, true><<<grid, 256, 0, s>>>(x, m, k, stride, rows, q, scale);
  } else {
    if (vec) fp8_quant_kernel<T, true, false><<<grid, 256, 0, s>>>(x, m, k, stride, rows, q, scale);
    else fp8_quant_kernel<T, false, false><<<grid, 256, 0, s>>>(x, m, k, stride, rows, q, scale);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t pack_t(const T *w, int experts, int rows, int cols, uint8_t *q, float *scale, hipStream_t s) {
  const int64_t kb = (cols + kBlk - 1) / kBlk, nb = (rows + kBlk - 1) / kBlk;
  fp8_pack_kernel<T><<<dim3((unsigned)(kb * nb), experts), 256, 0, s>>>(w, rows, cols, q, scale);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_quant(const void *x, int dtype, int m, int k, int64_t stride, bool swiglu, uint8_t *q,
                            float *scale, hipStream_t s) {
  if (dtype == BQM_F32) return quant_t((const float *)x, m, k, stride, swiglu, q, scale, s);
  if (dtype == BQM_BF16) return quant_t((const __bf16 *)x, m, k, stride, swiglu, q, scale, s);
  return quant_t((const _Float16 *)x, m, k, stride, swiglu, q, scale, s);
}

hipError_t launch_fp8_pack(const void *w, int dtype, int experts, int rows, int cols, uint8_t *q, float *scale,
                           hipStream_t s) {
  if (dtype == BQM_F32) return pack_t((const float *)w, experts, rows, cols, q, scale, s);
  if (dtype == BQM_BF16) return pack_t((const __bf16 *)w, experts, rows, cols, q, scale, s);
  return pack_t((const _Float16 *)w, experts, rows, cols, q, scale, s);
}

}  // namespace bqm
