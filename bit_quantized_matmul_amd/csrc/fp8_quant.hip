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

// |v| as an integer: ordered as the values are, infinities and NaN above all others,
// so an integer maximum finds a block's largest value and whether it is finite.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

template <int CTRL>
__device__ __forceinline__ uint32_t max_row_ror(uint32_t a) {
  const uint32_t b = (uint32_t)__builtin_amdgcn_update_dpp((int)a, (int)a, CTRL, 0xF, 0xF, false);
  return a > b ? a : b;
}

// max over 16 consecutive lanes
__device__ __forceinline__ uint32_t max16(uint32_t a) {
  return max_row_ror<0x128>(max_row_ror<0x124>(max_row_ror<0x122>(max_row_ror<0x121>(a))));
}

__device__ __forceinline__ uint32_t magnitude8(const float (&v)[8], uint32_t a) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t b = magnitude(v[j]);
    a = a > b ? a : b;
  }
  return a;
}

__device__ __forceinline__ float block_scale(uint32_t a) {
  if (a >= 0x7F800000u) return __builtin_nanf("");
  return a ? fmaxf(__fdiv_rn(__uint_as_float(a), kE4M3Max), 0x1p-126f) : 1.0f;
}

// The codes of 8 values of a block with scale s.  RN(v / s) without a division an
// element: with y = RN(1 / s) and q = v y, one step q + (v - q s) y is the correctly
// rounded quotient (Markstein), as long as the remainder v - q s is no subnormal; tiny
// scales divide.
__device__ __forceinline__ u32x2_t codes8(const float (&v)[8], float s) {
  float c[8];
  const float y = __fdiv_rn(1.0f, s);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float q = v[j] * y;
    c[j] = fmaf(fmaf(-q, s, v[j]), y, q);
  }
  if (!(s >= 0x1p-60f)) {
    if (s != s) return u32x2_t{0x7F7F7F7Fu, 0x7F7F7F7Fu};
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = __fdiv_rn(v[j], s);
  }
  u32x2_t p;
#pragma unroll
  for (int j = 0; j < 8; ++j) c[j] = __builtin_amdgcn_fmed3f(c[j], -kE4M3Max, kE4M3Max);
#pragma unroll
  for (int h = 0; h < 2; ++h) p[h] = e4m3_quad(c[4 * h], c[4 * h + 1], c[4 * h + 2], c[4 * h + 3]);
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

// silu(g) u = g / (1 + exp(-g)) u.  exp(-g) = 2^p with p = -g log2(e) in two parts, the
// rounded product and what it lost; the quotient is one step from g times the
// approximate reciprocal.  Each of the three is within about a unit.  From 69 on the quotient
// is g.  Below -69, where exp(-g) may overflow and the value does not vanish, 1 + exp(-g) is
// exp(-g), and g exp(g) u = (g h u) h with h = exp(g / 2) leaves the range only where the
// value does.
__device__ __forceinline__ void silu_mul8(float (&g)[8], const float (&u)[8]) {
  constexpr float kL = 0x1.715476p+0f, kLlo = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;   // log2(e) = kL + kLlo
  float q[8], far = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float p = -g[j] * kL;
    const float lost = fmaf(-g[j], kLlo, fmaf(-g[j], kL, -p));
    const float e = __builtin_amdgcn_exp2f(p);
    const float d = 1.0f + fmaf(e, lost * kLn2, e);
    const float r = __builtin_amdgcn_rcpf(d);
    const float a = g[j] * r;
    q[j] = fmaf(fmaf(-a, d, g[j]), r, a);
    far = fmaxf(far, fabsf(g[j]));
    if (g[j] != g[j]) far = INFINITY;
  }
  if (!(far < 69.0f)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float h = expf(0.5f * g[j]);
      const float near = (g[j] >= 69.0f ? g[j] : q[j]) * u[j];
      g[j] = g[j] < -69.0f ? g[j] * h * u[j] * h : near;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) g[j] = q[j] * u[j];
}

// 16 lanes hold a block; a workgroup of 256 takes kRows tokens x 16 / kRows blocks.
// Neighbouring workgroups take neighbouring blocks of the same rows.
template <typename T, bool kVec, bool kSwiglu, int kRows>
__global__ __launch_bounds__(256) void fp8_quant_kernel(const T *__restrict__ x, int m, int k, int64_t stride,
                                                        uint8_t *__restrict__ q, float *__restrict__ scale) {
  const int kb = (k + kBlk - 1) / kBlk;
  const int grp = threadIdx.x >> 4, sub = threadIdx.x & 15;
  const int b = (int)blockIdx.x * (16 / kRows) + grp / kRows;
  const int c = b * kBlk + sub * 8;
  if (b >= kb) return;                               // whole 16-lane groups leave together
  for (int64_t row = (int64_t)blockIdx.y * kRows + grp % kRows; row < m; row += (int64_t)gridDim.y * kRows) {
    const T *xr = x + row * stride;
    float v[8];
    load8<T, kVec>(xr, c, k, v);
    if constexpr (kSwiglu) {
      float u[8];
      load8<T, kVec>(xr + k, c, k, u);
      silu_mul8(v, u);
    }
    const float s = block_scale(max16(magnitude8(v, 0)));
    *reinterpret_cast<u32x2_t *>(q + (row * kb + b) * kBlk + sub * 8) = codes8(v, s);
    if (sub == 0) scale[(int64_t)b * m + row] = s;
  }
}

// One workgroup of 256 per 128 x 128 block: 16 lanes a row, 8 rows each.  Weights are packed
// once, of any alignment, by loads of elements: 14336x4096 bf16 80 us, 2.2 TB/s.
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
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = rb * kBlk + i * 16 + grp;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[i][j] = r < rows && c + j < cols ? to_f32(we[(int64_t)r * cols + c + j]) : 0.0f;
    a = magnitude8(v[i], a);
  }
  a = max16(a);
  __shared__ uint32_t red[16];
  if (sub == 0) red[grp] = a;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 16; ++i) a = a > red[i] ? a : red[i];
  const float s = block_scale(a);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = rb * kBlk + i * 16 + grp;
    if (r < rows)
      *reinterpret_cast<u32x2_t *>(q + ((e * rows + r) * kb + b) * kBlk + sub * 8) = codes8(v[i], s);
  }
  if (threadIdx.x == 0) scale[(e * nb + rb) * kb + b] = s;
}

template <typename T, int kRows>
hipError_t quant_rows(const T *x, int m, int k, int64_t stride, bool swiglu, uint8_t *q, float *scale, hipStream_t s) {
  const int kb = (k + kBlk - 1) / kBlk;
  const int64_t tiles = ((int64_t)m + kRows - 1) / kRows;
  const dim3 grid((kb + 16 / kRows - 1) / (16 / kRows), (unsigned)(tiles < 65535 ? tiles : 65535));
  // 16-byte loads where every row (and, with SwiGLU, its second half) starts on 16 bytes, else
  // elements (us, bf16: 4096x4096 10.6 and 24; SwiGLU 2048x14336 26 and 65)
  const int per = 16 / (int)sizeof(T);
  const bool vec = ((uintptr_t)x & 15u) == 0 && (m == 1 || stride % per == 0) && (!swiglu || k % per == 0);
  if (swiglu) {
    if (vec) fp8_quant_kernel<T, true, true, kRows><<<grid, 256, 0, s>>>(x, m, k, stride, q, scale);
    else fp8_quant_kernel<T, false, true, kRows><<<grid, 256, 0, s>>>(x, m, k, stride, q, scale);
  } else {
    if (vec) fp8_quant_kernel<T, true, false, kRows><<<grid, 256, 0, s>>>(x, m, k, stride, q, scale);
    else fp8_quant_kernel<T, false, false, kRows><<<grid, 256, 0, s>>>(x, m, k, stride, q, scale);
  }
  return hipGetLastError();
}

// 16 tokens a workgroup, so that it stores 16 neighbouring scales; few tokens: 16 blocks of one.
template <typename T>
hipError_t quant_t(const T *x, int m, int k, int64_t stride, bool swiglu, uint8_t *q, float *scale, hipStream_t s) {
  return m >= 16 ? quant_rows<T, 16>(x, m, k, stride, swiglu, q, scale, s)
                 : quant_rows<T, 1>(x, m, k, stride, swiglu, q, scale, s);
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
