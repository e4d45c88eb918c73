// Products of E4M3 activations and weights with a scale for each block of 128,
// dense and grouped by expert.
//
//   y[t, r] = sum_b sx[b, t] * sw[r / 128, b] * sum_{j < 128} q[t, 128 b + j] * w[r, 128 b + j]
//
// A block's products are summed in fp32, the sum is scaled in fp32 and the blocks
// are added in fp32; y is rounded once.  One thread an element: the plain kernel.
#include "lowp_types.h"

namespace bqm {
namespace {

constexpr int kBlk = 128;

struct Fp8Args {
  const uint8_t *w;          // [experts, rows, 128 kb]
  const float *ws;           // [experts, ceil(rows / 128), kb]
  const uint8_t *q;          // [m, 128 kb]
  const float *qs;           // [kb, m]
  const int32_t *offsets;    // [experts + 1], or null: one matrix, rows of y = m
  const int32_t *row_ids;    // [slots], or null: row p of y is activation row p
  int experts, rows, kb, m, slots;
};

// The first and last+1 row of y of expert e, within [0, slots] whatever the array holds.
__device__ __forceinline__ int clamp_off(const Fp8Args &A, int e) {
  const int v = A.offsets[e];
  return v < 0 ? 0 : v > A.slots ? A.slots : v;
}

template <typename Y>
__global__ __launch_bounds__(256) void fp8_plain_kernel(Fp8Args A, Y *__restrict__ y) {
  const int r = (int)blockIdx.y * 256 + (int)threadIdx.x;
  const int p = blockIdx.x;
  int e = 0, t = p;
  if (A.offsets) {
    if (p >= clamp_off(A, A.experts)) return;
    while (e < A.experts && p >= clamp_off(A, e + 1)) ++e;
    if (e >= A.experts || p < clamp_off(A, e)) return;
  }
  if (A.row_ids) t = A.row_ids[p];
  if (r >= A.rows) return;
  t = t < 0 ? 0 : t >= A.m ? A.m - 1 : t;
  const int64_t kp = (int64_t)A.kb * kBlk;
  const uint8_t *w = A.w + ((int64_t)e * A.rows + r) * kp;
  const uint8_t *q = A.q + t * kp;
  const float *ws = A.ws + ((int64_t)e * ((A.rows + kBlk - 1) / kBlk) + r / kBlk) * A.kb;
  float acc = 0.0f;
  for (int b = 0; b < A.kb; ++b) {
    float part = 0.0f;
    for (int j = 0; j < kBlk; j += 4) {
      const int a = *reinterpret_cast<const int *>(w + b * kBlk + j);
      const int c = *reinterpret_cast<const int *>(q + b * kBlk + j);
      part = fmaf(__builtin_amdgcn_cvt_f32_fp8(a, 0), __builtin_amdgcn_cvt_f32_fp8(c, 0), part);
      part = fmaf(__builtin_amdgcn_cvt_f32_fp8(a, 1), __builtin_amdgcn_cvt_f32_fp8(c, 1), part);
      part = fmaf(__builtin_amdgcn_cvt_f32_fp8(a, 2), __builtin_amdgcn_cvt_f32_fp8(c, 2), part);
      part = fmaf(__builtin_amdgcn_cvt_f32_fp8(a, 3), __builtin_amdgcn_cvt_f32_fp8(c, 3), part);
    }
    acc = fmaf(part, ws[b] * A.qs[(int64_t)b * A.m + t], acc);
  }
  y[(int64_t)p * A.rows + r] = from_f32<Y>(acc);
}

template <typename Y>
hipError_t run(const Fp8Args &A, Y *y, hipStream_t s) {
  fp8_plain_kernel<Y><<<dim3(A.slots, (A.rows + 255) / 256), 256, 0, s>>>(A, y);
  return hipGetLastError();
}

hipError_t run_any(const Fp8Args &A, void *y, int ydtype, hipStream_t s) {
  if (ydtype == BQM_F32) return run(A, (float *)y, s);
  if (ydtype == BQM_BF16) return run(A, (__bf16 *)y, s);
  return run(A, (_Float16 *)y, s);
}

}  // namespace

hipError_t launch_fp8_gemm(const uint8_t *w, const float *ws, int rows, int cols, const uint8_t *q, const float *qs,
                           int m, void *y, int ydtype, int num_cus, hipStream_t s) {
  const Fp8Args A{w, ws, q, qs, nullptr, nullptr, 1, rows, (cols + kBlk - 1) / kBlk, m, m};
  return run_any(A, y, ydtype, s);
}

hipError_t launch_fp8_gemm_grouped(const uint8_t *w, const float *ws, int experts, int rows, int cols,
                                   const uint8_t *q, const float *qs, int m, const int32_t *offsets,
                                   const int32_t *row_ids, int slots, void *y, int ydtype, int num_cus,
                                   hipStream_t s) {
  const Fp8Args A{w, ws, q, qs, offsets, row_ids, experts, rows, (cols + kBlk - 1) / kBlk, m, slots};
  return run_any(A, y, ydtype, s);
}

}  // namespace bqm
