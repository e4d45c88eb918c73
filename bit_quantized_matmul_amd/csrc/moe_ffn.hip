// The expert layer of a few tokens, from router logits to combined rows:
//
//   out[t] = sum_j w[t, j] W2[e_j] (silu(G[e_j] x_t) * (U[e_j] x_t)),   W13 = [G | U]
//
// with the top experts e_j of a token and their weights as moe_route gives them, weights in E4M3 with a
// scale for each 128 x 128 block, and everything else in fp32.
#include "lowp_types.h"

namespace bqm {
namespace {

constexpr int kBlk = 128;
constexpr float kHuge = 3.4028234663852886e38f;

struct MoeArgs {
  const void *logits;
  int ltype;                              // the logits' type
  int64_t xs, ls;                         // strides of x's and logits' rows
  int tokens, experts, top, renorm, hidden, ffn;
  const uint8_t *w13, *w2;
  const float *s13, *s2;
  int32_t *ids;                           // workspace: [tokens, top]
  float *weights, *act;                   // [tokens, top], [tokens, top, ffn]
};

__device__ __forceinline__ float logit(const MoeArgs &A, int64_t i) {
  if (A.ltype == BQM_F32) return ((const float *)A.logits)[i];
  if (A.ltype == BQM_BF16) return to_f32(((const __bf16 *)A.logits)[i]);
  return to_f32(((const _Float16 *)A.logits)[i]);
}

__global__ __launch_bounds__(64) void moe_pick_kernel(MoeArgs A) {
  const int lane = threadIdx.x;
  float v[16], all = 0.0f, first = 0.0f, total = 0.0f;
  for (int i = 0; i < 16; ++i) {
    const int e = lane + 64 * i;
    const float a = e < A.experts ? logit(A, blockIdx.x * A.ls + e) : -INFINITY;
    v[i] = a != a ? -INFINITY : fminf(a, kHuge);
  }
  for (int j = 0; j < A.top; ++j) {
    float b = -INFINITY;
    int at = 1 << 30;
    for (int i = 0; i < 16; ++i)
      if (v[i] > b) b = v[i], at = lane + 64 * i;
    const float w = wave_max(b);
    at = b == w ? at : 1 << 30;
    for (int o = 32; o >= 1; o >>= 1) at = min(at, __shfl_xor(at, o, 64));
    if (j == 0) {
      first = w > -INFINITY ? w : 0.0f;
      for (int i = 0; i < 16; ++i) all += expf(v[i] - first);
      all = group_sum<64>(all);
    }
    for (int i = 0; i < 16; ++i)
      if (at == lane + 64 * i) v[i] = -INFINITY;
    const float p = w > -INFINITY ? expf(w - first) : 0.0f;
    total += p;
    if (lane == 0) {
      A.ids[blockIdx.x * A.top + j] = w > -INFINITY ? at : -1;
      A.weights[blockIdx.x * A.top + j] = p;
    }
  }
  __syncthreads();
  const float by = A.renorm ? total : all;
  for (int j = lane; j < A.top; j += 64) {
    float *p = A.weights + blockIdx.x * A.top + j;
    *p = *p > 0.0f ? *p / by : 0.0f;
  }
}

// sum over a row's codes: lanes take neighbouring columns of a block
template <typename X>
__device__ __forceinline__ float row_dot(const uint8_t *w, const float *s, int k, X x) {
  const int lane = threadIdx.x & 63;
  float acc = 0.0f;
  for (int b = 0; b * kBlk < k; ++b) {
    float part = 0.0f;
    for (int i = lane; i < kBlk && b * kBlk + i < k; i += 64)
      part = fmaf(__builtin_amdgcn_cvt_f32_fp8((int)w[b * kBlk + i], 0), x(b * kBlk + i), part);
    acc = fmaf(part, s[b], acc);
  }
  return group_sum<64>(acc);
}

template <typename T>
__global__ __launch_bounds__(64) void moe_up_kernel(MoeArgs A, const T *__restrict__ x) {
  const int pair = blockIdx.y, f = blockIdx.x, e = A.ids[pair];
  if (e < 0) return;
  const int kb = (A.hidden + kBlk - 1) / kBlk, nb = (2 * A.ffn + kBlk - 1) / kBlk;
  const T *xr = x + pair / A.top * A.xs;
  float h[2];
  for (int i = 0; i < 2; ++i) {
    const int r = f + i * A.ffn;
    h[i] = row_dot(A.w13 + ((int64_t)e * 2 * A.ffn + r) * kb * kBlk, A.s13 + ((int64_t)e * nb + r / kBlk) * kb, A.hidden,
                   [&](int c) { return to_f32(xr[c]); });
  }
  if (threadIdx.x == 0) A.act[(int64_t)pair * A.ffn + f] = h[0] / (1.0f + expf(-h[0])) * h[1];
}

template <typename T>
__global__ __launch_bounds__(64) void moe_down_kernel(MoeArgs A, T *__restrict__ out) {
  const int t = blockIdx.y, r = blockIdx.x;
  const int kb = (A.ffn + kBlk - 1) / kBlk, nb = (A.hidden + kBlk - 1) / kBlk;
  float sum = 0.0f;
  for (int j = 0; j < A.top; ++j) {
    const int pair = t * A.top + j, e = A.ids[pair];
    if (e < 0) continue;
    const float *a = A.act + (int64_t)pair * A.ffn;
    sum = fmaf(A.weights[pair], row_dot(A.w2 + ((int64_t)e * A.hidden + r) * kb * kBlk, A.s2 + ((int64_t)e * nb + r / kBlk) * kb,
                                        A.ffn, [&](int c) { return a[c]; }), sum);
  }
  if (threadIdx.x == 0) out[(int64_t)t * A.hidden + r] = from_sum<T>(sum);
}

template <typename T>
hipError_t run(const MoeArgs &A, const void *x, void *out, hipStream_t s) {
  moe_pick_kernel<<<A.tokens, 64, 0, s>>>(A);
  moe_up_kernel<T><<<dim3(A.ffn, A.tokens * A.top), 64, 0, s>>>(A, (const T *)x);
  moe_down_kernel<T><<<dim3(A.hidden, A.tokens), 64, 0, s>>>(A, (T *)out);
  return hipGetLastError();
}

}  // namespace

int64_t moe_ffn_scratch(int tokens, int, int top, int, int ffn) { return (int64_t)tokens * top * (8 + 4 * (int64_t)ffn); }

hipError_t launch_moe_ffn(const void *x, int dtype, int tokens, int hidden, int64_t xs, const void *logits, int ltype, int64_t ls,
                          int experts, int top, bool renorm, const uint8_t *w13, const float *s13, const uint8_t *w2,
                          const float *s2, int ffn, void *out, void *scratch, hipStream_t s) {
  int32_t *ids = (int32_t *)scratch;
  float *weights = (float *)(ids + tokens * top);
  const MoeArgs A{logits, ltype, xs, ls, tokens, experts, top, renorm, hidden, ffn, w13, w2, s13, s2, ids, weights, weights + tokens * top};
  if (dtype == BQM_F32) return run<float>(A, x, out, s);
  if (dtype == BQM_BF16) return run<__bf16>(A, x, out, s);
  return run<_Float16>(A, x, out, s);
}

}  // namespace bqm
