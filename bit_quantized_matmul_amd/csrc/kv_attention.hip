// Attention over the paged 8-bit cache.
//
//   o[t, h] = sum_j p_j v_j,   p = softmax_j(scale q[t, h] . k_j),   position - window < j <= position
//
// One wave a row and head: a lane takes a token of a page for the scores and columns for the sum, with the
// running maximum m and sum l of the softmax: a page with a larger maximum scales what was summed before
// by exp(m - m').
#include "kv_common.h"

namespace bqm {
namespace {

struct AttnArgs {
  KvBatch B;
  int heads, kv_heads, dim, dp, window;
  int64_t qt, qh;                         // strides of q's tokens and heads
  float scale;                            // times log2(e)
  const uint8_t *kc, *vc;
  const float *ks, *vs;
};

template <typename T>
__global__ __launch_bounds__(64) void kv_attention_kernel(AttnArgs A, const T *__restrict__ q, T *__restrict__ out) {
  __shared__ float qs[kMaxKvDim], p[kPage];
  KvSeq s;
  int i;
  if (!kv_find(A.B, blockIdx.x, 1, [](const KvSeq &x) { return x.n; }, &s, &i)) return;
  const int h = blockIdx.y, kh = h / (A.heads / A.kv_heads), lane = threadIdx.x;
  const int64_t row = s.lo + i;
  for (int c = lane; c < A.dp; c += 64) qs[c] = c < A.dim ? to_f32(q[row * A.qt + h * A.qh + c]) : 0.0f;
  const int pos = s.first() + i, end = min(pos + 1, kv_limit(A.B, s));
  const int begin = A.window ? max(0, pos - A.window + 1) : 0;
  float m = -INFINITY, l = 0.0f, o[kMaxKvDim / 64] = {};
  for (int pi = begin / kPage; pi * kPage < end; ++pi) {
    const int page = kv_page(A.B, s, pi);
    if (page < 0) continue;
    const int64_t ph = (int64_t)page * A.kv_heads + kh;
    const int j = pi * kPage + lane;
    const bool see = j >= begin && j < end;
    __syncthreads();
    float sum = 0.0f;
    const int *kr = reinterpret_cast<const int *>(A.kc + (ph * kPage + lane) * A.dp);
    for (int c = 0; c < A.dp; c += 4) {
      const int w = kr[c / 4];
      sum = fmaf(qs[c], __builtin_amdgcn_cvt_f32_fp8(w, 0), sum);
      sum = fmaf(qs[c + 1], __builtin_amdgcn_cvt_f32_fp8(w, 1), sum);
      sum = fmaf(qs[c + 2], __builtin_amdgcn_cvt_f32_fp8(w, 2), sum);
      sum = fmaf(qs[c + 3], __builtin_amdgcn_cvt_f32_fp8(w, 3), sum);
    }
    const float x = see ? sum * (A.ks[ph] * A.scale) : -INFINITY;
    const float m1 = fmaxf(m, wave_max(x)), ref = m1 > -INFINITY ? m1 : 0.0f;
    const float e = exp2f(x - ref), alpha = exp2f(m - ref);
    p[lane] = e;
    l = fmaf(l, alpha, group_sum<64>(e));
    m = m1;
    __syncthreads();
    const float vs = A.vs[ph];
    const int lo = max(0, begin - pi * kPage), hi = min(kPage, end - pi * kPage);
#pragma unroll
    for (int d = 0; d < kMaxKvDim / 64; ++d) {
      const int c = d * 64 + lane;
      if (c >= A.dim) continue;
      const uint8_t *vr = A.vc + (ph * A.dp + c) * kPage;
      float part = 0.0f;
      for (int t = lo; t < hi; ++t) part = fmaf(p[t], __builtin_amdgcn_cvt_f32_fp8((int)vr[t], 0), part);
      o[d] = fmaf(part, vs, o[d] * alpha);
    }
  }
#pragma unroll
  for (int d = 0; d < kMaxKvDim / 64; ++d) {
    const int c = d * 64 + lane;
    if (c < A.dim) out[(row * A.heads + h) * A.dim + c] = from_sum<T>(l != 0.0f ? o[d] / l : 0.0f);
  }
}

template <typename T>
hipError_t run(const AttnArgs &A, const void *q, void *out, hipStream_t s) {
  kv_attention_kernel<T><<<dim3((unsigned)A.B.tokens, (unsigned)A.heads), 64, 0, s>>>(A, (const T *)q, (T *)out);
  return hipGetLastError();
}

}  // namespace

int64_t kv_attention_scratch(int, int, int, int, int, int) { return 0; }

hipError_t launch_kv_attention(const KvBatch &B, const void *q, int dtype, int heads, int dim, int64_t qt, int64_t qh,
                               const uint8_t *kc, const uint8_t *vc, const float *ks, const float *vs, int kv_heads,
                               float scale, int window, void *out, void *, hipStream_t s) {
  const AttnArgs A{B, heads, kv_heads, dim, kv_padded_dim(dim), window, qt, qh, scale * 1.44269504f, kc, vc, ks, vs};
  if (dtype == BQM_F32) return run<float>(A, q, out, s);
  if (dtype == BQM_BF16) return run<__bf16>(A, q, out, s);
  return run<_Float16>(A, q, out, s);
}

}  // namespace bqm
