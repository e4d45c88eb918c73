// Rotary positions.  The first `rotary` columns of a head are pairs, columns (i, i + rotary / 2) or
// (2 i, 2 i + 1); pair i of a token at position p is turned by the angle p f_i and scaled:
//
//   y1 = s (x1 cos - x2 sin),  y2 = s (x1 sin + x2 cos)
//
// and the gradient goes through the transposed matrix: the same with -sin.  The other columns are
// copied.  A row is read and written once, which bounds the time: 16384 tokens of 32 heads of 128 bf16 columns, half of
// them turned, 53 us, 5.1 TB/s (fp32 125 us, 4.3 TB/s); one token 2.1 us.  Elements one by one, where rows do not start on 16 bytes
// or the turned columns are no whole loads: 92 us; 32 x 80 with 40 turned 56 us, 12 x 26 10 us, 2 to 3 TB/s.
//
// A workgroup takes a few tokens: its threads first compute one angle each into LDS (cos and sin cost about
// 50 instructions, and the heads share them), then turn the tokens' heads.
#include "kv_common.h"

namespace bqm {
namespace {

constexpr int kRopeThreads = 256;

struct RopeArgs {
  Rope R;
  int tokens, heads, dim;
  int64_t xt, xh, yt, yh;                 // strides of tokens and heads
};

template <typename T, int N>
__device__ __forceinline__ void store_n(T *p, const float (&v)[N]) {
  typedef T txn __attribute__((ext_vector_type(N)));
  if constexpr (N == 1) {
    *p = from_sum<T>(v[0]);
  } else {
    txn o;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = from_sum<T>(v[i]);
    *reinterpret_cast<txn *>(p) = o;
  }
}

// N: columns a load, 8 or 1; per: tokens a workgroup
template <typename T, int N>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs A, int per, const T *x, T *y) {
  extern __shared__ float2 cs[];          // [per][rotary / 2]
  const int half = A.R.rotary / 2;
  const int t0 = blockIdx.x * per, n = min(per, A.tokens - t0);
  for (int i = threadIdx.x; i < n * half; i += kRopeThreads) {
    const int t = i / half, j = i - t * half;
    turn(A.R.positions[t0 + t], turns_of(A.R.freqs[j]), A.R.mscale, A.R.sign, &cs[i].x, &cs[i].y);
  }
  __syncthreads();
  const int units = (A.dim + 2 * N - 1) / (2 * N);
  for (int i = threadIdx.x; i < n * A.heads * units; i += kRopeThreads) {
    const int th = i / units, u = i - th * units, t = th / A.heads, h = th - t * A.heads;
    int c1, c2;
    const bool turned = unit_columns<N>(A.R, u, &c1, &c2);
    const T *xr = x + (t0 + t) * A.xt + h * A.xh;
    T *yr = y + (t0 + t) * A.yt + h * A.yh;
    float a[N] = {}, b[N] = {};
    if constexpr (N == 1) {
      a[0] = to_f32(xr[c1]);
      if (c2 < A.dim) b[0] = to_f32(xr[c2]);
    } else {
      load_vec<N>(xr + c1, a);
      if (c2 < A.dim) load_vec<N>(xr + c2, b);
    }
    if (turned) unit_turn<N>(A.R, cs + t * half + u * N, a, b);
    store_n<T, N>(yr + c1, a);
    if (c2 < A.dim) store_n<T, N>(yr + c2, b);
  }
}

template <typename T>
hipError_t run(const RopeArgs &A, const void *x, void *y, hipStream_t s) {
  // an angle a thread where there are tokens enough for a workgroup on every CU; loads of 8 columns where rows start on
  // 16 bytes and pairs come in whole loads, else of one
  const int half = A.R.rotary / 2;
  const int per = A.tokens <= 512 ? 1 : max(1, kRopeThreads / max(half, 32));
  const unsigned grid = (unsigned)((A.tokens + per - 1) / per), lds = (unsigned)(per * half * sizeof(float2));
  const int64_t unit = 16 / (int)sizeof(T);
  const bool vec = A.R.rotary % 16 == 0 && A.dim % 8 == 0 && (((uintptr_t)x | (uintptr_t)y) & 15u) == 0 &&
                   A.xt % unit == 0 && A.xh % unit == 0 && A.yt % unit == 0 && A.yh % unit == 0;
  if (vec) rope_kernel<T, 8><<<grid, kRopeThreads, lds, s>>>(A, per, (const T *)x, (T *)y);
  else rope_kernel<T, 1><<<grid, kRopeThreads, lds, s>>>(A, per, (const T *)x, (T *)y);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const void *x, int dtype, int tokens, int heads, int dim, int64_t xt, int64_t xh,
                       const int32_t *positions, const double *freqs, int rotary, bool interleaved, float mscale,
                       bool backward, void *y, int64_t yt, int64_t yh, hipStream_t s) {
  const RopeArgs A{{positions, freqs, rotary, interleaved, mscale, backward ? -1.0f : 1.0f}, tokens, heads, dim, xt, xh, yt, yh};
  if (dtype == BQM_F32) return run<float>(A, x, y, s);
  if (dtype == BQM_BF16) return run<__bf16>(A, x, y, s);
  return run<_Float16>(A, x, y, s);
}

}  // namespace bqm
