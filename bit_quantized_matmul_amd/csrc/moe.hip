// Mixture-of-experts routing and the combination of the experts' rows.
//
// Route.  Per token the k largest logits, their softmax weights, and the
// (token, expert) pairs in a stable order by expert.  Logits are compared as
// they are (never after an exp, which could make unequal ones equal); equal
// ones go to the lower expert; NaN counts as -inf, which is never chosen, and
// +inf as the largest fp32 value, so that exp(l - max) stays defined.
//
// The order is a counting sort over chunks of kChunkTokens tokens: the first
// kernel chooses and counts each chunk's experts, the second adds up the counts
// of the chunks before its own and places the chunk's pairs.  The counts are sums
// of integers, so nothing depends on the order of atomics, and a pair's rank
// among its chunk's is found 64 pairs at a time from ballots over the expert's
// bits.  One chunk needs no second launch.
//
// Combine.  out[t] = sum_j weights[t, j] * y[slots[t, j]] in fp32, j ascending.
#include "lowp_types.h"

namespace bqm {
namespace {

constexpr int kChunkTokens = 64;
constexpr int kMaxExperts = 1024, kMaxTop = 32;
constexpr int kRouteThreads = 1024;
constexpr float kHuge = 3.4028234663852886e38f;

struct RouteArgs {
  const void *logits;
  int64_t stride;
  int tokens, experts, top, renorm;
  int32_t *ids;
  float *weights;
  int32_t *offsets, *row_ids, *slots;
  int32_t *hist;             // [chunks, experts]
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Order-preserving integer of a logit that is no NaN and no -0.
__device__ __forceinline__ int order_key(float v) {
  const int b = __float_as_int(v);
  return b >= 0 ? b : b ^ 0x7FFFFFFF;
}

// One wave chooses one token's experts.  Lane l holds experts l, l + 64, ...
template <typename T, int kPer>
__device__ void choose(const RouteArgs &A, int token, int32_t *ids_lds) {
  const int lane = threadIdx.x & 63;
  const T *x = reinterpret_cast<const T *>(A.logits) + (int64_t)token * A.stride;
  float v[kPer];
  float best = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 64 * i;
    float l = e < A.experts ? to_f32(x[e]) : -INFINITY;
    l = l != l ? -INFINITY : fminf(l, kHuge) + 0.0f;          // -0 becomes +0
    v[i] = l;
    best = fmaxf(best, l);
  }
  const float top = wave_max(best);
  const float ref = top > -INFINITY ? top : 0.0f;
  float total = 0.0f;
  if (!A.renorm) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) total += expf(v[i] - ref);
    total = wave_sum(total);
  }
  float mine = 0.0f;                                           // lane j: the j-th choice
  int my_id = -1;
  for (int j = 0; j < A.top; ++j) {
    float b = -INFINITY;
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (v[i] > b) {
        b = v[i];
        at = lane + 64 * i;
      }
    const float w = wave_max(b);
    if (w == -INFINITY) break;
    at = b == w ? at : 0x7FFFFFFF;
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) at = min(at, __shfl_xor(at, o, 64));
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (at == lane + 64 * i) v[i] = -INFINITY;
    if (lane == j) {
      mine = expf(w - ref);
      my_id = at;
    }
  }
  if (A.renorm) total = wave_sum(mine);
  if (lane < A.top) {
    const int64_t o = (int64_t)token * A.top + lane;
    A.ids[o] = my_id;
    A.weights[o] = my_id >= 0 ? mine / total : 0.0f;
    ids_lds[lane] = my_id;
  }
}

// Places a chunk's pairs; base[e]: the first slot of the chunk's pairs of
// expert e (advanced here).  One wave.
__device__ void place(const RouteArgs &A, int chunk, int pairs, const int32_t *ids, int32_t *base) {
  const int lane = threadIdx.x & 63;
  const int64_t first = (int64_t)chunk * kChunkTokens * A.top;
  for (int p0 = 0; p0 < pairs; p0 += 64) {
    const int p = p0 + lane;
    const int e = p < pairs ? ids[p] : -1;
    uint64_t same = __ballot(e >= 0);
#pragma unroll
    for (int bit = 0; bit < 10; ++bit) {
      const uint64_t set = __ballot((e >> bit) & 1);
      same &= ((e >> bit) & 1) ? set : ~set;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    int slot = -1;
    if (e >= 0) {
      slot = base[e] + rank;
      A.row_ids[slot] = (int)((first + p) / A.top);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");      // every lane has read base[e]
    if (e >= 0 && rank == 0) base[e] += __popcll(same);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (p < pairs) A.slots[first + p] = slot;
  }
}

// From before[e] (pairs of e in earlier chunks) and total[e]: the offsets into
// before (added) and, for the first chunk, into A.offsets; row_ids past the end.
__device__ void finish(const RouteArgs &A, int chunk, int chunks, int pairs, const int32_t *ids, int32_t *before,
                       int32_t *total) {
  const int t = threadIdx.x;
  __shared__ int32_t wsum[kRouteThreads / 64];
  // exclusive prefix of total over the experts: thread t holds expert t
  const int mine = t < A.experts ? total[t] : 0;
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(inc, o, 64);
    if ((t & 63) >= o) inc += u;
  }
  if ((t & 63) == 63) wsum[t >> 6] = inc;
  __syncthreads();
  int add = 0, all = 0;
  for (int w = 0; w < kRouteThreads / 64; ++w) {
    if (w < (t >> 6)) add += wsum[w];
    all += wsum[w];
  }
  const int start = add + inc - mine;
  if (t < A.experts) {
    before[t] += start;
    if (chunk == 0) A.offsets[t] = start;
  }
  if (chunk == 0 && t == 0) A.offsets[A.experts] = all;
  // row_ids past the last pair, the chunk's share of them by its own range
  const int64_t lo = (int64_t)chunk * kChunkTokens * A.top;
  for (int64_t p = lo + t; p < lo + pairs; p += kRouteThreads)
    if (p >= all) A.row_ids[p] = -1;
  __syncthreads();
  if (t < 64) place(A, chunk, pairs, ids, before);
}

template <typename T, int kPer>
__global__ __launch_bounds__(kRouteThreads) void route_choose_kernel(RouteArgs A, int chunks) {
  __shared__ int32_t ids[kChunkTokens * kMaxTop];
  __shared__ int32_t count[kMaxExperts], before[kMaxExperts];
  const int chunk = blockIdx.x, t = threadIdx.x;
  for (int e = t; e < A.experts; e += kRouteThreads) count[e] = before[e] = 0;
  __syncthreads();
  const int t0 = chunk * kChunkTokens, n = min(kChunkTokens, A.tokens - t0);
  for (int i = t >> 6; i < n; i += kRouteThreads / 64) choose<T, kPer>(A, t0 + i, ids + i * A.top);
  __syncthreads();
  for (int p = t; p < n * A.top; p += kRouteThreads)
    if (ids[p] >= 0) atomicAdd(&count[ids[p]], 1);
  __syncthreads();
  if (chunks > 1) {
    for (int e = t; e < A.experts; e += kRouteThreads) A.hist[(int64_t)chunk * A.experts + e] = count[e];
    return;
  }
  finish(A, chunk, chunks, n * A.top, ids, before, count);
}

__global__ __launch_bounds__(kRouteThreads) void route_place_kernel(RouteArgs A, int chunks) {
  __shared__ int32_t ids[kChunkTokens * kMaxTop];
  __shared__ int32_t total[kMaxExperts], before[kMaxExperts];
  const int chunk = blockIdx.x, t = threadIdx.x;
  const int t0 = chunk * kChunkTokens, n = min(kChunkTokens, A.tokens - t0);
  for (int e = t; e < A.experts; e += kRouteThreads) total[e] = before[e] = 0;
  for (int p = t; p < n * A.top; p += kRouteThreads) ids[p] = A.ids[(int64_t)t0 * A.top + p];
  __syncthreads();
  // every thread adds one expert's counts over every `step`-th chunk
  const int step = kRouteThreads / A.experts;                  // >= 1
  if (t < step * A.experts) {
    const int e = t % A.experts;
    int all = 0, pre = 0;
    for (int c = t / A.experts; c < chunks; c += step) {
      const int h = A.hist[(int64_t)c * A.experts + e];
      all += h;
      pre += c < chunk ? h : 0;
    }
    atomicAdd(&total[e], all);
    atomicAdd(&before[e], pre);
  }
  __syncthreads();
  finish(A, chunk, chunks, n * A.top, ids, before, total);
}

template <typename T>
hipError_t route_t(const RouteArgs &A, hipStream_t s) {
  const int chunks = (A.tokens + kChunkTokens - 1) / kChunkTokens;
  if (A.experts <= 64) route_choose_kernel<T, 1><<<chunks, kRouteThreads, 0, s>>>(A, chunks);
  else if (A.experts <= 256) route_choose_kernel<T, 4><<<chunks, kRouteThreads, 0, s>>>(A, chunks);
  else route_choose_kernel<T, 16><<<chunks, kRouteThreads, 0, s>>>(A, chunks);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || chunks == 1) return e;
  route_place_kernel<<<chunks, kRouteThreads, 0, s>>>(A, chunks);
  return hipGetLastError();
}

// One workgroup of 256 a token and 2048 columns, 8 columns a thread.
template <typename T, bool kVec>
__global__ __launch_bounds__(256) void combine_kernel(const T *__restrict__ y, int64_t rows, int d,
                                                      const int32_t *__restrict__ slots,
                                                      const float *__restrict__ weights, int top,
                                                      T *__restrict__ out) {
  const int64_t token = blockIdx.x;
  const int c = ((int)blockIdx.y * 256 + (int)threadIdx.x) * 8;
  if (c >= d) return;
  float acc[8] = {};
  for (int j = 0; j < top; ++j) {
    const int slot = slots[token * top + j];
    if (slot < 0 || slot >= rows) continue;
    const float w = weights[token * top + j];
    const T *p = y + (int64_t)slot * d + c;
    float v[8];
    if (kVec) {
      load_vec<8>(p, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = c + i < d ? to_f32(p[i]) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, v[i], acc[i]);
  }
  T *o = out + token * d + c;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (kVec || c + i < d) o[i] = from_f32<T>(acc[i]);
}

template <typename T>
hipError_t combine_t(const T *y, int64_t rows, int d, const int32_t *slots, const float *weights, int tokens,
                     int top, T *out, hipStream_t s) {
  const dim3 grid(tokens, (d + 2047) / 2048);
  if (d % 8 == 0) combine_kernel<T, true><<<grid, 256, 0, s>>>(y, rows, d, slots, weights, top, out);
  else combine_kernel<T, false><<<grid, 256, 0, s>>>(y, rows, d, slots, weights, top, out);
  return hipGetLastError();
}

}  // namespace

bool moe_route_supported(int experts, int top) { return experts <= kMaxExperts && top <= kMaxTop; }

int64_t moe_route_scratch(int tokens, int experts) {
  const int64_t chunks = ((int64_t)tokens + kChunkTokens - 1) / kChunkTokens;
  return chunks > 1 ? chunks * experts * 4 : 0;
}

hipError_t launch_moe_route(const void *logits, int dtype, int tokens, int experts, int64_t stride, int top,
                            bool renorm, int32_t *ids, float *weights, int32_t *offsets, int32_t *row_ids,
                            int32_t *slots, void *scratch, hipStream_t s) {
  const RouteArgs A{logits, stride, tokens, experts, top, renorm ? 1 : 0, ids, weights, offsets, row_ids, slots,
                    (int32_t *)scratch};
  if (dtype == BQM_F32) return route_t<float>(A, s);
  if (dtype == BQM_BF16) return route_t<__bf16>(A, s);
  return route_t<_Float16>(A, s);
}

hipError_t launch_moe_combine(const void *y, int dtype, int64_t rows, int d, const int32_t *slots,
                              const float *weights, int tokens, int top, void *out, hipStream_t s) {
  if (dtype == BQM_F32) return combine_t((const float *)y, rows, d, slots, weights, tokens, top, (float *)out, s);
  if (dtype == BQM_BF16) return combine_t((const __bf16 *)y, rows, d, slots, weights, tokens, top, (__bf16 *)out, s);
  return combine_t((const _Float16 *)y, rows, d, slots, weights, tokens, top, (_Float16 *)out, s);
}

}  // namespace bqm
