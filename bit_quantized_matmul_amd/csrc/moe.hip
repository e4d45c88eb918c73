// Mixture-of-experts routing and the combination of the experts' rows.
//
// Route.  Per token the k largest logits, their softmax weights, and the
// (token, expert) pairs in a stable order by expert.  Logits are compared as
// they are (never after an exp, which could make unequal ones equal); equal
// ones go to the lower expert; NaN counts as -inf, which is never chosen, and
// +inf as the largest fp32 value, so that exp(l - max) stays defined.
//
// The order is a counting sort over chunks of neighbouring tokens: the first kernel
// chooses and counts each chunk's experts, the second adds up the counts of the chunks
// before its own and places the chunk's pairs.  The counts are sums of integers, so
// nothing depends on the order of atomics.  One chunk needs no second launch.
//
// Combine.  out[t] = sum_j weights[t, j] * y[slots[t, j]] in fp32, j ascending.
#include "moe_choose.h"

namespace bqm {
namespace {

constexpr int kChunkTokens = 64;      // of a chunk, while there are at most kMaxChunks of them
constexpr int kMaxChunks = 512;       // every chunk reads all chunks' counts
constexpr int kRouteThreads = 1024;

struct RouteArgs {
  const void *logits;
  int64_t stride;
  int tokens, experts, top, renorm;
  int32_t *ids;
  float *weights;
  int32_t *offsets, *row_ids, *slots;
  uint16_t *hist;            // [chunks, experts rounded up to even]
  int chunk_tokens, chunks;
};

// counts (LDS): the chunk's, by expert.
template <typename T, int LANES, int kPer>
__device__ void choose(const RouteArgs &A, int token, int32_t *ids_lds, int32_t *counts) {
  choose_experts<T, LANES, kPer>(reinterpret_cast<const T *>(A.logits) + (int64_t)token * A.stride, A.experts, A.top,
                                 A.renorm, [&](int j, int id, float w) {
    const int64_t o = (int64_t)token * A.top + j;
    A.ids[o] = id;
    A.weights[o] = w;
    ids_lds[j] = id;
    if (id >= 0) atomicAdd(&counts[id], 1);
  });
}

// From before[e] (pairs of e in earlier chunks) and total[e]: the offsets (into A.offsets
// by the first chunk), row_ids past the end, and the chunk's pairs in their places, 1024 at
// a time: a pair's rank is the number of its expert's pairs before it in its wave (from
// ballots over the expert's bits) and in the waves before (their counts in a byte each,
// an expert's 16 side by side).
template <typename Ids>
__device__ void finish(const RouteArgs &A, int chunk, int pairs, Ids ids, int32_t *before, const int32_t *total) {
  constexpr int kWaves = kRouteThreads / 64;
  static_assert(kWaves == 16, "16 counts an expert");
  __shared__ int32_t wsum[kWaves];
  __shared__ u32x4_t counts[kMaxExperts];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  int e = t < pairs ? ids[t] : -1;                             // on its way during the scan
  if (t < A.experts) counts[t] = u32x4_t{0, 0, 0, 0};
  // exclusive prefix of total over the experts: thread t holds expert t
  const int mine = t < A.experts ? total[t] : 0;
  const int inc = wave_prefix(mine);
  if (lane == 63) wsum[wave] = inc;
  __syncthreads();
  int add = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) add += wsum[w];
    all += wsum[w];
  }
  const int start = add + inc - mine;
  if (t < A.experts) {
    before[t] += start;
    if (chunk == 0) A.offsets[t] = start;
  }
  if (chunk == 0 && t == 0) A.offsets[A.experts] = all;
  const int64_t first = (int64_t)chunk * A.chunk_tokens * A.top;
  for (int p0 = 0; p0 < pairs; p0 += kRouteThreads) {
    const int p = p0 + t;
    if (p0 > 0) {                                              // the round before counts as earlier pairs
      __syncthreads();
      if (t < A.experts) {
        const u32x4_t c = counts[t];
        uint32_t n = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) n = __builtin_amdgcn_udot4(c[i], 0x01010101u, n, false);
        before[t] += (int)n;
        counts[t] = u32x4_t{0, 0, 0, 0};
      }
      e = p < pairs ? ids[p] : -1;
      __syncthreads();
    }
    uint64_t same = __ballot(e >= 0);
#pragma unroll
    for (int bit = 0; bit < 10; ++bit) {
      const uint64_t set = __ballot((e >> bit) & 1);
      same &= ((e >> bit) & 1) ? set : ~set;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    if (e >= 0 && rank == 0) reinterpret_cast<uint8_t *>(&counts[e])[wave] = (uint8_t)__popcll(same);
    __syncthreads();
    int slot = -1;
    if (e >= 0) {
      const u32x4_t c = counts[e];
      uint32_t n = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {                            // the bytes of the waves before
        const int k = wave - 4 * i;
        const uint32_t mask = k <= 0 ? 0u : k >= 4 ? ~0u : (1u << (8 * k)) - 1u;
        n = __builtin_amdgcn_udot4(c[i] & mask, 0x01010101u, n, false);
      }
      slot = before[e] + (int)n + rank;
      A.row_ids[slot] = chunk * A.chunk_tokens + p / A.top;
    }
    if (p < pairs) {
      A.slots[first + p] = slot;
      if (first + p >= all) A.row_ids[first + p] = -1;
    }
  }
}

template <typename T, int LANES, int kPer>
__global__ __launch_bounds__(kRouteThreads) void route_choose_kernel(RouteArgs A) {
  __shared__ int32_t ids[kChunkTokens * kMaxTop];              // read back where this is the only chunk
  __shared__ int32_t count[kMaxExperts], before[kMaxExperts];
  const int chunk = blockIdx.x, t = threadIdx.x;
  for (int e = t; e < A.experts; e += kRouteThreads) count[e] = before[e] = 0;
  __syncthreads();
  const int t0 = chunk * A.chunk_tokens, n = min(A.chunk_tokens, A.tokens - t0);
  for (int i = t / LANES; i < n; i += kRouteThreads / LANES)
    choose<T, LANES, kPer>(A, t0 + i, ids + (i & (kChunkTokens - 1)) * A.top, count);
  __syncthreads();
  if (A.chunks > 1) {
    const int ep = (A.experts + 1) & ~1;
    for (int e = t; e < ep; e += kRouteThreads) A.hist[(int64_t)chunk * ep + e] = e < A.experts ? count[e] : 0;
    return;
  }
  finish(A, chunk, n * A.top, ids, before, count);
}

__global__ __launch_bounds__(kRouteThreads) void route_place_kernel(RouteArgs A) {
  __shared__ int32_t total[kMaxExperts], before[kMaxExperts];
  const int chunk = blockIdx.x, t = threadIdx.x;
  const int t0 = chunk * A.chunk_tokens, n = min(A.chunk_tokens, A.tokens - t0);
  for (int e = t; e < A.experts; e += kRouteThreads) total[e] = before[e] = 0;
  __syncthreads();
  // every thread adds two experts' counts over every `step`-th chunk, eight loads at a time
  const int half = (A.experts + 1) >> 1, step = kRouteThreads / half;
  const uint32_t *hist = reinterpret_cast<const uint32_t *>(A.hist);
  if (t < step * half) {
    const int e = 2 * (t % half);
    int all[2] = {0, 0}, pre[2] = {0, 0};
    for (int c0 = t / half; c0 < A.chunks; c0 += 8 * step) {
      uint32_t h[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int c = c0 + u * step;
        h[u] = c < A.chunks ? hist[(int64_t)c * half + (e >> 1)] : 0u;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const uint32_t p = c0 + u * step < chunk ? h[u] : 0u;
        all[0] += h[u] & 0xFFFFu;
        all[1] += h[u] >> 16;
        pre[0] += p & 0xFFFFu;
        pre[1] += p >> 16;
      }
    }
    atomicAdd(&total[e], all[0]);
    atomicAdd(&before[e], pre[0]);
    if (e + 1 < A.experts) {
      atomicAdd(&total[e + 1], all[1]);
      atomicAdd(&before[e + 1], pre[1]);
    }
  }
  __syncthreads();
  finish(A, chunk, n * A.top, A.ids + (int64_t)t0 * A.top, before, total);
}

// Tokens of a chunk: at most kMaxChunks chunks, until a chunk has 32768 tokens (counts are 16
// bits) and their number grows (past 2^24 tokens, 2^23 of many experts).  Past 256 experts
// a wave chooses for one token at a time, a chunk is one token a wave, and half as many
// chunks read all counts, which are longer (us, 4096 tokens of 512, 10 each: 38 with 64 tokens a
// chunk, 22 with 16).
int chunk_tokens(int tokens, int experts) {
  const bool wide = experts > 256;
  int c = wide ? kRouteThreads / 64 : kChunkTokens;
  while ((int64_t)c * (wide ? kMaxChunks / 2 : kMaxChunks) < tokens && c < 32768) c *= 2;
  return c;
}

template <typename T>
hipError_t route_t(RouteArgs A, hipStream_t s) {
  if (A.experts <= 64) route_choose_kernel<T, 16, 4><<<A.chunks, kRouteThreads, 0, s>>>(A);
  else if (A.experts <= 128) route_choose_kernel<T, 16, 8><<<A.chunks, kRouteThreads, 0, s>>>(A);
  else if (A.experts <= 256) route_choose_kernel<T, 16, 16><<<A.chunks, kRouteThreads, 0, s>>>(A);
  else if (A.experts <= 512) route_choose_kernel<T, 64, 8><<<A.chunks, kRouteThreads, 0, s>>>(A);
  else route_choose_kernel<T, 64, 16><<<A.chunks, kRouteThreads, 0, s>>>(A);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || A.chunks == 1) return e;
  route_place_kernel<<<A.chunks, kRouteThreads, 0, s>>>(A);
  return hipGetLastError();
}

// One workgroup of 256 a token and 2048 columns, 8 columns a thread: with 16-byte loads where
// rows are whole groups of 8, else by elements (us, 8192 tokens of 8, bf16: 4096 columns 121,
// 4100 306).
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

// More tokens than a launch takes: half of that a launch.
template <typename T>
hipError_t combine_t(const T *y, int64_t rows, int d, const int32_t *slots, const float *weights, int tokens,
                     int top, T *out, hipStream_t s) {
  constexpr int64_t kTokens = kMaxGroups256 / 2;
  for (int64_t t = 0; t < tokens; t += kTokens) {
    const dim3 grid((unsigned)(tokens - t < kTokens ? tokens - t : kTokens), (d + 2047) / 2048);
    const int32_t *sl = slots + t * top;
    const float *w = weights + t * top;
    T *o = out + t * d;
    if (d % 8 == 0) combine_kernel<T, true><<<grid, 256, 0, s>>>(y, rows, d, sl, w, top, o);
    else combine_kernel<T, false><<<grid, 256, 0, s>>>(y, rows, d, sl, w, top, o);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

bool moe_route_supported(int experts, int top) { return experts <= kMaxExperts && top <= kMaxTop; }

int64_t moe_route_scratch(int tokens, int experts) {
  const int64_t c = chunk_tokens(tokens, experts), chunks = (tokens + c - 1) / c;
  return chunks > 1 ? chunks * ((experts + 1) & ~1) * 2 : 0;
}

hipError_t launch_moe_route(const void *logits, int dtype, int tokens, int experts, int64_t stride, int top,
                            bool renorm, int32_t *ids, float *weights, int32_t *offsets, int32_t *row_ids,
                            int32_t *slots, void *scratch, hipStream_t s) {
  const int c = chunk_tokens(tokens, experts);
  const RouteArgs A{logits, stride, tokens, experts, top, renorm ? 1 : 0, ids, weights, offsets, row_ids, slots,
                    (uint16_t *)scratch, c, (int)(((int64_t)tokens + c - 1) / c)};
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
