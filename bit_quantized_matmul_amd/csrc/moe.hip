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
#include "lowp_types.h"

namespace bqm {
namespace {

constexpr int kChunkTokens = 64;      // of a chunk, while there are at most kMaxChunks of them
constexpr int kMaxChunks = 512;       // every chunk reads all chunks' counts
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
  uint16_t *hist;            // [chunks, experts rounded up to even]
  int chunk_tokens, chunks;
};

// Reductions over 16 consecutive lanes (DPP row rotations) or the wave (then swaps of rows).
template <int CTRL>
__device__ __forceinline__ int row_move(int v) {
  return __builtin_amdgcn_update_dpp(v, v, CTRL, 0xF, 0xF, false);
}

template <int LANES, typename F>
__device__ __forceinline__ int lanes_reduce(int v, F op) {
  v = op(v, row_move<0x121>(v));                               // row_ror 1, 2, 4, 8
  v = op(v, row_move<0x122>(v));
  v = op(v, row_move<0x124>(v));
  v = op(v, row_move<0x128>(v));
  if constexpr (LANES == 64) {
    auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);     // rows 0, 0, 2, 2 and 1, 1, 3, 3
    v = op((int)s[0], (int)s[1]);
    s = __builtin_amdgcn_permlane32_swap(v, v, false, false);          // the lower half twice, the upper twice
    v = op((int)s[0], (int)s[1]);
  }
  return v;
}

template <int LANES>
__device__ __forceinline__ float lanes_max(float v) {
  return __int_as_float(lanes_reduce<LANES>(__float_as_int(v), [](int a, int b) {
    return __float_as_int(fmaxf(__int_as_float(a), __int_as_float(b)));
  }));
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  return __int_as_float(lanes_reduce<LANES>(__float_as_int(v), [](int a, int b) {
    return __float_as_int(__int_as_float(a) + __int_as_float(b));
  }));
}

template <int LANES>
__device__ __forceinline__ int lanes_min(int v) {
  return lanes_reduce<LANES>(v, [](int a, int b) { return min(a, b); });
}

// Sorts N = 4, 8 or 16 keys, largest first: Batcher's odd-even merge sort.
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t (&k)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int h = p; h >= 1; h /= 2)
#pragma unroll
      for (int j = h % p; j + h < N; j += 2 * h)
#pragma unroll
        for (int i = 0; i < h; ++i)
          if (i + j + h < N && (i + j) / (2 * p) == (i + j + h) / (2 * p)) {
            const uint32_t x = k[i + j], y = k[i + j + h];
            k[i + j] = x > y ? x : y;
            k[i + j + h] = x > y ? y : x;
          }
}

// A lane's logits of one token, and the search for the largest of all lanes'.
// 32-bit logits: the largest of the lane's, then of the lanes', then the lowest index
// that has it.
template <typename T, int LANES, int kPer>
struct Logits {
  struct Pick {
    float w = -INFINITY;
    int at = -1;
  };
  float v[kPer];
  int lane;

  __device__ __forceinline__ void load(const T *x, int experts, int l) {
    lane = l;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane + LANES * i;
      const float a = e < experts ? to_f32(x[e]) : -INFINITY;
      v[i] = a != a ? -INFINITY : fminf(a, kHuge);
    }
  }
  __device__ __forceinline__ float value(int i) const { return v[i]; }
  static __device__ __forceinline__ float logit(Pick p) { return p.w; }
  static __device__ __forceinline__ int expert(Pick p) { return p.w > -INFINITY ? p.at : -1; }
  // the largest left, which leaves (-inf if there is none)
  __device__ __forceinline__ Pick next() {
    float b = -INFINITY;
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (v[i] > b) {
        b = v[i];
        at = lane + LANES * i;
      }
    const float w = lanes_max<LANES>(b);
    const int got = lanes_min<LANES>(b == w ? at : 0x7FFFFFFF);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (got == lane + LANES * i) v[i] = -INFINITY;
    return {w, got};
  }
};

// 16-bit logits: a key of the ordered bits over the inverted index, 0 for NaN and -inf, so
// that one integer maximum finds value and lowest index.  The lane sorts its keys once and
// offers its first (16384 tokens of 256: 14.0 us with the search above, 10.8 us so).
template <typename T, int LANES, int kPer>
struct Keys {
  using Pick = uint32_t;
  uint32_t k[kPer];

  __device__ __forceinline__ void load(const T *x, int experts, int lane) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane + LANES * i;
      uint32_t h = 0;
      if (e < experts) {
        const float f = to_f32(x[e]);
        uint32_t b = __builtin_bit_cast(uint16_t, x[e]);
        b = b == 0x8000u ? 0u : b;                             // -0 is 0
        h = f > -INFINITY ? ((b & 0x8000u) ? ~b & 0xFFFFu : b | 0x8000u) << 16 | (0xFFFFu - (uint32_t)e) : 0u;
      }
      k[i] = h;
    }
    sort_keys(k);
  }
  static __device__ __forceinline__ int expert(Pick key) { return key ? (int)(0xFFFFu - (key & 0xFFFFu)) : -1; }
  static __device__ __forceinline__ float logit(Pick key) {
    if (key == 0) return -INFINITY;
    const uint32_t u = key >> 16;
    const uint16_t b = (uint16_t)((u & 0x8000u) ? u & 0x7FFFu : ~u);
    return fminf(to_f32(__builtin_bit_cast(T, b)), kHuge);
  }
  __device__ __forceinline__ float value(int i) const { return logit(k[i]); }
  __device__ __forceinline__ Pick next() {
    const uint32_t w = (uint32_t)lanes_reduce<LANES>((int)k[0], [](int a, int b) {
      return (uint32_t)a > (uint32_t)b ? a : b;
    });
    const bool mine = k[0] == w;
#pragma unroll
    for (int i = 0; i + 1 < kPer; ++i) k[i] = mine ? k[i + 1] : k[i];
    k[kPer - 1] = mine ? 0u : k[kPer - 1];
    return w;
  }
};

template <int LANES, int kPer> struct Keys<float, LANES, kPer> : Logits<float, LANES, kPer> {};

// LANES lanes choose one token's experts; lane l of them holds experts l, l + LANES, ...
// counts (LDS): the chunk's, by expert.
template <typename T, int LANES, int kPer>
__device__ void choose(const RouteArgs &A, int token, int32_t *ids_lds, int32_t *counts) {
  const int lane = threadIdx.x & (LANES - 1);
  Keys<T, LANES, kPer> x;
  x.load(reinterpret_cast<const T *>(A.logits) + (int64_t)token * A.stride, A.experts, lane);
  float ref = 0.0f, total = 0.0f;                              // the largest logit; the sum of exp(l - ref)
  if (!A.renorm) {
    float best = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPer; ++i) best = fmaxf(best, x.value(i));
    best = lanes_max<LANES>(best);
    ref = best > -INFINITY ? best : 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) total += expf(x.value(i) - ref);
    total = lanes_sum<LANES>(total);
  }
  using K = Keys<T, LANES, kPer>;
  typename K::Pick first{}, mine[2] = {};                      // the largest; the choices lane and lane + LANES
  for (int j = 0; j < A.top; ++j) {
    const typename K::Pick p = x.next();
    if (j == 0) first = p;
    if (j == lane) mine[0] = p;
    if (j == lane + LANES) mine[1] = p;
  }
  const float most = K::logit(first);
  ref = most > -INFINITY ? most : 0.0f;
  float e[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) e[h] = K::expert(mine[h]) >= 0 ? expf(K::logit(mine[h]) - ref) : 0.0f;
  if (A.renorm) total = lanes_sum<LANES>(e[0] + e[1]);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = lane + h * LANES, id = K::expert(mine[h]);
    if (j < A.top) {
      const int64_t o = (int64_t)token * A.top + j;
      A.ids[o] = id;
      A.weights[o] = id >= 0 ? e[h] / total : 0.0f;
      ids_lds[j] = id;
      if (id >= 0) atomicAdd(&counts[id], 1);
    }
  }
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
