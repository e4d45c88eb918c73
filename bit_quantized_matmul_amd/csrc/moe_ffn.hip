// The expert layer of a few tokens, from router logits to combined rows:
//
//   out[t] = sum_j W2[e_j] w[t, j] (silu(G[e_j] x_t) * (U[e_j] x_t)),   W13 = [G | U]
//
// The chosen experts' codes are read once and bound the time, so activations stay as they are: no
// quantizer, no sort, two launches.
//
// First launch: every workgroup makes all tokens' choices for itself (a fraction of a launch's time) and lists the
// experts that have tokens; then it takes 16 gate rows and the 16 up rows beside them of one expert at a time.
// Its waves take every NW-th block of 128 columns, straight into the matrix cores' registers, the next expert
// rows' codes on their way while the waves' sums meet in LDS.  silu(gate) * up times the token's weight goes out.
// Second launch: 16 rows of W2, the waves take (expert, block) pairs and add up all experts of all tokens in
// the same registers, so the combination is part of the sum.
//
// Operands.  Codes are exact in fp16 and bf16, so 16-bit rows of x enter as they are; an fp32 x is three bf16 terms,
// which hold its 24 bits.  Hidden rows are two bf16 terms (2^-17), for an fp32 x three.
#include "moe_choose.h"

#include <type_traits>

namespace bqm {
namespace {

constexpr int kBlk = 128, kTile = 16;
constexpr int kUpWaves = 8, kDownWaves = 8;
constexpr int kMaxPairs = kMoeFewTokens * kMaxTop;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// What the first launch leaves for the second; experts that have tokens, ascending, and their pairs in order.
struct MoeList {
  int count;
  int expert[kMaxExperts];
  uint32_t tokens[kMaxExperts];           // bit t: token t
  int first[kMaxExperts];                 // of the expert's pairs, tokens ascending
};

struct MoeArgs {
  const void *logits;
  int ltype;                              // the logits' type
  int64_t xs, ls;                         // strides of x's and logits' rows
  int tokens, experts, top, renorm, hidden, ffn;
  const uint8_t *w13, *w2;
  const float *s13, *s2;
  MoeList *list;                          // workspace
  __bf16 *act;                            // [terms, tokens * top, 128 ceil(ffn / 128)]
};

template <typename T> constexpr int kXTerms = sizeof(T) == 4 ? 3 : 1;
template <typename T> constexpr int kActTerms = sizeof(T) == 4 ? 3 : 2;
template <typename T> using Half8 = std::conditional_t<std::is_same_v<T, _Float16>, f16x8, bf16x8>;

template <typename H>
__device__ __forceinline__ H widen_as(int lo, int hi) {
  H h;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (std::is_same_v<H, f16x8>) {
      const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(i ? hi : lo, 1.0f, false);
      const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(i ? hi : lo, 1.0f, true);
      h[4 * i] = a[0], h[4 * i + 1] = a[1], h[4 * i + 2] = b[0], h[4 * i + 3] = b[1];
    } else {
      const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(i ? hi : lo, 1.0f, false);
      const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(i ? hi : lo, 1.0f, true);
      h[4 * i] = a[0], h[4 * i + 1] = a[1], h[4 * i + 2] = b[0], h[4 * i + 3] = b[1];
    }
  }
  return h;
}

__device__ __forceinline__ f32x4_t product(f16x8 a, f16x8 b, f32x4_t c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ f32x4_t product(bf16x8 a, bf16x8 b, f32x4_t c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }

// 8 columns of a row of x from c on as operand terms, zeros past `cols`.
template <typename T>
__device__ __forceinline__ void load_x8(const T *p, int c, int cols, bool vec, Half8<T> (&t)[kXTerms<T>]) {
  T v[8];
  if (vec && c + 8 <= cols) {
    typedef T tx8 __attribute__((ext_vector_type(8)));
    const tx8 a = *reinterpret_cast<const tx8 *>(p + c);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = a[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const T a = p[min(c + i, cols - 1)];
      v[i] = c + i < cols ? a : (T)0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(T) == 2) {
      t[0][i] = v[i];
    } else {
      float r = v[i];
#pragma unroll
      for (int z = 0; z < 3; ++z) {
        t[z][i] = (__bf16)r;
        r -= (float)t[z][i];
      }
    }
  }
}

// ------------------------------------------------------------------ choices

struct Choices {
  uint32_t tokens[kMaxExperts];           // by expert
  int16_t ids[kMaxPairs];                 // [tokens, top]
  float weights[kMaxPairs];
  float by_place[kMaxPairs];              // in the pairs' order
  uint32_t sums[kUpWaves];
};

template <typename T>
__device__ __forceinline__ void choose_all(const MoeArgs &A, Choices &C) {
  const T *logits = reinterpret_cast<const T *>(A.logits);
  const int wave = threadIdx.x >> 6;
  const auto put = [&](int t) {
    return [&C, &A, t](int j, int id, float w) {
      C.ids[t * A.top + j] = (int16_t)id;
      C.weights[t * A.top + j] = w;
      if (id >= 0) atomicOr(&C.tokens[id], 1u << t);
    };
  };
  // 16 lanes a token up to 256 experts, as in routing
  if (A.experts <= 256) {
    const int t = threadIdx.x >> 4;
    if (t >= A.tokens) return;            // tokens <= 32 = 512 / 16
    const T *row = logits + t * A.ls;
    if (A.experts <= 64) choose_experts<T, 16, 4>(row, A.experts, A.top, A.renorm, put(t));
    else if (A.experts <= 128) choose_experts<T, 16, 8>(row, A.experts, A.top, A.renorm, put(t));
    else choose_experts<T, 16, 16>(row, A.experts, A.top, A.renorm, put(t));
  } else {
    for (int t = wave; t < A.tokens; t += kUpWaves)
      choose_experts<T, 64, 16>(logits + t * A.ls, A.experts, A.top, A.renorm, put(t));
  }
}
static_assert(kUpWaves * 64 / 16 >= kMoeFewTokens, "16 lanes a token");

// The experts that have tokens into `L` (LDS), the weights in the pairs' order.
__device__ void list_experts(const MoeArgs &A, Choices &C, MoeList &L) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int kThreads = kUpWaves * 64, kPer = kMaxExperts / kThreads;
  for (int e = tid; e < A.experts; e += kThreads) C.tokens[e] = 0;
  __syncthreads();
  if (A.ltype == BQM_F32) choose_all<float>(A, C);
  else if (A.ltype == BQM_BF16) choose_all<__bf16>(A, C);
  else choose_all<_Float16>(A, C);
  __syncthreads();
  // thread t holds experts kPer t ..: experts with tokens in the upper half, pairs in the lower
  uint32_t mask[kPer];
  int mine = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    mask[i] = e < A.experts ? C.tokens[e] : 0;
    mine += (mask[i] ? 1 << 16 : 0) + __popc(mask[i]);
  }
  const int inc = wave_prefix(mine);
  if (lane == 63) C.sums[wave] = (uint32_t)inc;
  __syncthreads();
  uint32_t at = (uint32_t)(inc - mine), all = 0;
#pragma unroll
  for (int w = 0; w < kUpWaves; ++w) {
    if (w < wave) at += C.sums[w];
    all += C.sums[w];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (!mask[i]) continue;
    L.expert[at >> 16] = tid * kPer + i;
    L.tokens[at >> 16] = mask[i];
    L.first[at >> 16] = (int)(at & 0xFFFFu);
    at += (1u << 16) + (uint32_t)__popc(mask[i]);
  }
  if (tid == 0) L.count = (int)(all >> 16);
  __syncthreads();
  // a pair's place: its expert's first, and the expert's tokens before it
  for (int a = wave; a < L.count; a += kUpWaves) {
    const int e = L.expert[a], t = lane & 31;
    const uint32_t m = L.tokens[a];
    if (lane < 32 && (m >> t & 1)) {
      float w = 0.0f;
      for (int j = 0; j < A.top; ++j)
        if (C.ids[t * A.top + j] == e) w = C.weights[t * A.top + j];
      C.by_place[L.first[a] + __popc(m & ((1u << t) - 1u))] = w;
    }
  }
  __syncthreads();
}

// Bit number n (from 0) of m that is set, for n < popc(m).
__device__ __forceinline__ int nth_bit(uint32_t m, int n) {
  int at = 0;
#pragma unroll
  for (int w = 16; w >= 1; w /= 2) {
    const int below = __popc(m >> at & ((1u << w) - 1u));
    if (n >= below) n -= below, at += w;
  }
  return at;
}

// silu(g) u; NaN where either has left fp32, so that a row of x that is not finite stays so
__device__ __forceinline__ float silu_mul(float g, float u) {
  if (!(fabsf(g) < INFINITY && fabsf(u) < INFINITY)) return __builtin_nanf("");
  // below -80 exp(-g) may overflow: g exp(g) u = (g h u) h with h = exp(g / 2)
  if (g < -80.0f) {
    const float h = expf(0.5f * g);
    return g * h * u * h;
  }
  return g / (1.0f + expf(-g)) * u;
}

// ------------------------------------------------------------------ gate and up

template <typename T>
__global__ __launch_bounds__(64 * kUpWaves, 2) void moe_up_kernel(MoeArgs A, bool xvec, const T *__restrict__ x) {
  using H = Half8<T>;
  constexpr int NW = kUpWaves, kTerms = kXTerms<T>, kDepth = 2;
  __shared__ Choices C;
  __shared__ MoeList L;
  __shared__ f32x4_t red[NW][2][64];
  list_experts(A, C, L);
  if (blockIdx.x == 0) {
    const int *from = reinterpret_cast<const int *>(&L);
    for (int i = threadIdx.x; i < (int)(sizeof(MoeList) / 4); i += NW * 64) reinterpret_cast<int *>(A.list)[i] = from[i];
  }
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, grp = lane >> 4;
  const int kb = (A.hidden + kBlk - 1) / kBlk, nb = (2 * A.ffn + kBlk - 1) / kBlk;
  const int fp = (A.ffn + kBlk - 1) / kBlk * kBlk, tiles = fp / kTile;
  const int64_t kp = (int64_t)kb * kBlk;
  const int items = L.count * tiles;
  i32x4 wl[kDepth][2][2] = {};
  auto load_w = [&](int item, int b0) {
    const int a = item / tiles, n0 = (item - a * tiles) * kTile;
    if (n0 >= A.ffn) return;
    const uint8_t *g = A.w13 + ((int64_t)L.expert[a] * 2 * A.ffn + min(n0 + row, A.ffn - 1)) * kp + grp * 16;
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int b = b0 + d * NW;
      if (b < kb) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t *p = g + h * A.ffn * kp + (int64_t)b * kBlk;
          wl[d][h][0] = *reinterpret_cast<const i32x4 *>(p);
          wl[d][h][1] = *reinterpret_cast<const i32x4 *>(p + 64);
        }
      }
    }
  };
  int item = blockIdx.x;
  if (item < items) load_w(item, wave);
  for (; item < items; item += gridDim.x) {
    const int a = item / tiles, n0 = (item - a * tiles) * kTile, e = L.expert[a];
    const uint32_t mask = L.tokens[a];
    const int count = __popc(mask), p0 = L.first[a], next = item + gridDim.x;
    const int64_t plane = (int64_t)A.tokens * A.top * fp;
    if (n0 >= A.ffn) {                                                   // columns that pad the hidden rows: zeros
      for (int i = threadIdx.x; i < count * kTile * kActTerms<T>; i += NW * 64) {
        const int z = i / (count * kTile), j = i - z * count * kTile;
        A.act[z * plane + (int64_t)(p0 + j / kTile) * fp + n0 + j % kTile] = (__bf16)0.0f;
      }
      if (next < items) load_w(next, wave);
      continue;
    }
    // scales: the gate rows lie in one block; the up rows may cross into the next from row `cross` on
    const float *sg = A.s13 + ((int64_t)e * nb + n0 / kBlk) * kb;
    const int u0 = A.ffn + n0, ub = u0 / kBlk, cross = (ub + 1) * kBlk - u0;
    const float *su = A.s13 + ((int64_t)e * nb + ub) * kb, *su1 = ub + 1 < nb ? su + kb : su;
    for (int c0 = 0; c0 < count; c0 += 16) {                             // 16 tokens at a time
      const bool last = c0 + 16 >= count;
      const int tok = nth_bit(mask, min(c0 + row, count - 1));
      const T *xr = x + tok * A.xs;
      f32x4_t acc[2] = {};
      for (int b0 = wave; b0 < kb; b0 += NW * kDepth) {
        H wh[kDepth][2][4];
#pragma unroll
        for (int d = 0; d < kDepth; ++d)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k) wh[d][h][k] = widen_as<H>(wl[d][h][k / 2][2 * (k & 1)], wl[d][h][k / 2][2 * (k & 1) + 1]);
        // the codes after these: of this item, of its next tokens, of the next item
        if (b0 + NW * kDepth < kb) load_w(item, b0 + NW * kDepth);
        else if (!last) load_w(item, wave);
        else if (next < items) load_w(next, wave);
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
          const int b = b0 + d * NW;
          if (b < kb) {
            f32x4_t part[2] = {};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              H xh[kTerms];
              load_x8(xr, b * kBlk + (k / 2) * 64 + grp * 16 + (k & 1) * 8, A.hidden, xvec, xh);
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int z = 0; z < kTerms; ++z) part[h] = product(wh[d][h][k], xh[z], part[h]);
            }
            const float g = sg[b], u = su[b], u1 = su1[b];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              acc[0][i] = fmaf(part[0][i], g, acc[0][i]);
              acc[1][i] = fmaf(part[1][i], grp * 4 + i < cross ? u : u1, acc[1][i]);
            }
          }
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) red[wave][h][lane] = acc[h];
      __syncthreads();
      if (wave == 0 && c0 + row < count) {
        f32x4_t s[2] = {red[0][0][lane], red[0][1][lane]};
#pragma unroll
        for (int v = 1; v < NW; ++v)
#pragma unroll
          for (int h = 0; h < 2; ++h) s[h] += red[v][h][lane];
        const float w = C.by_place[p0 + c0 + row];
        bf16x4 t[kActTerms<T>];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float r = n0 + grp * 4 + i < A.ffn ? silu_mul(s[0][i], s[1][i]) * w : 0.0f;
#pragma unroll
          for (int z = 0; z < kActTerms<T>; ++z) {
            t[z][i] = (__bf16)r;
            r -= (float)t[z][i];
          }
        }
#pragma unroll
        for (int z = 0; z < kActTerms<T>; ++z)
          *reinterpret_cast<bf16x4 *>(A.act + z * plane + (int64_t)(p0 + c0 + row) * fp + n0 + grp * 4) = t[z];
      }
      __syncthreads();
    }
  }
}

// ------------------------------------------------------------------ down and combination

template <typename T, int MF>
__global__ __launch_bounds__(64 * kDownWaves, 2) void moe_down_kernel(MoeArgs A, T *__restrict__ out) {
  constexpr int NW = kDownWaves, kTerms = kActTerms<T>, kDepth = MF * kTerms <= 2 ? 4 : MF * kTerms <= 4 ? 2 : 1;
  __shared__ f32x4_t red[NW][MF][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, grp = lane >> 4, n0 = blockIdx.x * kTile;
  const int fb = (A.ffn + kBlk - 1) / kBlk, nb = (A.hidden + kBlk - 1) / kBlk;
  const int64_t fp = (int64_t)fb * kBlk, plane = A.tokens * A.top * fp;
  const MoeList &L = *A.list;
  const int items = L.count * fb;
  f32x4_t acc[MF] = {};
  const int64_t r0 = min(n0 + row, A.hidden - 1);
  i32x4 wl[kDepth][2];
  float sl[kDepth];
  auto load_w = [&](int i0) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int i = i0 + d * NW;
      if (i < items) {
        const int a = i / fb, b = i - a * fb, e = L.expert[a];
        const uint8_t *p = A.w2 + ((int64_t)e * A.hidden + r0) * fp + b * kBlk + grp * 16;
        wl[d][0] = *reinterpret_cast<const i32x4 *>(p);
        wl[d][1] = *reinterpret_cast<const i32x4 *>(p + 64);
        sl[d] = A.s2[((int64_t)e * nb + n0 / kBlk) * fb + b];
      }
    }
  };
  load_w(wave);
  for (int i0 = wave; i0 < items; i0 += NW * kDepth) {
    bf16x8 al[kDepth][MF][4][kTerms], wh[kDepth][4];
    float s[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int i = i0 + d * NW;
      if (i >= items) break;
      const int a = i / fb, b = i - a * fb;
      const uint32_t mask = L.tokens[a];
#pragma unroll
      for (int f = 0; f < MF; ++f) {
        const int t = f * 16 + row;
        const bool has = mask >> t & 1;
        const __bf16 *q = A.act + (L.first[a] + __popc(mask & ((1u << t) - 1u))) * fp + b * kBlk + grp * 16;
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int z = 0; z < kTerms; ++z) {
            al[d][f][k][z] = bf16x8{};
            if (has) al[d][f][k][z] = *reinterpret_cast<const bf16x8 *>(q + z * plane + (k / 2) * 64 + (k & 1) * 8);
          }
      }
    }
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      s[d] = sl[d];
#pragma unroll
      for (int k = 0; k < 4; ++k) wh[d][k] = widen_as<bf16x8>(wl[d][k / 2][2 * (k & 1)], wl[d][k / 2][2 * (k & 1) + 1]);
    }
    load_w(i0 + NW * kDepth);
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      if (i0 + d * NW >= items) break;
#pragma unroll
      for (int f = 0; f < MF; ++f) {
        f32x4_t part = {};
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int z = 0; z < kTerms; ++z) part = product(wh[d][k], al[d][f][k][z], part);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[f][i] = fmaf(part[i], s[d], acc[f][i]);
      }
    }
  }
#pragma unroll
  for (int f = 0; f < MF; ++f) red[wave][f][lane] = acc[f];
  __syncthreads();
  if (wave >= MF) return;
  f32x4_t sum = red[0][wave][lane];
#pragma unroll
  for (int v = 1; v < NW; ++v) sum += red[v][wave][lane];
  const int t = wave * 16 + row;
  if (t >= A.tokens) return;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n0 + grp * 4 + i < A.hidden) out[(int64_t)t * A.hidden + n0 + grp * 4 + i] = from_sum<T>(sum[i]);
}

template <typename T>
hipError_t run(const MoeArgs &A, const void *x, void *out, int num_cus, hipStream_t s) {
  const bool vec = ((uintptr_t)x & 15u) == 0 && A.xs % (16 / (int)sizeof(T)) == 0;
  const int pairs = A.tokens * A.top, tiles = (A.ffn + kBlk - 1) / kBlk * (kBlk / kTile);
  const int64_t items = (int64_t)(pairs < A.experts ? pairs : A.experts) * tiles;
  const unsigned grid = (unsigned)(items < 2 * num_cus ? items : 2 * num_cus);
  moe_up_kernel<T><<<grid, 64 * kUpWaves, 0, s>>>(A, vec, (const T *)x);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const unsigned rows = (unsigned)((A.hidden + kTile - 1) / kTile);
  if (A.tokens <= 16) moe_down_kernel<T, 1><<<rows, 64 * kDownWaves, 0, s>>>(A, (T *)out);
  else moe_down_kernel<T, 2><<<rows, 64 * kDownWaves, 0, s>>>(A, (T *)out);
  return hipGetLastError();
}

}  // namespace

int64_t moe_ffn_scratch(int tokens, int, int top, int, int ffn) {
  // three terms: the workspace is asked for without the type
  return (sizeof(MoeList) + 15) / 16 * 16 + (int64_t)tokens * top * ((ffn + kBlk - 1) / kBlk * kBlk) * 6;
}

hipError_t launch_moe_ffn(const void *x, int dtype, int tokens, int hidden, int64_t xs, const void *logits, int ltype,
                          int64_t ls, int experts, int top, bool renorm, const uint8_t *w13, const float *s13,
                          const uint8_t *w2, const float *s2, int ffn, void *out, void *scratch, int num_cus, hipStream_t s) {
  __bf16 *act = (__bf16 *)((char *)scratch + (sizeof(MoeList) + 15) / 16 * 16);
  const MoeArgs A{logits, ltype, xs, ls, tokens, experts, top, renorm, hidden, ffn, w13, w2, s13, s2, (MoeList *)scratch, act};
  if (dtype == BQM_F32) return run<float>(A, x, out, num_cus, s);
  if (dtype == BQM_BF16) return run<__bf16>(A, x, out, num_cus, s);
  return run<_Float16>(A, x, out, num_cus, s);
}

}  // namespace bqm
