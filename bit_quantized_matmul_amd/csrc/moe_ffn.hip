// The expert layer of a few tokens, from router logits to combined rows:
//
//   out[t] = sum_j W2[e_j] w[t, j] (silu(G[e_j] x_t) * (U[e_j] x_t)),   W13 = [G | U]
//
// The chosen experts' codes are read once and bound the time, so activations stay as they are: no
// quantizer, no sort, two launches.  One token to 8 of 64 experts of 2048 x 1024: 19.7 us, of which 8.6 are the codes
// (both launches at 5 TB/s, by clock stamps), 3 the choices (logits, the search, the list), and the rest two launches, the
// sums' way through LDS and the last workgroup's sum; 32 tokens: 95 us, 4.2 TB/s.  fp32, three products a code and two waves a
// SIMD: 31 and 141 us.  Rows of x that do not start on 16 bytes are loaded an element at a time, for every item anew: 2047 x 1023
// 24 and 161 us, in fp32 33 and 192.
//
// First launch: every workgroup makes all tokens' choices for itself (a fraction of a launch's time) and lists the
// experts that have tokens; then it takes 16 gate rows and the 16 up rows beside them of one expert at a time.
// Its waves take every NW-th block of 128 columns, straight into the matrix cores' registers, the next expert
// rows' codes on their way while the waves' sums meet in LDS.  silu(gate) * up times the token's weight goes out.
// Second launch: 16 rows of W2, the waves take (expert, block) pairs and add up all experts of all tokens in
// the same registers, so the combination is part of the sum.
//
// Operands.  Codes are exact in fp16 and bf16, so 16-bit rows of x enter as they are; an fp32 x is three bf16 terms,
// which hold its 24 bits.  Hidden rows are two bf16 terms (2^-17 against half a step of 2^-8 or, in fp16, 2^-11 of the result; a third
// would be half as much to read again), for an fp32 x three.
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
  float *part;                            // [row tiles, splits, 32 tokens, 16 rows], with splits > 1
  int *arrived;                           // [row tiles]
  int splits;
};

template <typename T> constexpr int kXTerms = sizeof(T) == 4 ? 3 : 1;
template <typename T> constexpr int kActTerms = sizeof(T) == 4 ? 3 : 2;
template <typename T> using Half8 = std::conditional_t<std::is_same_v<T, _Float16>, f16x8, bf16x8>;

// Codes go into bf16 products as 2^-17 of themselves, exactly: sums of 128 products of up to 448 times fp32's largest number stay in
// fp32 so, and a block's scale can bring them back.  What was summed is 2^17 times that (fp16 rows reach no such sums).
template <typename H> constexpr float kCode = std::is_same_v<H, f16x8> ? 1.0f : 0x1p-17f;

template <typename H>
__device__ __forceinline__ H widen_as(int lo, int hi) {
  H h;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (std::is_same_v<H, f16x8>) {
      const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(i ? hi : lo, kCode<H>, false);
      const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(i ? hi : lo, kCode<H>, true);
      h[4 * i] = a[0], h[4 * i + 1] = a[1], h[4 * i + 2] = b[0], h[4 * i + 3] = b[1];
    } else {
      const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(i ? hi : lo, kCode<H>, false);
      const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(i ? hi : lo, kCode<H>, true);
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
      // the first term is cut, so that it is finite where x is; what it leaves, 16 bits, are two more, exactly
      t[0][i] = __builtin_bit_cast(__bf16, (uint16_t)(__float_as_uint(v[i]) >> 16));
      float r = v[i] - __uint_as_float(__float_as_uint(v[i]) & 0xFFFF0000u);
#pragma unroll
      for (int z = 1; z < 3; ++z) {
        t[z][i] = (__bf16)r;
        r -= (float)t[z][i];
      }
    }
  }
}

// ------------------------------------------------------------------ choices

struct Choices {
  uint32_t tokens[kMaxExperts];           // by expert
  int16_t first[kMaxExperts];             // of its pairs
  int16_t ids[kMaxPairs];                 // [tokens, top]
  float weights[kMaxPairs];
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

// Hidden rows go out as half of themselves, so that the nearest bf16 of each is finite.
constexpr float kHidden = 0.5f;

// The experts that have tokens into `L` and the weights, times kHidden, in the pairs' order into `by_place` (LDS).
__device__ void list_experts(const MoeArgs &A, Choices &C, MoeList &L, float *by_place) {
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
    C.first[tid * kPer + i] = (int16_t)(at & 0xFFFFu);
    at += (1u << 16) + (uint32_t)__popc(mask[i]);
  }
  if (tid == 0) L.count = (int)(all >> 16);
  __syncthreads();
  // a pair's place: its expert's first, and the expert's tokens before it
  for (int i = tid; i < A.tokens * A.top; i += kThreads) {
    const int e = C.ids[i], tok = i / A.top;
    if (e >= 0) by_place[C.first[e] + __popc(C.tokens[e] & ((1u << tok) - 1u))] = kHidden * C.weights[i];
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
//
// kGroups groups of waves take an item each, so that short rows keep all waves busy.  The sums of an item meet in one
// of two buffers; its group's waves add them up and form the hidden rows in turn, while the others go on.
template <typename T, int kGroups>
__global__ __launch_bounds__(64 * kUpWaves, sizeof(T) == 2 ? 4 : 2) void moe_up_kernel(MoeArgs A, bool xvec, const T *__restrict__ x) {
  using H = Half8<T>;
  constexpr int NW = kUpWaves / kGroups, kTerms = kXTerms<T>, kDepth = 2;
  __shared__ union {
    Choices C;
    f32x4_t red[2][kGroups][NW][2][64];
  } lds;
  __shared__ MoeList L;
  __shared__ float by_place[kMaxPairs];
  list_experts(A, lds.C, L, by_place);
  if (blockIdx.x == 0) {
    const int *from = reinterpret_cast<const int *>(&L);
    for (int i = threadIdx.x; i < (int)(sizeof(MoeList) / 4); i += kUpWaves * 64) reinterpret_cast<int *>(A.list)[i] = from[i];
    for (int i = threadIdx.x; i < (A.hidden + kTile - 1) / kTile; i += kUpWaves * 64) A.arrived[i] = 0;
  }
  const int lane = threadIdx.x & 63, wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = wave_all / NW, wave = wave_all % NW, row = lane & 15, grp = lane >> 4;
  const int kb = (A.hidden + kBlk - 1) / kBlk, nb = (2 * A.ffn + kBlk - 1) / kBlk;
  const int fp = (A.ffn + kBlk - 1) / kBlk * kBlk, tiles = fp / kTile;
  const int64_t kp = (int64_t)kb * kBlk, plane = (int64_t)A.tokens * A.top * fp;
  const int items = L.count * tiles, stride = gridDim.x * kGroups;
  i32x4 wl[kDepth][2][2] = {};
  auto load_w = [&](int item, int b0) {
    const int a = item / tiles, n0 = (item - a * tiles) * kTile;
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
  int item = blockIdx.x * kGroups + group, turn = 0, c0 = 0;             // c0: the first of an item's tokens, 16 at a time
  if (item < items) load_w(item, wave);
  // every group of the workgroup makes as many turns as the longest: they meet once a turn
  const int lead = blockIdx.x * kGroups;
  int turns = items > lead ? (items - lead + stride - 1) / stride : 0;
  for (int g = 0; g < kGroups && A.tokens > 16; ++g) {                   // items of several turns
    int n = 0;
    for (int i = lead + g; i < items; i += stride) n += (__popc(L.tokens[i / tiles]) + 15) / 16;
    turns = max(turns, n);
  }
  for (; turn < turns; ++turn) {
    const bool live = item < items;
    const int a = live ? item / tiles : 0, n0 = (item - a * tiles) * kTile;
    const uint32_t mask = L.tokens[a];
    const int count = __popc(mask), p0 = L.first[a] + c0;
    const bool last = c0 + 16 >= count;
    const int next = last ? item + stride : item;
    if (live) {
      const int e = L.expert[a];
      // scales: the gate rows lie in one block; the up rows may cross into the next from row `cross` on
      const float *sg = A.s13 + ((int64_t)e * nb + min(n0, A.ffn - 1) / kBlk) * kb;
      const int u0 = A.ffn + min(n0, A.ffn - 1), ub = u0 / kBlk, cross = (ub + 1) * kBlk - u0;
      const float *su = A.s13 + ((int64_t)e * nb + ub) * kb, *su1 = ub + 1 < nb ? su + kb : su;
      const T *xr = x + nth_bit(mask, min(c0 + row, count - 1)) * A.xs;
      f32x4_t acc[2] = {};
      for (int b0 = wave; b0 < kb; b0 += NW * kDepth) {
        H xh[kDepth][4][kTerms];
        float s[kDepth][3];
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
          const int b = b0 + d * NW;
          if (b < kb) {
#pragma unroll
            for (int k = 0; k < 4; ++k) load_x8(xr, b * kBlk + (k / 2) * 64 + grp * 16 + (k & 1) * 8, A.hidden, xvec, xh[d][k]);
            s[d][0] = sg[b], s[d][1] = su[b], s[d][2] = su1[b];
          }
        }
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
          const int b = b0 + d * NW;
          if (b < kb) {
            f32x4_t part[2] = {};
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const H w = widen_as<H>(wl[d][h][k / 2][2 * (k & 1)], wl[d][h][k / 2][2 * (k & 1) + 1]);
#pragma unroll
                for (int z = 0; z < kTerms; ++z) part[h] = product(w, xh[d][k][z], part[h]);
              }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              acc[0][i] = fmaf(part[0][i], s[d][0], acc[0][i]);
              acc[1][i] = fmaf(part[1][i], grp * 4 + i < cross ? s[d][1] : s[d][2], acc[1][i]);
            }
          }
        }
        // the codes after these: of this item, or of the next turn
        if (b0 + NW * kDepth < kb) load_w(item, b0 + NW * kDepth);
        else if (next < items) load_w(next, wave);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) lds.red[turn & 1][group][wave][h][lane] = acc[h];
    }
    __syncthreads();
    if (live && wave == turn % NW && c0 + row < count) {
      f32x4_t s[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        s[h] = lds.red[turn & 1][group][0][h][lane];
#pragma unroll
        for (int v = 1; v < NW; ++v) s[h] += lds.red[turn & 1][group][v][h][lane];
        s[h] *= 1.0f / kCode<H>;
      }
      const float w = by_place[p0 + row];
      bf16x4 t[kActTerms<T>];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float r = n0 + grp * 4 + i < A.ffn ? silu_mul(s[0][i], s[1][i]) * w : 0.0f;      // zeros in the columns that pad
#pragma unroll
        for (int z = 0; z < kActTerms<T>; ++z) {
          t[z][i] = (__bf16)r;
          r -= (float)t[z][i];
        }
      }
#pragma unroll
      for (int z = 0; z < kActTerms<T>; ++z)
        *reinterpret_cast<bf16x4 *>(A.act + z * plane + (int64_t)(p0 + row) * fp + n0 + grp * 4) = t[z];
    }
    c0 = last ? 0 : c0 + 16;
    item = next;
  }
}

// ------------------------------------------------------------------ down and combination
//
// An item is kDepth blocks of an expert's 16 rows for 16 of its tokens; its products go to the tokens' sums in the
// wave's own part of LDS.  The hidden rows come through LDS as well, without passing through registers: an
// expert has few tokens, and a load of an operand, of which most lanes would hold no token, takes as long as a load
// of codes (32 tokens of 64 experts of 2048 x 1024: 43 us with operands loaded, 24 without them).
// Where there are fewer row tiles than CUs the items of one are shared out to several workgroups; the last to
// arrive adds up their sums, in their order.
typedef __attribute__((address_space(3))) void lds_void;

template <typename T>
__global__ __launch_bounds__(64 * kDownWaves, 2) void moe_down_kernel(MoeArgs A, T *__restrict__ out) {
  constexpr int NW = kDownWaves, kTerms = kActTerms<T>, kDepth = kTerms == 2 ? 2 : 1;
  constexpr int kChunks = 16 * kTerms, kActBytes = 16 * kChunks * 16;    // 16-byte chunks of a token's block; of 16 tokens
  __shared__ __align__(1024) uint8_t rows_lds[NW][kDepth][kActBytes];
  __shared__ f32x4_t sums[NW][kMoeFewTokens][4];                         // [wave][token][rows / 4]
  __shared__ uint32_t tokens[kMaxExperts];
  __shared__ uint32_t expert_first[kMaxExperts];                         // expert, and its first pair in the upper half
  __shared__ int before;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int row = lane & 15, grp = lane >> 4, n0 = blockIdx.x * kTile;
  const int most = min(A.experts, A.tokens * A.top), listed = A.list->count;
  for (int i = tid; i < most; i += NW * 64) {
    expert_first[i] = (uint32_t)A.list->expert[i] | (uint32_t)A.list->first[i] << 16;
    tokens[i] = A.list->tokens[i];
  }
#pragma unroll
  for (int i = 0; i < kMoeFewTokens * 4 / 64; ++i) (&sums[wave][0][0])[i * 64 + lane] = f32x4_t{};
  __syncthreads();
  const int fb = (A.ffn + kBlk - 1) / kBlk, nb = (A.hidden + kBlk - 1) / kBlk, each = (fb + kDepth - 1) / kDepth;
  const int64_t fp = (int64_t)fb * kBlk, plane = (int64_t)A.tokens * A.top * fp;
  const int items = listed * each, stride = NW * A.splits;
  const int64_t r0 = min(n0 + row, A.hidden - 1);

  i32x4 wl[kDepth][2] = {};
  float sl[kDepth] = {};
  auto load = [&](int item, int c0) {
    const int a = item / each, b0 = (item - a * each) * kDepth;
    const uint32_t ef = __builtin_amdgcn_readfirstlane((int)expert_first[a]), e = ef & 0xFFFFu;
    const int count = min((int)__popc(__builtin_amdgcn_readfirstlane((int)tokens[a])) - c0, 16);
    const uint8_t *p = A.w2 + ((int64_t)e * A.hidden + r0) * fp + grp * 16;
    const __bf16 *q = A.act + (int64_t)((ef >> 16) + c0) * fp;
    const float *s = A.s2 + ((int64_t)e * nb + n0 / kBlk) * fb;
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int b = min(b0 + d, fb - 1);
      wl[d][0] = *reinterpret_cast<const i32x4 *>(p + b * kBlk);
      wl[d][1] = *reinterpret_cast<const i32x4 *>(p + b * kBlk + 64);
      sl[d] = s[b];
      // chunk c of token t lies at c ^ t: 16 tokens' chunks c in 16 groups of four banks
#pragma unroll
      for (int i = 0; i < kActBytes / 1024; ++i) {
        if (i * 64 < count * kChunks) {
          const int slot = i * 64 + lane, t = slot / kChunks, c = (slot - t * kChunks) ^ t;
          const __bf16 *from = q + min(t, count - 1) * fp + (c / 16) * plane + b * kBlk + (c % 16) * 8;
          __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from,
                                           (lds_void *)(&rows_lds[wave][d][0] + i * 1024), 16, 0, 0);
        }
      }
    }
  };
  int item = blockIdx.y * NW + wave, c0 = 0;
  if (item < items) load(item, 0);
  while (item < items) {
    const uint32_t mask = tokens[item / each];
    const int count = __popc(mask), at = min(c0 + row, count - 1), tok = nth_bit(mask, at), b0 = item % each * kDepth;
    const bool mine = c0 + row < count, last = c0 + 16 >= count;
    const int next = last ? item + stride : item, next_c = last ? 0 : c0 + 16;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");                     // this item's rows and codes have landed
    bf16x8 al[kDepth][4][kTerms], wh[kDepth][4];
    float s[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      s[d] = sl[d];
      const uint8_t *from = &rows_lds[wave][d][0] + (at - c0) * (kChunks * 16);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = ((k / 2) * 8 + grp * 2 + (k & 1)) ^ (at - c0);
#pragma unroll
        for (int z = 0; z < kTerms; ++z) al[d][k][z] = *reinterpret_cast<const bf16x8 *>(from + z * 256 + c * 16);
        wh[d][k] = widen_as<bf16x8>(wl[d][k / 2][2 * (k & 1)], wl[d][k / 2][2 * (k & 1) + 1]);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");                   // and are read: their place is free
    if (next < items) load(next, next_c);
    f32x4_t part[kDepth] = {};
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int z = 0; z < kTerms; ++z) part[d] = product(wh[d][k], al[d][k][z], part[d]);
    if (mine) {
      f32x4_t sum = sums[wave][tok][grp];
#pragma unroll
      for (int d = 0; d < kDepth; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = b0 + d < fb ? fmaf(part[d][i], s[d], sum[i]) : sum[i];   // no block past the last
      sums[wave][tok][grp] = sum;
    }
    item = next;
    c0 = next_c;
  }
  __syncthreads();
  // a thread a token and row
  static_assert(NW * 64 == kMoeFewTokens * kTile, "a thread a result");
  const int t = tid / kTile, r = tid % kTile;
  float sum = 0.0f;
#pragma unroll
  for (int v = 0; v < NW; ++v) sum += reinterpret_cast<const float *>(&sums[v][t][0])[r];
  if (A.splits > 1) {
    float *mine = A.part + (int64_t)blockIdx.x * A.splits * (NW * 64) + tid;
    // Each sum is stored and loaded as an atomic of the device's scope: such a store goes through the XCD's own L2 to where all
    // XCDs' loads of that scope look, and vmcnt falls when it is there.  So the wait, the barrier and the count after them
    // are what orders a workgroup's sums before the last one's loads.  That is this chip's order: the language promises it only between release
    // and acquire, which here write back and empty the whole L2 (40 us).
    __hip_atomic_store(mine + blockIdx.y * NW * 64, sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid == 0) before = __hip_atomic_fetch_add(A.arrived + blockIdx.x, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (before != A.splits - 1) return;
    sum = 0.0f;
    for (int z = 0; z < A.splits; ++z) sum += __hip_atomic_load(mine + z * NW * 64, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (t < A.tokens && n0 + r < A.hidden) out[(int64_t)t * A.hidden + n0 + r] = from_sum<T>(sum * (1.0f / (kCode<bf16x8> * kHidden)));
}

int row_tiles(int hidden) { return (hidden + kTile - 1) / kTile; }

// Workgroups of a row tile: as many as it takes for one a CU, while each wave has an item (us a layer with 1 / 2 / 4: one
// token to 8 of 64 experts of 2048 x 1024 22.3 / 20.2 / 20.7, 32 tokens 139 / 105 / 105; 7 tokens to 3 of 12 of 312 x 1092
// 31 / 24 / 21, with 8 19).
int down_splits(int tokens, int experts, int top, int hidden, int ffn) {
  const int64_t most = tokens * top < experts ? tokens * top : experts;
  const int64_t items = most * (((ffn + kBlk - 1) / kBlk + 1) / 2);
  const int64_t want = (256 + row_tiles(hidden) - 1) / row_tiles(hidden), can = (items + kDownWaves - 1) / kDownWaves;
  return (int)(want < can ? want : can);
}

template <typename T>
hipError_t run(const MoeArgs &A, const void *x, void *out, hipStream_t s) {
  const bool vec = ((uintptr_t)x & 15u) == 0 && A.xs % (16 / (int)sizeof(T)) == 0;
  const int pairs = A.tokens * A.top, tiles = (A.ffn + kBlk - 1) / kBlk * (kBlk / kTile), kb = (A.hidden + kBlk - 1) / kBlk;
  const int64_t items = (int64_t)(pairs < A.experts ? pairs : A.experts) * tiles;
  const int groups = kb >= 8 ? 1 : kb >= 4 ? 2 : 4;
  const int64_t need = (items + groups - 1) / groups;
  const unsigned grid = (unsigned)(need < 512 ? need : 512);
  if (groups == 1) moe_up_kernel<T, 1><<<grid, 64 * kUpWaves, 0, s>>>(A, vec, (const T *)x);
  else if (groups == 2) moe_up_kernel<T, 2><<<grid, 64 * kUpWaves, 0, s>>>(A, vec, (const T *)x);
  else moe_up_kernel<T, 4><<<grid, 64 * kUpWaves, 0, s>>>(A, vec, (const T *)x);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  moe_down_kernel<T><<<dim3(row_tiles(A.hidden), A.splits), 64 * kDownWaves, 0, s>>>(A, (T *)out);
  return hipGetLastError();
}

int64_t align16(int64_t n) { return (n + 15) / 16 * 16; }

}  // namespace

// The list, the row tiles' counts, the workgroups' sums, the hidden rows (three terms: the workspace is asked
// for without the type).
int64_t moe_ffn_scratch(int tokens, int experts, int top, int hidden, int ffn) {
  const int64_t parts = (int64_t)row_tiles(hidden) * down_splits(tokens, experts, top, hidden, ffn) * kMoeFewTokens * kTile * 4;
  return align16(sizeof(MoeList)) + align16(row_tiles(hidden) * 4) + parts +
         (int64_t)tokens * top * ((ffn + kBlk - 1) / kBlk * kBlk) * 6;
}

hipError_t launch_moe_ffn(const void *x, int dtype, int tokens, int hidden, int64_t xs, const void *logits, int ltype,
                          int64_t ls, int experts, int top, bool renorm, const uint8_t *w13, const float *s13,
                          const uint8_t *w2, const float *s2, int ffn, void *out, void *scratch, hipStream_t s) {
  const int splits = down_splits(tokens, experts, top, hidden, ffn);
  char *at = (char *)scratch;
  MoeList *list = (MoeList *)at;
  int *arrived = (int *)(at += align16(sizeof(MoeList)));
  float *part = (float *)(at += align16(row_tiles(hidden) * 4));
  __bf16 *act = (__bf16 *)(at + (int64_t)row_tiles(hidden) * splits * kMoeFewTokens * kTile * 4);
  const MoeArgs A{logits, ltype, xs, ls, tokens, experts, top, renorm, hidden, ffn, w13, w2, s13, s2, list, act, part, arrived, splits};
  if (dtype == BQM_F32) return run<float>(A, x, out, s);
  if (dtype == BQM_BF16) return run<__bf16>(A, x, out, s);
  return run<_Float16>(A, x, out, s);
}

}  // namespace bqm
