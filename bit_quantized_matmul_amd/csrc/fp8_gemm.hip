// Products of E4M3 activations and weights with a scale for each block of 128,
// dense and grouped by expert.
//
//   y[t, r] = sum_b sx[b, t] * sw[r / 128, b] * sum_{j < 128} q[t, 128 b + j] * w[r, 128 b + j]
//
// The codes become fp16 in registers (E4M3 is exact there, two codes an instruction), the fp16
// matrix instructions sum a block's products in fp32, the sums are scaled and added in fp32 and
// y is rounded once.  The 8-bit matrix instructions have twice the rate and need no conversions, but of
// each 8 products they keep only the 13 bits below the largest: 2e-5 to 4e-5 of the result's
// norm before it is rounded, and 2% of the elements of a bf16 result of 4096 x 14336 x 4096
// round the other way.  So no product takes them.
//
// The weights are the instruction's A operand, the tokens its B operand, so a lane's
// results are groups of four neighbouring rows of one token: one scale a lane and
// block, and stores of four elements.  Any order of the 128 columns does, as long as both
// operands use the same one.
#include <type_traits>

#include "lowp_types.h"

namespace bqm {
namespace {

constexpr int kBlk = 128;

typedef int i32x4 __attribute__((ext_vector_type(4)));

struct Fp8Args {
  const uint8_t *w;          // [experts, rows, 128 kb]
  const float *ws;           // [experts, ceil(rows / 128), kb]
  const uint8_t *q;          // [m, 128 kb]
  const float *qs;           // [kb, m]
  const int32_t *offsets;    // [experts + 1], or null: one matrix, rows of y = m
  const int32_t *row_ids;    // [slots], or null: row p of y is activation row p
  int experts, rows, kb, m, slots;
};

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// Eight codes as fp16.
__device__ __forceinline__ f16x8 widen(int lo, int hi) {
  f16x8 h;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(i ? hi : lo, 1.0f, false);
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(i ? hi : lo, 1.0f, true);
    h[4 * i] = a[0];
    h[4 * i + 1] = a[1];
    h[4 * i + 2] = b[0];
    h[4 * i + 3] = b[1];
  }
  return h;
}

// A workgroup's part of y: rows [p0, p1) (at most BM) of expert e, weight rows from n0.
struct Tile {
  int e, p0, p1, n0;
};

__device__ __forceinline__ int clamp_off(const Fp8Args &A, int e) {
  const int v = A.offsets[e];
  return v < 0 ? 0 : v > A.slots ? A.slots : v;
}

// Tiles [0, total) handed to the workgroups so that the ones of one XCD (every
// eighth workgroup) are neighbours: they share weights and activations in its L2.
__device__ __forceinline__ int xcd_order(int bid, int total) {
  const int per = total >> 3, extra = total & 7;
  const int x = bid & 7, i = bid >> 3;
  return x * per + (x < extra ? x : extra) + i;
}

// Place `l` of an expert's mt x nt tiles: bands of 8 tiles of rows, rows first.
__device__ __forceinline__ void place_tile(int l, int mt, int nt, int *mi, int *ni) {
  const int band = l / (8 * nt);
  const int h = min(8, mt - band * 8);
  const int in = l - band * 8 * nt;
  *mi = band * 8 + in % h;
  *ni = in / h;
}

// The tile of workgroup `bid`; false past the last one.  Every wave searches the
// expert for itself, 64 experts at a time.
template <int BM, int BN>
__device__ __forceinline__ bool find_tile(const Fp8Args &A, int bid, Tile *t) {
  const int nt = (A.rows + BN - 1) / BN;
  int mi, ni;
  if (!A.offsets) {
    const int mt = (A.m + BM - 1) / BM;
    place_tile(xcd_order(bid, mt * nt), mt, nt, &mi, &ni);
    *t = {0, mi * BM, min(A.m, mi * BM + BM), ni * BN};
    return true;
  }
  const int lane = threadIdx.x & 63;
  int total = 0, lo = 0, hi = 0, inc = 0;
  for (int pass = 0, want = 0; pass < 2; ++pass) {
    int before = 0;
    for (int e0 = 0; e0 < A.experts; e0 += 64) {
      const int e = e0 + lane;
      if (pass == 0 || A.experts > 64) {              // up to 64 experts stay in the lanes
        lo = e < A.experts ? clamp_off(A, e) : 0;
        hi = e < A.experts ? max(lo, clamp_off(A, e + 1)) : 0;
        inc = (hi - lo + BM - 1) / BM;
        inc = wave_prefix(inc);
      }
      const int sum = __builtin_amdgcn_readlane(inc, 63);
      if (pass == 1 && want < (before + sum) * nt) {
        const int at = __popcll(__ballot((before + inc) * nt <= want));
        const int first = before + (at ? __builtin_amdgcn_readlane(inc, at - 1) : 0);
        const int p0 = __builtin_amdgcn_readlane(lo, at), p1 = __builtin_amdgcn_readlane(hi, at);
        place_tile(want - first * nt, (p1 - p0 + BM - 1) / BM, nt, &mi, &ni);
        // ascending offsets always pass; others, whose counts may overflow, stay in their buffers
        if (e0 + at >= A.experts || (unsigned)mi >= (unsigned)((p1 - p0 + BM - 1) / BM) || (unsigned)ni >= (unsigned)nt)
          return false;
        *t = {e0 + at, p0 + mi * BM, min(p1, p0 + mi * BM + BM), ni * BN};
        return true;
      }
      before += sum;
    }
    if (pass == 0) {
      total = before * nt;
      if (bid >= total) return false;
      want = xcd_order(bid, total);
    }
  }
  return false;
}

// The activation row of row p of y.
__device__ __forceinline__ int token_of(const Fp8Args &A, int p) {
  if (!A.row_ids) return p;
  const int t = A.row_ids[p];
  return t < 0 ? 0 : t >= A.m ? A.m - 1 : t;
}

// Four neighbouring results of row p from column r on.
template <typename Y>
__device__ __forceinline__ void store4(Y *y, const Fp8Args &A, int p, int r, f32x4_t v) {
  typedef Y yx4 __attribute__((ext_vector_type(4)));
  Y *o = y + (int64_t)p * A.rows + r;
  if ((A.rows & 3) == 0 && r + 4 <= A.rows && ((uintptr_t)y & (4 * sizeof(Y) - 1)) == 0) {
    yx4 c;
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = from_f32<Y>(v[i]);
    *reinterpret_cast<yx4 *>(o) = c;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r + i < A.rows) o[i] = from_f32<Y>(v[i]);
  }
}

// ------------------------------------------------------------------ scales whose product is far
//
// The kernels multiply a block's two scales with each other and then with the block's sum.
// Where the product is no normal number although both are numbers other than 0, it
// overflows, or loses bits that the sum would bring back.  Rows that may hold such a product are
// looked at after they are stored, and those that do are computed once more, one code after the
// other.  How a wave knows: a tile keeps the largest past_normal of its products (two
// instructions a token and block; at most 0.5% of the time); the stream kernel, where that cost 5%
// to 8%, looks at its results: an overflow leaves an infinity or a NaN, and bits lost below
// 2^-149 of a scale are at most 2^-125 a block, which is below the rounding of
// results from 2^-100 on.  (Applying one scale after the other in every block cost 2% to 8%.)

// 0xFE000000 and more for 0, subnormals, infinities and NaN.
__device__ __forceinline__ uint32_t past_normal(float s) { return (__float_as_uint(s) << 1) - 0x01000000u; }
constexpr uint32_t kPast = 0xFE000000u;

__device__ __forceinline__ bool product_far(float a, float b) {
  constexpr int kNumber = 0x198;                               // the classes of normal and subnormal numbers
  return past_normal(a * b) >= kPast && __builtin_amdgcn_classf(a, kNumber) && __builtin_amdgcn_classf(b, kNumber);
}

// acc + sum a b.  The exponents of a and b are shared out: sum times 2^h is exact, and that
// times s leaves fp32's range only where the sum of the three does; past 2^180 either
// way every sum but 0 does.
__device__ __forceinline__ float add_scaled(float sum, float a, float b, float acc) {
  const int e = min(max(__builtin_amdgcn_frexp_expf(a) + __builtin_amdgcn_frexp_expf(b), -180), 180), h = e >> 1;
  const float s = ldexpf(__builtin_amdgcn_frexp_mantf(a) * __builtin_amdgcn_frexp_mantf(b), e - h);
  return fmaf(ldexpf(sum, h), s, acc);
}

// The wave's N rows of y from p0 on (below p1), columns r0 .. r0 + R - 1 (of one scale block).
template <typename Y, int N, int R>
__device__ __forceinline__ void redo_far(const Fp8Args &A, Y *y, int e, int p0, int p1, int r0, int lane) {
  if (p0 >= p1) return;
  const float *ws = A.ws + ((int64_t)e * ((A.rows + kBlk - 1) / kBlk) + r0 / kBlk) * A.kb;
  const float *qs = A.qs + token_of(A, min(p0 + lane % N, p1 - 1));
  bool far = false;
  for (int b = lane / N; b < A.kb; b += 64 / N) far |= product_far(qs[(int64_t)b * A.m], ws[b]);
  uint64_t rows = __ballot(far);                               // bit i of any N: row p0 + i
#pragma unroll
  for (int n = 32; n >= N; n /= 2) rows |= rows >> n;
  __threadfence();                                             // the rows' first stores come first
  const int64_t kp = (int64_t)A.kb * kBlk;
  const int r = r0 + lane;
  const uint32_t *w = reinterpret_cast<const uint32_t *>(A.w + ((int64_t)e * A.rows + min(r, A.rows - 1)) * kp);
  for (int i = 0; i < N && p0 + i < p1; ++i) {
    if (!(rows >> i & 1)) continue;
    const int tok = token_of(A, p0 + i);
    const uint32_t *q = reinterpret_cast<const uint32_t *>(A.q + tok * kp);
    float acc = 0.0f;
    for (int b = 0; b < A.kb; ++b) {
      float sum = 0.0f;
      for (int j = b * (kBlk / 4); j < (b + 1) * (kBlk / 4); ++j) {
        const int u = (int)w[j], v = (int)q[j];
        sum = fmaf(__builtin_amdgcn_cvt_f32_fp8(u, 0), __builtin_amdgcn_cvt_f32_fp8(v, 0), sum);
        sum = fmaf(__builtin_amdgcn_cvt_f32_fp8(u, 1), __builtin_amdgcn_cvt_f32_fp8(v, 1), sum);
        sum = fmaf(__builtin_amdgcn_cvt_f32_fp8(u, 2), __builtin_amdgcn_cvt_f32_fp8(v, 2), sum);
        sum = fmaf(__builtin_amdgcn_cvt_f32_fp8(u, 3), __builtin_amdgcn_cvt_f32_fp8(v, 3), sum);
      }
      acc = add_scaled(sum, A.qs[(int64_t)b * A.m + tok], ws[b], acc);
    }
    if (lane < R && r < A.rows) y[(int64_t)(p0 + i) * A.rows + r] = from_f32<Y>(acc);
  }
}

// ------------------------------------------------------------------ few rows a matrix
//
// The weights are read once and bound the time.  A workgroup takes 16 weight
// rows and up to 16 MF tokens; its waves take every NW-th block of the columns and
// load operands straight into the matrix cores' registers, kDepth blocks ahead; the
// waves' sums meet in LDS.  A lane loads the 16-byte chunks g and g + 4 of a row (g its
// group of 16 lanes), so one load reads 64 neighbouring bytes of each of 16 rows.  One token
// of 4096x4096: 5.6 us for 3.4 us of bytes, the rest an empty launch (1.7) and the chain
// from tile to loads to sum; of 32768x4096: 30 us, 4.5 TB/s.
template <typename Y, int MF, int NW, int kDepth>
__global__ __launch_bounds__(64 * NW) void fp8_stream_kernel(Fp8Args A, Y *__restrict__ y) {
  Tile t;
  if (!find_tile<16 * MF, 16>(A, blockIdx.x, &t)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, grp = lane >> 4;
  const int64_t kp = (int64_t)A.kb * kBlk;
  const uint8_t *w = A.w + ((int64_t)t.e * A.rows + min(t.n0 + row, A.rows - 1)) * kp + grp * 16;
  const float *ws = A.ws + ((int64_t)t.e * ((A.rows + kBlk - 1) / kBlk) + t.n0 / kBlk) * A.kb;
  // the weights' addresses depend on the tile alone: they go out before the tokens are known
  i32x4 wl[kDepth][2] = {};
  auto load_w = [&](int b0) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int b = b0 + d * NW;
      if (b < A.kb) {
        const uint8_t *p = w + (int64_t)b * kBlk;
        wl[d][0] = *reinterpret_cast<const i32x4 *>(p);
        wl[d][1] = *reinterpret_cast<const i32x4 *>(p + 64);
      }
    }
  };
  load_w(wave);
  const uint8_t *q[MF];
  const float *qs[MF];
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    const int tok = token_of(A, min(t.p0 + f * 16 + row, t.p1 - 1));
    q[f] = A.q + tok * kp + grp * 16;
    qs[f] = A.qs + tok;
  }
  f32x4_t acc[MF] = {};
  for (int b0 = wave; b0 < A.kb; b0 += NW * kDepth) {
    i32x4 ql[kDepth][MF][2];
    float sc[kDepth][MF], sw[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int b = b0 + d * NW;
      if (b < A.kb) {
        sw[d] = ws[b];
#pragma unroll
        for (int f = 0; f < MF; ++f) {
          const uint8_t *p = q[f] + (int64_t)b * kBlk;
          ql[d][f][0] = *reinterpret_cast<const i32x4 *>(p);
          ql[d][f][1] = *reinterpret_cast<const i32x4 *>(p + 64);
          sc[d][f] = qs[f][(int64_t)b * A.m];
        }
      }
    }
    f16x8 wh[kDepth][4];
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
#pragma unroll
      for (int k = 0; k < 4; ++k) wh[d][k] = widen(wl[d][k / 2][2 * (k & 1)], wl[d][k / 2][2 * (k & 1) + 1]);
    load_w(b0 + NW * kDepth);
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      if (b0 + d * NW < A.kb) {
#pragma unroll
        for (int f = 0; f < MF; ++f) {
          f32x4_t part = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            part = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                wh[d][k], widen(ql[d][f][k / 2][2 * (k & 1)], ql[d][f][k / 2][2 * (k & 1) + 1]), part, 0, 0, 0);
          const float s = sc[d][f] * sw[d];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[f][i] = fmaf(part[i], s, acc[f][i]);
        }
      }
    }
  }
  static_assert(MF <= NW, "a wave for every fragment");
  __shared__ f32x4_t red[NW][MF][64];
#pragma unroll
  for (int f = 0; f < MF; ++f) red[wave][f][lane] = acc[f];
  __syncthreads();
  if (wave >= MF) return;
  f32x4_t sum = red[0][wave][lane];                   // wave f adds up and stores fragment f
#pragma unroll
  for (int v = 1; v < NW; ++v) sum += red[v][wave][lane];
  const int p = t.p0 + wave * 16 + row;
  if (p < t.p1) store4(y, A, p, t.n0 + grp * 4, sum);
  bool look = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) look |= !(fabsf(sum[i]) >= 0x1p-100f && fabsf(sum[i]) < INFINITY);
  if (__builtin_expect(__ballot(look) != 0, 0))
    redo_far<Y, 16, 16>(A, y, t.e, t.p0 + wave * 16, t.p1, t.n0, lane);
}

// ------------------------------------------------------------------ tiles
//
// BM tokens x BN weight rows, WM x WN waves.  Per block of 128 columns both
// operands' tiles and scales go to LDS without passing through registers, into one of
// NS buffers while others are multiplied.  A tile's rows are 128 bytes; chunk c of
// row r is stored at chunk c ^ ((r >> 1) & 7), so that the 16 rows a fragment load
// touches at one chunk lie in 16 different groups of four banks (the loads counted none).
// They are buffer loads: the next block costs one scalar addition, where flat addresses
// cost a 64-bit vector addition a load.

typedef __attribute__((address_space(3))) void lds_void;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void *base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, -1, 0x00020000);
}

// A wave's 1 KiB (8 rows of 128 bytes) of each of N loads, `step` bytes apart in LDS.
template <int N>
__device__ __forceinline__ void stage_rows(const uint8_t *base, const uint32_t *off, int add, uint8_t *to, int step) {
  const __amdgpu_buffer_rsrc_t r = rsrc_of(base);
#pragma unroll
  for (int i = 0; i < N; ++i)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)(to + i * step), 16, off[i], add, 0, 0);
}

// 64 scales, one a lane.
__device__ __forceinline__ void stage_scales(const float *base, uint32_t off, uint8_t *to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc_of(base), (lds_void *)to, 4, off, 0, 0, 0);
}

// All but the wave's last N loads to LDS have landed and its reads are done, then so
// are everyone's.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// kTurn tokens' results from LDS (kRow bytes each, 16-byte piece c of token t at c ^ t) to
// y's rows from p0 and columns from r0 on, a unit U a lane and neighbouring lanes side by
// side; rows from p1 and columns past the matrix are left out.
template <typename U, typename Y, int kTurn, int kRow>
__device__ __forceinline__ void store_turned(const uint8_t *from, Y *y, const Fp8Args &A, int p0, int p1, int r0,
                                             int lane) {
  constexpr int kUnits = kRow / (int)sizeof(U), kPieces = kRow / 16;
  static_assert(64 % kUnits == 0, "a wave stores whole tokens");
#pragma unroll
  for (int i = 0; i < kTurn * kUnits / 64; ++i) {
    const int tt = i * (64 / kUnits) + lane / kUnits, byte = lane % kUnits * (int)sizeof(U);
    const U v = *reinterpret_cast<const U *>(from + tt * kRow + (((byte >> 4) ^ (tt & (kPieces - 1))) << 4) + (byte & 15));
    const int p = p0 + tt, r = r0 + byte / (int)sizeof(Y);
    if (p < p1 && r < A.rows) *reinterpret_cast<U *>(y + (int64_t)p * A.rows + r) = v;
  }
}

template <typename Y, int BM, int BN, int WM, int WN, int NS>
__global__ __launch_bounds__(64 * WM * WN, 2) void fp8_tile_kernel(Fp8Args A, Y *__restrict__ y) {
  constexpr int NW = WM * WN;
  constexpr int TM = BM / WM / 32, TN = BN / WN / 32;
  constexpr int kRowsPerLoad = NW * 8;
  constexpr int LM = BM / kRowsPerLoad, LN = BN / kRowsPerLoad, kLoads = LM + LN + 1;
  static_assert(BM % kRowsPerLoad == 0 && BN % kRowsPerLoad == 0, "whole loads");
  static_assert(BN <= kBlk && kBlk % BN == 0 && BM % 64 == 0 && BM / 64 < NW, "one scale block of weights a tile");
  constexpr int kScale = (BM + BN) * kBlk;                      // scales behind the codes
  constexpr int kStage = kScale + (BM + 64) * 4;
  __shared__ __align__(1024) uint8_t lds[NS * kStage];

  Tile t;
  if (!find_tile<BM, BN>(A, blockIdx.x, &t)) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int row = lane & 31, half = lane >> 5;
  const int64_t kp = (int64_t)A.kb * kBlk;

  // loads: wave w brings rows 8 w .. 8 w + 7 of every kRowsPerLoad, from a uniform base
  // (the tile's first row, or, for gathered rows, the first activation) and 32-bit offsets
  const int lr = wave * 8 + (lane >> 3), slot = lane & 7;
  const uint32_t kp32 = (uint32_t)A.kb * kBlk;
  const uint8_t *qb = A.q + (A.row_ids ? 0 : t.p0 * kp);
  const uint8_t *wb = A.w + ((int64_t)t.e * A.rows + t.n0) * kp;
  const int pmax = t.p1 - 1 - t.p0, nmax = A.rows - 1 - t.n0;   // last valid rows of the tile
  auto q_row = [&](int r) {
    const int i = min(r, pmax);
    return A.row_ids ? token_of(A, t.p0 + i) : i;
  };
  uint32_t src[LM + LN];
#pragma unroll
  for (int i = 0; i < LM + LN; ++i) {
    const int r = (i < LM ? i : i - LM) * kRowsPerLoad + lr;
    src[i] = (uint32_t)(i < LM ? q_row(r) : min(r, nmax)) * kp32 + ((slot ^ ((r >> 1) & 7)) << 4);
  }
  // scales: the first BM / 64 waves bring the tokens', the others the weights'
  const bool token_wave = wave < BM / 64;
  const int nblk = (A.rows + kBlk - 1) / kBlk;
  const float *sb = token_wave ? A.qs + (A.row_ids ? 0 : t.p0) : A.ws + ((int64_t)t.e * nblk + t.n0 / kBlk) * A.kb;
  const int64_t sstep = token_wave ? A.m : 1;
  const uint32_t soff = token_wave ? (uint32_t)q_row(wave * 64 + lane) * 4 : 0;
  const int sdst = kScale + (token_wave ? wave * 256 : BM * 4);
  auto load_stage = [&](int at, int b) {
    stage_rows<LM>(qb, src, b * kBlk, lds + at + wave * 1024, kRowsPerLoad * kBlk);
    stage_rows<LN>(wb, src + LM, b * kBlk, lds + at + wave * 1024 + BM * kBlk, kRowsPerLoad * kBlk);
    stage_scales(sb + b * sstep, soff, lds + at + sdst);
  };
  auto load_one = [&](int at, int b, int i) {                  // load i of load_stage's kLoads
    uint8_t *to = lds + at + wave * 1024 + i * kRowsPerLoad * kBlk;
    if (i < LM) stage_rows<1>(qb, src + i, b * kBlk, to, 0);
    else if (i < LM + LN) stage_rows<1>(wb, src + i, b * kBlk, to, 0);
    else if (i == LM + LN) stage_scales(sb + b * sstep, soff, lds + at + sdst);
  };

  // The pipeline.  Chain c of a block multiplies row fragment c / TM and token fragment
  // c % TM in 8 steps of 16 columns.  By chain kMeet
  // every wave has read the block's last fragments: there the waves meet, the next
  // block's loads have landed, and the buffer takes the block NS ahead, the loads
  // spread over the steps left: a compute unit's loads to LDS go 64 bytes a cycle, and a wave
  // that issues all of them at once waits for its turns (8 of them held up the first
  // chain by 500 of the block's 2600 cycles).  Between a chain's steps the next step's
  // codes are widened, the sums of the chain before are scaled and added, and fragments and
  // scales of the chains ahead are read, the next block's first ones during the last
  // (4096 x 14336 x 4096: 438 us with loads and reads at the block's start, 406 so;
  // 256 x 4096 x 4096 on 64 x 64 tiles 20.3, 17.0).
  constexpr int C = TN * TM, kMeet = TN > 1 ? (TN - 2) * TM + 1 : 0;
  constexpr int kEvery = 8 * (C - kMeet) / kLoads;           // steps a load
  static_assert(kEvery >= 1, "every load has a step");
  const int sz = (row >> 1) & 7;
  int coff[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) coff[j] = row * kBlk + (((2 * j + half) ^ sz) << 4);
  const int fq = wm * TM * 32 * kBlk, fw = BM * kBlk + wn * TN * 32 * kBlk;
  auto chunk = [&](int at, int j) { return *reinterpret_cast<const i32x4 *>(lds + at + coff[j]); };
  auto scale_of = [&](int at, int i) { return reinterpret_cast<const float *>(lds + at + kScale)[i]; };
  f32x16 acc[TN][TM] = {}, last = {};
  float s[TM], s_last = 0.0f;
  uint32_t past = 0;                                           // the largest past_normal of the scales' products
  i32x4 rw[TN][4], rq[TM][4];
#pragma unroll
  for (int i = 0; i < NS; ++i)
    if (i < A.kb) load_stage(i * kStage, i);
  if (NS <= A.kb) wait_and_meet<(NS - 1) * kLoads>();
  else wait_and_meet<0>();
  const bool any_row = wm * TM * 32 <= pmax;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    rw[0][j] = chunk(fw, j);
    rq[0][j] = chunk(fq, j);
  }
#pragma unroll
  for (int f = 0; f < TM; ++f) {
    s[f] = scale_of(0, (wm * TM + f) * 32 + row) * scale_of(0, BM);
    past = max(past, past_normal(s[f]));
  }
  f16x8 qh[TM][8], wh[8];
  auto eighth = [](const i32x4 (&r)[4], int k) { return widen(r[k / 2][2 * (k & 1)], r[k / 2][2 * (k & 1) + 1]); };
  wh[0] = eighth(rw[0], 0);
  qh[0][0] = eighth(rq[0], 0);
  if (!any_row) {                                              // only loads and meets
    for (int b = 0, at = 0; b + 1 < A.kb; ++b) {
      if (b + NS - 1 < A.kb) wait_and_meet<(NS - 2) * kLoads>();
      else wait_and_meet<0>();
      if (b + NS < A.kb) load_stage(at, b + NS);
      at = at + kStage < NS * kStage ? at + kStage : 0;
    }
    return;
  }
  int at = 0;
  // one block; kMore: with loads of the block NS ahead, kNext: with another block after it
  auto block = [&](int b, auto more, auto next) __attribute__((always_inline)) {
    constexpr bool kMore = decltype(more)::value, kNext = decltype(next)::value;
    const int nx = at + kStage < NS * kStage ? at + kStage : 0;
    i32x4 rwn[4], rqn[4];
    float sn[TM], swn;
    f32x16 part[2];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int g = c / TM, f = c % TM;
      if (kNext && c == kMeet) {
        if (kMore || b + NS - 1 < A.kb) wait_and_meet<(NS - 2) * kLoads>();
        else wait_and_meet<0>();
      }
      const int pc = c ? c - 1 : C - 1, pg = pc / TM, pf = pc % TM;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int step = (c - kMeet) * 8 + k;
        if (kMore && step >= 0 && step % kEvery == 0 && step / kEvery < kLoads) load_one(at, b + NS, step / kEvery);
        if (k < 4) {
          if (g == 0 && f + 1 < TM) rq[f + 1][k] = chunk(at + fq + (f + 1) * 32 * kBlk, k);
          if (f == 0 && g + 1 < TN) rw[g + 1][k] = chunk(at + fw + (g + 1) * 32 * kBlk, k);
          if (kNext && c == C - 1) {
            rwn[k] = chunk(nx + fw, k);
            rqn[k] = chunk(nx + fq, k);
          }
        } else if (kNext && c == C - 1 && k == 4) {
#pragma unroll
          for (int i = 0; i < TM; ++i) sn[i] = scale_of(nx, (wm * TM + i) * 32 + row);
          swn = scale_of(nx, BM);
        }
        const f32x16 zero = {};
        part[c & 1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(wh[k], qh[f][k], k ? part[c & 1] : zero, 0, 0, 0);
        const int k1 = (k + 1) & 7, c1 = k == 7 ? c + 1 : c, g1 = c1 / TM, f1 = c1 % TM;
        if (c1 < C) {
          if (f1 == 0) wh[k1] = eighth(rw[g1], k1);
          if (g1 == 0) qh[f1][k1] = eighth(rq[f1], k1);
        } else if (kNext) {
          wh[0] = eighth(rwn, 0);
          qh[0][0] = eighth(rqn, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 2 * k; i < 2 * k + 2; ++i)
          acc[pg][pf][i] = fmaf(c ? part[(c - 1) & 1][i] : last[i], c ? s[pf] : s_last, acc[pg][pf][i]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    last = part[(C - 1) & 1];
    s_last = s[TM - 1];
    if constexpr (kNext) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        rw[0][j] = rwn[j];
        rq[0][j] = rqn[j];
      }
#pragma unroll
      for (int f = 0; f < TM; ++f) {
        s[f] = sn[f] * swn;
        past = max(past, past_normal(s[f]));
      }
    }
    at = nx;
  };
  int b = 0;
  for (; b + NS < A.kb; ++b) block(b, std::true_type{}, std::true_type{});
  for (; b + 1 < A.kb; ++b) block(b, std::false_type{}, std::true_type{});
  block(b, std::false_type{}, std::false_type{});
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[TN - 1][TM - 1][i] = fmaf(last[i], s_last, acc[TN - 1][TM - 1][i]);
  // Results.  A lane holds four neighbouring rows of a token at a time, 8 bytes of 16
  // bits; written as they are, every token's 16 bytes would be a write of its own in L2.
  // Each wave turns 32 tokens around (16 where they are too long) in a part of its own
  // of the buffer after the last block's, which nobody reads or loads any more, and stores
  // whole stretches of TN x 32 rows, 16 bytes a lane.  Piece c of token t lies at c ^ t,
  // modulo the pieces.  (4096 x 4096 x 2048: 71.5 us stored as they are, 62.7 so.)
  constexpr int kRow = TN * 32 * (int)sizeof(Y), kPieces = kRow / 16;
  constexpr int kTurn = NW * 32 * kRow <= kStage ? 32 : 16;
  static_assert(NW * kTurn * kRow <= kStage, "a buffer holds every wave's tokens");
  typedef Y yx4 __attribute__((ext_vector_type(4)));
  uint8_t *mine = lds + at + wave * kTurn * kRow;
  // the widest unit that every row's start is a multiple of
  const uint64_t align = (uint64_t)A.rows * sizeof(Y) | (uintptr_t)y;
  const int unit = (align & 15u) == 0 ? 16 : (align & 3u) == 0 ? 4 : 2;
#pragma unroll
  for (int h = 0; h < TM * 32 / kTurn; ++h) {
    const int f = h * kTurn / 32, first = h * kTurn % 32;        // tokens [first, first + kTurn) of fragment f
#pragma unroll
    for (int g = 0; g < TN; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (row < first || row >= first + kTurn) continue;
        const int o = (g * 32 + 8 * i + 4 * half) * (int)sizeof(Y);
        yx4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float a = acc[g][f][4 * i + j];
          // the fp32 sum is what is rounded: joined by the compiler, some elements' last
          // addition and rounding to fp16 were one instruction, which rounds another sum
          if constexpr (std::is_same_v<Y, _Float16>) asm("" : "+v"(a));
          v[j] = from_f32<Y>(a);
        }
        *reinterpret_cast<yx4 *>(mine + (row - first) * kRow + (((o >> 4) ^ (row & (kPieces - 1))) << 4) + (o & 15)) = v;
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int p0 = t.p0 + (wm * TM + f) * 32 + first, r0 = t.n0 + wn * TN * 32;
    if (unit == 16) store_turned<u32x4_t, Y, kTurn, kRow>(mine, y, A, p0, t.p1, r0, lane);
    else if (sizeof(Y) == 4 || unit == 4) store_turned<uint32_t, Y, kTurn, kRow>(mine, y, A, p0, t.p1, r0, lane);
    else if constexpr (sizeof(Y) == 2) store_turned<uint16_t, Y, kTurn, kRow>(mine, y, A, p0, t.p1, r0, lane);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
  if (__builtin_expect(__ballot(past >= kPast) != 0, 0)) {
#pragma unroll 1
    for (int f = 0; f < TM; ++f)
      redo_far<Y, 32, TN * 32>(A, y, t.e, t.p0 + (wm * TM + f) * 32, t.p1, t.n0 + wn * TN * 32, lane);
  }
}

// ------------------------------------------------------------------ dispatch

// Workgroups that cover every tile whatever the offsets are: an expert's rows take
// at most one tile more than they fill.
int64_t tiles(int rows, int slots, int experts, int bm, int bn) {
  const int64_t nt = ((int64_t)rows + bn - 1) / bn;
  return nt * (experts ? slots / bm + (experts < slots ? experts : slots) : ((int64_t)slots + bm - 1) / bm);
}
int64_t tiles(const Fp8Args &A, int bm, int bn) { return tiles(A.rows, A.slots, A.offsets ? A.experts : 0, bm, bn); }

// rows a matrix has to multiply: exact for one matrix, the mean for experts
int rows_each(int slots, int experts) { return experts ? (int)(((int64_t)slots + experts - 1) / experts) : slots; }
constexpr int kManyRows = 96;             // from here on 128 x 128 tiles, see run

template <typename Y, int MF, int NW, int kDepth>
hipError_t stream(const Fp8Args &A, Y *y, hipStream_t s) {
  fp8_stream_kernel<Y, MF, NW, kDepth><<<(unsigned)tiles(A, 16 * MF, 16), 64 * NW, 0, s>>>(A, y);
  return hipGetLastError();
}

template <typename Y, int BM, int BN, int WM, int WN, int NS>
hipError_t tile(const Fp8Args &A, Y *y, hipStream_t s) {
  fp8_tile_kernel<Y, BM, BN, WM, WN, NS><<<(unsigned)tiles(A, BM, BN), 64 * WM * WN, 0, s>>>(A, y);
  return hipGetLastError();
}

// One fragment of tokens.  8 waves a workgroup, 4 where the rows are short and there are
// workgroups enough (us with 4 / 8 waves, one token: 4096x4096 8.2 / 6.3, 14336x4096 16.2 /
// 16.0, 4096x14336 24.3 / 17.3, 8 of 64 matrices of 2048x2048 11.8 / 13.4, 1092x312 2.6 / 2.7)
template <typename Y>
hipError_t stream1(const Fp8Args &A, Y *y, int num_cus, hipStream_t s) {
  const bool four = A.kb <= 4 || (A.kb <= 16 && tiles(A, 16, 16) > 2 * num_cus);
  return four ? stream<Y, 1, 4, 2>(A, y, s) : stream<Y, 1, 8, 2>(A, y, s);
}

template <typename Y>
hipError_t run(const Fp8Args &A, Y *y, int num_cus, hipStream_t s) {
  const int per = rows_each(A.slots, A.offsets ? A.experts : 0);
  // few tiles: the smallest token tile that leaves none of them waiting for a CU (us at 64
  // tokens: 1024x4096 6.3 with 16 a tile, 4096x4096 12.4 with 64; 64 x 64 tiles 15.5, 16.1)
  if (tiles(A, 16, 16) <= num_cus) return stream1(A, y, num_cus, s);
  if (tiles(A, 32, 16) <= num_cus) return stream<Y, 2, 8, 1>(A, y, s);
  if (tiles(A, 64, 16) <= num_cus) return stream<Y, 4, 8, 1>(A, y, s);
  // many: 128 x 128 tiles, two workgroups a CU (us, 512 tokens of 14336x4096: 62, with 64 x 128
  // tiles 73; 300 tokens 50, 51; 64 matrices of 2048x2048 with 128 rows each: 86 against 98, with
  // 96: 77 against 87)
  if (per >= kManyRows && tiles(A, 128, 128) >= num_cus) return tile<Y, 128, 128, 2, 2, 2>(A, y, s);
  // experts' matrices, and more than 8 tokens of one, as soon as tiles fill most CUs: 64 x 128,
  // three blocks deep, or 64 x 64, four deep (us, 64 matrices of 2048x2048 with 1/4, 2, 8 and
  // 32 rows each: 64 x 128 15 / 43 / 54 / 61, 16 rows a workgroup 17 / 49 / 74 / 154; one matrix
  // of 14336x4096 with 16, 32 and 128 tokens: 64 x 64 16.7 / 17.3 / 29.1, 64 x 128 21.2 / 21.6 /
  // 24.6, 16 or 32 rows a workgroup 20.0 / 26.0 / 79; of 32768x4096 with 8: 35 / 37 / 34)
  const int most = num_cus * 3 / 4;
  if (A.offsets || per > 8) {
    if (tiles(A, 64, 128) >= most) return tile<Y, 64, 128, 2, 2, 3>(A, y, s);
    if (tiles(A, 64, 64) >= most && per > 8) return tile<Y, 64, 64, 2, 2, 4>(A, y, s);
  }
  if (per <= 16) return stream1(A, y, num_cus, s);
  // too few tiles: up to 32 tokens reading the weights once counts (us at 32, 4096x14336: 16.6
  // against 48)
  if (per <= 32) return stream<Y, 2, 8, 1>(A, y, s);
  return tile<Y, 64, 64, 2, 2, 4>(A, y, s);
}

hipError_t run_any(const Fp8Args &A, void *y, int ydtype, int num_cus, hipStream_t s) {
  if (ydtype == BQM_F32) return run(A, (float *)y, num_cus, s);
  if (ydtype == BQM_BF16) return run(A, (__bf16 *)y, num_cus, s);
  return run(A, (_Float16 *)y, num_cus, s);
}

}  // namespace

// The most workgroups that run may launch; its other choices are for few tiles.
bool fp8_gemm_fits(int rows, int slots, int experts) {
  const int bm = rows_each(slots, experts) >= kManyRows ? 128 : 64;
  return tiles(rows, slots, experts, bm, 128) < kMaxGroups256;
}

hipError_t launch_fp8_gemm(const uint8_t *w, const float *ws, int rows, int cols, const uint8_t *q, const float *qs,
                           int m, void *y, int ydtype, int num_cus, hipStream_t s) {
  const Fp8Args A{w, ws, q, qs, nullptr, nullptr, 1, rows, (cols + kBlk - 1) / kBlk, m, m};
  return run_any(A, y, ydtype, num_cus, s);
}

hipError_t launch_fp8_gemm_grouped(const uint8_t *w, const float *ws, int experts, int rows, int cols,
                                   const uint8_t *q, const float *qs, int m, const int32_t *offsets,
                                   const int32_t *row_ids, int slots, void *y, int ydtype, int num_cus,
                                   hipStream_t s) {
  const Fp8Args A{w, ws, q, qs, offsets, row_ids, experts, rows, (cols + kBlk - 1) / kBlk, m, slots};
  return run_any(A, y, ydtype, num_cus, s);
}

}  // namespace bqm
