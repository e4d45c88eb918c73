// Products of E4M3 activations and weights with a scale for each block of 128,
// dense and grouped by expert.
//
//   y[t, r] = sum_b sx[b, t] * sw[r / 128, b] * sum_{j < 128} q[t, 128 b + j] * w[r, 128 b + j]
//
// The blocks' sums are scaled and added in fp32 and y is rounded once.  A block's own
// sum is formed on the matrix cores in one of two ways:
//
//  * exactly: the codes become fp16 in registers (E4M3 is exact there), and the fp16
//    instruction sums products in fp32.  Results in fp32, few rows a matrix (bound by
//    reading the weights, so the conversions are free) and short rows take this.
//  * natively: v_mfma_f32_16x16x128_f8f6f4 spans a block in one instruction at four
//    times the fp16 instruction's rate a byte.  It keeps, of each 8 products, only 13
//    bits below the largest one: measured, 1.7e-5 of the result's norm.  That is 1 / 100
//    of a bf16 result's rounding and 1 / 14 of an fp16 one's, so results in 16 bits
//    take it, from 8 blocks on, where the errors of the blocks average out.
//
// The weights are the instruction's A operand (16 weight rows), the tokens its B
// operand (16 tokens), so a lane's four results are four neighbouring rows of one
// token: one scale a lane and block, and stores of four elements.  Any order of the 128
// columns does, as long as both operands use the same one: lane group g holds the
// 16-byte chunks g and g + 4 of a row, so that one load instruction reads 64
// neighbouring bytes of each of 16 rows.
#include "lowp_types.h"

namespace bqm {
namespace {

constexpr int kBlk = 128;

typedef int i32x8 __attribute__((ext_vector_type(8)));
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

__device__ __forceinline__ f32x4_t mma(i32x8 w, i32x8 q) {
  const f32x4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, q, zero, 0, 0, 0, 0, 0, 0);
}

// The block's sum with fp32's precision: the codes as fp16, in which E4M3 is exact,
// on v_mfma_f32_16x16x32_f16, which keeps products and sums of them to fp32.
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

struct Halves {
  f16x8 k[4];
};

__device__ __forceinline__ Halves widen(i32x8 c) {
  Halves h;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[2 * s + i], 1.0f, false);
      const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[2 * s + i], 1.0f, true);
      h.k[s][4 * i] = a[0];
      h.k[s][4 * i + 1] = a[1];
      h.k[s][4 * i + 2] = b[0];
      h.k[s][4 * i + 3] = b[1];
    }
  }
  return h;
}

__device__ __forceinline__ f32x4_t mma(const Halves &w, const Halves &q) {
  f32x4_t c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_16x16x32_f16(w.k[s], q.k[s], c, 0, 0, 0);
  return c;
}

__device__ __forceinline__ i32x8 join(i32x4 a, i32x4 b) {
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
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
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
          const int u = __shfl_up(inc, o, 64);
          if (lane >= o) inc += u;
        }
      }
      const int sum = __builtin_amdgcn_readlane(inc, 63);
      if (pass == 1 && want < (before + sum) * nt) {
        const int at = __popcll(__ballot((before + inc) * nt <= want));
        const int first = before + (at ? __builtin_amdgcn_readlane(inc, at - 1) : 0);
        const int p0 = __builtin_amdgcn_readlane(lo, at), p1 = __builtin_amdgcn_readlane(hi, at);
        place_tile(want - first * nt, (p1 - p0 + BM - 1) / BM, nt, &mi, &ni);
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

// ------------------------------------------------------------------ few rows a matrix
//
// The weights are read once and bound the time.  A workgroup takes 16 weight
// rows and up to 16 MF tokens; its waves take every NW-th block of the columns and
// load operands straight into the matrix cores' registers, kDepth blocks ahead; the
// waves' sums meet in LDS.
template <typename Y, int MF, int NW, int kDepth>
__global__ __launch_bounds__(64 * NW) void fp8_stream_kernel(Fp8Args A, Y *__restrict__ y) {
  Tile t;
  if (!find_tile<16 * MF, 16>(A, blockIdx.x, &t)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row = lane & 15, grp = lane >> 4;
  const int64_t kp = (int64_t)A.kb * kBlk;
  const uint8_t *w = A.w + ((int64_t)t.e * A.rows + min(t.n0 + row, A.rows - 1)) * kp + grp * 16;
  const float *ws = A.ws + ((int64_t)t.e * ((A.rows + kBlk - 1) / kBlk) + t.n0 / kBlk) * A.kb;
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
    i32x4 wl[kDepth][2], ql[kDepth][MF][2];
    float sc[kDepth][MF], sw[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int b = min(b0 + d * NW, A.kb - 1);
      const uint8_t *p = w + (int64_t)b * kBlk;
      wl[d][0] = __builtin_nontemporal_load(reinterpret_cast<const i32x4 *>(p));
      wl[d][1] = __builtin_nontemporal_load(reinterpret_cast<const i32x4 *>(p + 64));
    }
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int b = min(b0 + d * NW, A.kb - 1);
      sw[d] = ws[b];
#pragma unroll
      for (int f = 0; f < MF; ++f) {
        const uint8_t *p = q[f] + (int64_t)b * kBlk;
        ql[d][f][0] = *reinterpret_cast<const i32x4 *>(p);
        ql[d][f][1] = *reinterpret_cast<const i32x4 *>(p + 64);
        sc[d][f] = qs[f][(int64_t)b * A.m];
      }
    }
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      if (b0 + d * NW < A.kb) {
        const Halves wh = widen(join(wl[d][0], wl[d][1]));
#pragma unroll
        for (int f = 0; f < MF; ++f) {
          const f32x4_t part = mma(wh, widen(join(ql[d][f][0], ql[d][f][1])));
          const float s = sc[d][f] * sw[d];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[f][i] = fmaf(part[i], s, acc[f][i]);
        }
      }
    }
  }
  if constexpr (NW > 1) {
    __shared__ f32x4_t red[NW][MF][64];
#pragma unroll
    for (int f = 0; f < MF; ++f) red[wave][f][lane] = acc[f];
    __syncthreads();
    if (wave >= MF) return;
    f32x4_t sum = red[0][wave][lane];                 // wave f adds up and stores fragment f
#pragma unroll
    for (int v = 1; v < NW; ++v) sum += red[v][wave][lane];
    const int p = t.p0 + wave * 16 + row;
    if (p < t.p1) store4(y, A, p, t.n0 + grp * 4, sum);
  }
}

// ------------------------------------------------------------------ tiles
//
// BM tokens x BN weight rows, WM x WN waves.  Per block of 128 columns both
// operands' tiles go to LDS without passing through registers, into one of two
// buffers while the other is multiplied.  A tile's rows are 128 bytes; chunk c of
// row r is stored at chunk c ^ ((r >> 1) & 7), so that the 16 rows a fragment
// load touches at one chunk lie in 16 different groups of four banks.
template <typename Y, int BM, int BN, int WM, int WN, bool kExact>
__global__ __launch_bounds__(64 * WM * WN) void fp8_tile_kernel(Fp8Args A, Y *__restrict__ y) {
  constexpr int NW = WM * WN;
  constexpr int TM = BM / WM / 16, TN = BN / WN / 16;         // fragments a wave
  constexpr int kRowsPerLoad = NW * 8;                         // rows all waves bring in one load
  constexpr int LM = BM / kRowsPerLoad, LN = BN / kRowsPerLoad;
  static_assert(BM % kRowsPerLoad == 0 && BN % kRowsPerLoad == 0, "whole loads");
  constexpr int kStage = (BM + BN) * kBlk;
  __shared__ __align__(1024) uint8_t lds[2 * kStage];

  Tile t;
  if (!find_tile<BM, BN>(A, blockIdx.x, &t)) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int row = lane & 15, grp = lane >> 4;
  const int64_t kp = (int64_t)A.kb * kBlk;

  // loads: wave w brings rows 8 w .. 8 w + 7 of every kRowsPerLoad.  Addresses are a
  // uniform base and 32-bit offsets: from the tile's first row, or, for gathered rows,
  // from the first activation.
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
  auto load_stage = [&](int buf, int b) {
    uint8_t *base = lds + buf * kStage + wave * 1024;
#pragma unroll
    for (int i = 0; i < LM + LN; ++i) {
      const int off = i * kRowsPerLoad * kBlk;
      const uint8_t *from = (i < LM ? qb : wb) + (int64_t)b * kBlk;
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(from + src[i]),
                                       (__attribute__((address_space(3))) void *)(base + off), 16, 0, 0);
    }
  };

  uint32_t st[TM];
  const float *qsb = A.qs + (A.row_ids ? 0 : t.p0);
#pragma unroll
  for (int f = 0; f < TM; ++f) st[f] = (uint32_t)q_row((wm * TM + f) * 16 + row);
  const int nb = min((t.n0 + wn * TN * 16) / kBlk, (A.rows - 1) / kBlk);
  uint32_t zero = 0;
  asm volatile("v_mov_b32 %0, 0" : "=v"(zero));               // keeps the load below a vector load
  const float *ws = A.ws + ((int64_t)t.e * ((A.rows + kBlk - 1) / kBlk) + nb) * A.kb;

  f32x4_t acc[TN][TM] = {};
  float sx[TM], sw;
  load_stage(0, 0);
#pragma unroll
  for (int f = 0; f < TM; ++f) sx[f] = qsb[st[f]];
  sw = ws[zero];

  // a fragment's two chunks: g and g + 4 at the swizzled places of its row
  const int sz = (row >> 1) & 7;
  const int c0 = row * kBlk + ((grp ^ sz) << 4), c1 = row * kBlk + (((grp + 4) ^ sz) << 4);
  for (int b = 0; b < A.kb; ++b) {
    __syncthreads();                                           // waits for this block's loads too
    float s[TM];
#pragma unroll
    for (int f = 0; f < TM; ++f) s[f] = sx[f] * sw;
    if (b + 1 < A.kb) {
      load_stage((b + 1) & 1, b + 1);
      const float *next = qsb + (int64_t)(b + 1) * A.m;
#pragma unroll
      for (int f = 0; f < TM; ++f) sx[f] = next[st[f]];
      sw = (ws + b + 1)[zero];
    }
    const uint8_t *lq = lds + (b & 1) * kStage + wm * TM * 16 * kBlk;
    const uint8_t *lw = lds + (b & 1) * kStage + BM * kBlk + wn * TN * 16 * kBlk;
    auto frag = [&](const uint8_t *p, int i) {
      return join(*reinterpret_cast<const i32x4 *>(p + i * 16 * kBlk + c0),
                  *reinterpret_cast<const i32x4 *>(p + i * 16 * kBlk + c1));
    };
    if constexpr (kExact) {
      Halves qh[TM];
#pragma unroll
      for (int f = 0; f < TM; ++f) qh[f] = widen(frag(lq, f));
#pragma unroll
      for (int g = 0; g < TN; ++g) {
        const Halves wh = widen(frag(lw, g));
#pragma unroll
        for (int f = 0; f < TM; ++f) {
          const f32x4_t part = mma(wh, qh[f]);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[g][f][i] = fmaf(part[i], s[f], acc[g][f][i]);
        }
      }
      continue;
    }
    __builtin_amdgcn_sched_barrier(0);
    i32x8 qf[TM], wf[2];
    f32x4_t part[2][TM];
    wf[0] = frag(lw, 0);
#pragma unroll
    for (int f = 0; f < TM; ++f) qf[f] = frag(lq, f);
    // the products of row fragment g, while the sums of g - 1 are scaled and added
#pragma unroll
    for (int g = 0; g <= TN; ++g) {
      if (g + 1 < TN) wf[(g + 1) & 1] = frag(lw, g + 1);
#pragma unroll
      for (int f = 0; f < TM; ++f) {
        if (g < TN) part[g & 1][f] = mma(wf[g & 1], qf[f]);
        if (g > 0)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[g - 1][f][i] = fmaf(part[(g - 1) & 1][f][i], s[f], acc[g - 1][f][i]);
      }
    }
    // the order above, for the scheduler: reads ahead, then one product and four sums in turn
    __builtin_amdgcn_sched_group_barrier(0x100, 2 + 2 * TM, 0);
#pragma unroll
    for (int g = 0; g <= TN; ++g) {
      if (g + 1 < TN) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
      for (int f = 0; f < TM; ++f) {
        if (g < TN) __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        if (g > 0) __builtin_amdgcn_sched_group_barrier(0x2, 4, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int f = 0; f < TM; ++f) {
    const int p = t.p0 + (wm * TM + f) * 16 + row;
    if (p >= t.p1) continue;
#pragma unroll
    for (int g = 0; g < TN; ++g) store4(y, A, p, t.n0 + (wn * TN + g) * 16 + grp * 4, acc[g][f]);
  }
}

// ------------------------------------------------------------------ dispatch

// Workgroups that cover every tile whatever the offsets are: an expert's rows take
// at most one tile more than they fill.
int64_t tiles(const Fp8Args &A, int bm, int bn) {
  const int64_t nt = (A.rows + bn - 1) / bn;
  const int64_t mt = A.offsets ? A.slots / bm + (A.experts < A.slots ? A.experts : A.slots) : (A.m + bm - 1) / bm;
  return mt * nt;
}

template <typename Y, int MF, int NW, int kDepth>
hipError_t stream(const Fp8Args &A, Y *y, hipStream_t s) {
  fp8_stream_kernel<Y, MF, NW, kDepth><<<(unsigned)tiles(A, 16 * MF, 16), 64 * NW, 0, s>>>(A, y);
  return hipGetLastError();
}

template <typename Y, int BM, int BN, int WM, int WN, bool kExact>
hipError_t tile(const Fp8Args &A, Y *y, hipStream_t s) {
  fp8_tile_kernel<Y, BM, BN, WM, WN, kExact><<<(unsigned)tiles(A, BM, BN), 64 * WM * WN, 0, s>>>(A, y);
  return hipGetLastError();
}

template <typename Y>
hipError_t run(const Fp8Args &A, Y *y, int num_cus, hipStream_t s) {
  // rows a matrix has to multiply: exact for one matrix, the mean for experts
  const int per = A.offsets ? (A.slots + A.experts - 1) / A.experts : A.m;
  if (per <= 16) return A.kb >= 16 ? stream<Y, 1, 16, 2>(A, y, s) : stream<Y, 1, 4, 2>(A, y, s);
  if (per <= 32) return A.kb >= 16 ? stream<Y, 2, 16, 2>(A, y, s) : stream<Y, 2, 4, 2>(A, y, s);
  if (tiles(A, 256, 256) >= num_cus) return tile<Y, 256, 256, 4, 2, true>(A, y, s);
  if (tiles(A, 128, 128) >= num_cus) return tile<Y, 128, 128, 2, 2, true>(A, y, s);
  return tile<Y, 64, 64, 2, 2, true>(A, y, s);
}

hipError_t run_any(const Fp8Args &A, void *y, int ydtype, int num_cus, hipStream_t s) {
  if (ydtype == BQM_F32) return run(A, (float *)y, num_cus, s);
  if (ydtype == BQM_BF16) return run(A, (__bf16 *)y, num_cus, s);
  return run(A, (_Float16 *)y, num_cus, s);
}

}  // namespace

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
