// Attention over the paged 8-bit cache: many rows a sequence.
//
// Bound by arithmetic: 4 x 2048 rows of 8192 positions, 32 heads of 128 columns to 8: 1068 to 1117 us a call from one machine to
// another, 860 to 900 TFLOP/s.  The vector instructions (414 a wave and page: 128 conversions, 32 exponentials, and 64 that copy
// the sums to other registers and back, since the second product is written twice, in the common branch and in the rare one) are
// busy 69% of the time, the matrix instructions (32) 39%.  Each page also waits at its head for its number and its scales.
// Codes widened once a workgroup, to fp16 in LDS, took a fourth of the vector
// instructions away and 13% more time: twice the reads of LDS, whose latency two waves do not hide.
//
// Probabilities of 16-bit rows are one fp16 term: 2^-11 of each at most, of random sign, beside half a step of 2^-8 of a bf16
// result and 2^-11 of an fp16 one.  (Against 64 bits, 512 rows of 2048: bf16 results off by 1.665e-3 of them, 1.660e-3 with
// two terms; fp16 2.42e-4 and 2.08e-4.  Two terms take 30% more time: 1075 -> 1410 us.)
//
// Registers: 16 bits, 128 columns two waves a SIMD, with 8 registers spilled before the first page; 192 and 256 columns, and fp32
// from 96 on, one wave; 256 columns spill 94, 11 of which are read again every page.  4 x 2048 rows of 8192, us with
// 64 / 128 / 192 / 256 columns: bf16 712 / 1063 / 2425 / 4028, fp32 1143 / 2573 / 3620 / not here (6091 in tiles of 16).
//
// A tile is 128 queries of one key head, 32 a wave: the rows of a sequence times the heads
// that share the key head.  Pages go to LDS as codes, without passing through registers, into one of two buffers
// while the other is multiplied; every wave widens the codes it reads.  A wave holds its queries
// and sums in registers for all pages, so nothing is joined but the parts of long sequences with few tiles.
//
// The matrix instructions are 32 x 32 x 16.  A lane's 16 scores of a half page are tokens 16 (lane / 32) .. + 15 of it:
// row 8 b + 4 h + j of the first product is token 16 h + 4 b + j, which is what lane half h holds as operand of
// the second.
#include "kv_attention.h"

namespace bqm {
namespace attn {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kWaves = 4;

// 16-byte chunks of a key row in LDS (a power of two), and where chunk c of token t lies: 16 lanes that read one
// chunk of the tokens of a product's rows touch 16 different groups of four banks.
template <int kDp> constexpr int kRowChunks = kDp <= 32 ? 2 : kDp <= 64 ? 4 : kDp <= 128 ? 8 : 16;
template <int kDp>
__device__ __forceinline__ int key_swizzle(int t) {
  const int bits = (t & 7) | (t >> 1 & 8);                              // tokens of 16 rows differ in bits 0, 1, 2 and 4
  return bits / (16 / kRowChunks<kDp>);
}
__device__ __forceinline__ int value_swizzle(int d) { return d >> 2 & 3; }

template <typename T, int kDp>
__global__ __launch_bounds__(64 * kWaves, (kDp > 128 || kTermsOf<T> > 1) ? 1 : 2) void kv_tile_kernel(
    AttnArgs A, bool qvec, const T *__restrict__ q, T *__restrict__ out) {
  // The sums follow a row's maximum when it has grown by more than 2^kLag, or, with two terms, at once: some row of the
  // wave's 32 has a larger one in most pages, and to scale all sums takes a sixth of a page's time.
  constexpr float kLag = kTermsOf<T> == 1 ? 4.0f : 0.0f, kUpLag = kUp - kLag, kDown = kTermsOf<T> == 1 ? 0x1p-11f : 0x1p-15f;
  constexpr int kTerms = kTermsOf<T>, kSteps = kDp / 16, kCols = kDp / 32, kChunks = kRowChunks<kDp>;
  constexpr int kKeyBytes = kPage * kChunks * 16, kStage = kKeyBytes + kPage * kDp;
  constexpr int kLoads = kStage / 1024;                                  // of a wave's 64 lanes, 16 bytes each
  __shared__ __align__(1024) uint8_t lds[2 * kStage];

  const int bid = blockIdx.x, kh = bid % A.kv_heads, rep = A.rep;        // heads to the XCDs in turn: each reads its own
  KvSeq s;
  int job;
  const auto jobs = [rep](const KvSeq &x) { return (int)(((int64_t)x.n * rep + 127) / 128); };
  if (!kv_find(A.B, A.M, bid / A.kv_heads, jobs, &s, &job)) return;
  job = jobs(s) - 1 - job;                                               // the last rows see the most: they begin
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 31, hf = lane >> 5;
  const int all = s.n * rep, tile_last = min(all, job * 128 + 128) - 1;
  const int limit = kv_limit(A.B, s);
  int p0, p1;
  pages_of(A, s, s.first() + job * 128 / rep, s.first() + tile_last / rep, &p0, &p1);
  p0 += (int)blockIdx.y * A.chunk;
  p1 = min(p1, p0 + A.chunk);

  // the wave's queries; a wave past the last only loads
  const int c0 = job * 128 + wave * 32;
  const bool any = c0 <= tile_last;
  const int last_c = min(c0 + 31, tile_last), c = min(c0 + col, tile_last), i = c / rep, h = kh * rep + (c - i * rep);
  const int64_t row = s.lo + i, head = row * A.heads + h;
  const int pos = s.first() + i, first = s.first() + min(c0, tile_last) / rep, last = s.first() + last_c / rep;
  const int lo = A.window ? max(0, pos - A.window + 1) : 0, hi = min(pos + 1, limit);

  // A row's sums of values are in units of the scale of the last page that it sees, v_unit: pages' scales are powers of two
  // and mostly the same, and then the second product adds to them as they are.
  f32x16 o[kCols] = {};
  float m = -INFINITY, l = 0.0f, v_unit = 0.0f;
  if (p0 < p1) {
    // loads: load n of a stage brings 1 KiB, lane x the 16 bytes that go to slot 64 n + x
    auto load_page = [&](int to, int page) {
      const int64_t ph = (int64_t)page * A.kv_heads + kh;
      const uint8_t *kp = A.kc + ph * (kPage * kDp), *vp = A.vc + ph * (kPage * kDp);
#pragma unroll
      for (int n0 = 0; n0 < kLoads; n0 += kWaves) {
        const int n = n0 + wave;
        if (kLoads % kWaves && n >= kLoads) break;
        const uint8_t *from;
        if (n * 1024 < kKeyBytes) {
          const int slot = n * 64 + lane, t = slot / kChunks, ch = (slot % kChunks) ^ key_swizzle<kDp>(t);
          from = kp + t * kDp + (ch * 16 < kDp ? ch : 0) * 16;
        } else {
          const int slot = (n * 1024 - kKeyBytes) / 16 + lane, d = slot / 4, ch = (slot % 4) ^ value_swizzle(d);
          from = vp + d * kPage + ch * 16;
        }
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from, (lds_void *)(lds + to + n * 1024), 16, 0, 0);
      }
    };
    int page = kv_page(A.B, s, p0);
    if (page >= 0) load_page(0, page);

    f16x8 qf[kSteps][kTerms];
    float mul = 0.0f;
    int qe = 0;
    if (any) {
      const T *qr = q + row * A.qt + h * A.qh;
      uint32_t top = 0;
      float v[kSteps][8];
#pragma unroll
      for (int w = 0; w < kSteps; ++w) {
        load_q8(qr, (w / 2) * 32 + hf * 16 + (w & 1) * 8, A.dim, qvec, v[w]);
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[w][j]) & 0x7FFFFFFFu);
      }
      top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
      qe = top && top < 0x7F800000u ? __builtin_amdgcn_frexp_expf(__uint_as_float(top)) - 15 : 0;
      mul = top < 0x7F800000u ? fabsf(A.scale) : __builtin_nanf("");     // a row that is not finite is NaN
      const float sign = A.scale < 0.0f ? -1.0f : 1.0f;
#pragma unroll
      for (int w = 0; w < kSteps; ++w) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[w][j] = sign * ldexpf(v[w][j], -qe);
        to_terms<kTerms>(v[w], qf[w]);
      }
    }

    int at = 0;
    for (int pi = p0; pi < p1; ++pi, at ^= kStage) {
      const int64_t ph = (int64_t)max(page, 0) * A.kv_heads + kh;
      const float ks = A.ks[ph], vs = A.vs[ph];
      const bool there = page >= 0;
      page = pi + 1 < p1 ? kv_page(A.B, s, pi + 1) : -1;
      // this page has landed, and everyone is done with the one before
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      if (page >= 0) load_page(at ^ kStage, page);
      const int start = pi * kPage;
      if (!there || !any || start > last || (A.window && start + kPage <= first - A.window + 1)) continue;

      const uint8_t *kl = lds + at, *vl = lds + at + kKeyBytes;
      // Scores.  Fragments are read two ahead; left to itself the compiler reads all of them first and spills more.  The products
      // go before the other wave's softmax (4 x 2048 rows of 8192: 1180 us without, 1150 so).
      auto key = [&](int n) {                                            // fragment n: half page n / (kSteps / 2)
        // row 8 b + 4 h + j is token 16 h + 4 b + j
        const int tok = 32 * (n / (kSteps / 2)) + 16 * (col >> 2 & 1) + 4 * (col >> 3) + (col & 3);
        return *reinterpret_cast<const i32x4 *>(kl + (tok * kChunks + ((2 * (n % (kSteps / 2)) + hf) ^ key_swizzle<kDp>(tok))) * 16);
      };
      auto value = [&](int d, int t) {                                   // column 32 d + col, tokens 32 t + 16 hf .. + 15
        const int dd = d * 32 + col;
        return *reinterpret_cast<const i32x4 *>(vl + dd * kPage + (((2 * t + hf) ^ value_swizzle(dd)) << 4));
      };
      __builtin_amdgcn_s_setprio(1);
      f32x16 x[2] = {};
      i32x4 ahead[2] = {key(0), key(1)};
#pragma unroll
      for (int n = 0; n < kSteps; ++n) {
        const i32x4 kw = ahead[n & 1];
        if (n + 2 < kSteps) ahead[n & 1] = key(n + 2);
        __builtin_amdgcn_sched_barrier(0);
        const int t = n / (kSteps / 2), w = n % (kSteps / 2);
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          const f16x8 kf = widen(kw[2 * a], kw[2 * a + 1]);
#pragma unroll
          for (int z = 0; z < kTerms; ++z) x[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, qf[2 * w + a][z], x[t], 0, 0, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_setprio(0);
      const float f = ldexpf(mul * __builtin_amdgcn_frexp_mantf(ks), __builtin_amdgcn_frexp_expf(ks) + qe);
      const bool whole = start + kPage <= min(first + 1, limit) && (!A.window || start > last - A.window);
      uint32_t see = 0xFFFFFFFFu;                                        // bit 16 t + r: token start + 32 t + 16 hf + r
      if (!whole) {
        see = 0;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int j0 = start + 32 * t + 16 * hf, a = min(max(lo - j0, 0), 16), b = min(max(hi - j0, 0), 16);
          see |= (((1u << b) - 1u) & ~((1u << a) - 1u)) << (16 * t);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int r = 0; r < 16; ++r) x[t][r] = see >> (16 * t + r) & 1 ? x[t][r] : -INFINITY;
      }
      float top = -INFINITY;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, x[t][r]);
      top = halves_max(top);
      const float most = top > -INFINITY ? top * f : -INFINITY, m1 = fmaxf(m, most);
      if (__ballot(m1 - m > kLag)) {
        const float alpha = m1 > -INFINITY ? __builtin_amdgcn_exp2f(m - m1) : 0.0f;
        l *= alpha;
#pragma unroll
        for (int d = 0; d < kCols; ++d) o[d] *= alpha;
        m = m1;
      }
      // Past 2^20 steps of fp32 come near the largest probability's room in fp16: exponents are taken from the page's largest score
      // on, whatever its size.  (Always so: 1131 us for 4 x 2048 rows of 8192; in a branch of its own 1101, as without it.)
      float lead = kUpLag - (m > -INFINITY ? m : 0.0f);
      const bool large = fabsf(m1) >= 0x1p20f && m1 > -INFINITY;
      if (__builtin_expect(__ballot(large) != 0, 0)) {
        const float shift = large ? top : 0.0f;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int r = 0; r < 16; ++r) x[t][r] -= shift;
        lead = large ? (most - m) + kUpLag : lead;
      }
      f16x8 p[4][kTerms];
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        float e[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) e[r] = __builtin_amdgcn_exp2f(fmaf(x[a / 2][8 * (a & 1) + r], f, lead));
        if (!whole) {                                                    // also where -inf times f is no -inf
#pragma unroll
          for (int r = 0; r < 8; ++r) e[r] = see >> (8 * a + r) & 1 ? e[r] : 0.0f;
        }
        to_terms<kTerms>(e, p[a]);
        l = add_terms<kTerms>(p[a], l);
      }
      // What some row does not see may be NaN, and 0 times it would be too.
      int rare = 0;
      if (!whole) {
        bool bad = false;
#pragma unroll
        for (int d = 0; d < kCols; ++d)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const i32x4 vw = value(d, t);
#pragma unroll
            for (int w = 0; w < 4; ++w) bad |= has_nan(vw[w]);
          }
        rare = __ballot(bad) != 0;
      }
      // Another scale: the row's sums change to its units, exactly.  A page whose scale is outside [2^-40, 2^16] is summed apart
      // and added with its share of the nearer end.  From a scale of 2^16 on the units stay there.  Probabilities weigh up to 2^15
      // (2^11 above a maximum that lags by 2^4): where values times positions are below 2^128, as the caller sees to, sums in
      // units of 2^16 are below 2^127, and shares above 2^-142; else, after a step from 2^15 to 2^-40, below 448 x 2^15 x
      // 2^55 < 2^79 times the positions.
      constexpr float kLeast = 0x1p-40f, kMost = 0x1p16f;
      float share = 1.0f;
      if (top > -INFINITY && vs != v_unit) {
        const float unit = v_unit == kMost ? kMost : fminf(fmaxf(vs, kLeast), kMost);
        const float by = v_unit / unit;                                  // the first page's sums are of zeros
#pragma unroll
        for (int d = 0; d < kCols; ++d) o[d] *= by;
        v_unit = unit;
        share = vs / unit;
      }
      rare |= __ballot(share != 1.0f) != 0;
      if (__builtin_expect(!__builtin_amdgcn_readfirstlane(rare), 1)) {
        __builtin_amdgcn_s_setprio(1);
        i32x4 vn[2] = {value(0, 0), value(0, 1)};
#pragma unroll
        for (int d = 0; d < kCols; ++d) {
          const i32x4 now[2] = {vn[0], vn[1]};
          if (d + 1 < kCols) {
            vn[0] = value(d + 1, 0);
            vn[1] = value(d + 1, 1);
          }
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int a = 0; a < 2; ++a) {
              const f16x8 vf = widen(now[t][2 * a], now[t][2 * a + 1]);
#pragma unroll
              for (int z = 0; z < kTerms; ++z) o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, p[2 * t + a][z], o[d], 0, 0, 0);
            }
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
        // NaN codes are taken out, and the sums of the rows that see one made NaN
#pragma unroll
        for (int d = 0; d < kCols; ++d) {
          f32x16 part = {}, n = {};
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const i32x4 vw = value(d, t);
#pragma unroll
            for (int a = 0; a < 2; ++a) {
              f16x8 sees;
#pragma unroll
              for (int r = 0; r < 8; ++r) sees[r] = (_Float16)(see >> (16 * t + 8 * a + r) & 1 ? 1.0f : 0.0f);
              n = __builtin_amdgcn_mfma_f32_32x32x16_f16(widen(nan_ones(vw[2 * a]), nan_ones(vw[2 * a + 1])), sees, n, 0, 0, 0);
              const f16x8 vf = widen(without_nan(vw[2 * a]), without_nan(vw[2 * a + 1]));
#pragma unroll
              for (int z = 0; z < kTerms; ++z) part = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, p[2 * t + a][z], part, 0, 0, 0);
              __builtin_amdgcn_sched_barrier(0);
            }
          }
#pragma unroll
          for (int r = 0; r < 16; ++r) o[d][r] = n[r] != 0.0f ? __builtin_nanf("") : fmaf(part[r], share, o[d][r]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  }
  if (!any || c0 + col > tile_last) return;
  l = halves_sum(l);
  l *= kDown;
  if (A.splits > 1) {
    const int64_t at = head * A.splits + blockIdx.y;
    // sums and their weights 2^kLag smaller in every part, so that no probability weighs more than 1: sums near fp32's largest fit
    constexpr float kPart = kTermsOf<T> == 1 ? 0x1p-4f : 1.0f;
    if (hf == 0) A.ml[at] = float2{m, l * kPart};
    if (p0 >= p1) return;
    float *p = A.part + at * kDp;
#pragma unroll
    for (int d = 0; d < kCols; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[d][r] = o[d][r] * (kDown * kPart) * v_unit;
#pragma unroll
    for (int d = 0; d < kCols; ++d)
#pragma unroll
      for (int b = 0; b < 4; ++b)
        *reinterpret_cast<f32x4_t *>(p + d * 32 + 8 * b + 4 * hf) = f32x4_t{o[d][4 * b], o[d][4 * b + 1], o[d][4 * b + 2], o[d][4 * b + 3]};
    return;
  }
  const float by = l != 0.0f ? kDown / l : 0.0f;
  T *to = out + head * A.dim;
  typedef T tx4 __attribute__((ext_vector_type(4)));
  const bool four = (A.dim & 3) == 0 && ((uintptr_t)out & (4 * sizeof(T) - 1)) == 0;
#pragma unroll
  for (int d = 0; d < kCols; ++d)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int c1 = d * 32 + 8 * b + 4 * hf;
      T v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = from_sum<T>(o[d][4 * b + r] * by * v_unit);
      if (four && c1 < A.dim) {
        *reinterpret_cast<tx4 *>(to + c1) = tx4{v[0], v[1], v[2], v[3]};
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (c1 + r < A.dim) to[c1 + r] = v[r];
      }
    }
}

template <typename T, int kDp>
hipError_t start(const AttnArgs &A, bool qvec, const T *q, T *out, hipStream_t s) {
  kv_tile_kernel<T, kDp><<<dim3((unsigned)(A.M.groups * A.kv_heads), A.splits), 64 * kWaves, 0, s>>>(A, qvec, q, out);
  return hipGetLastError();
}

template <typename T>
hipError_t by_dim(const AttnArgs &A, bool vec, const void *q, void *out, hipStream_t s) {
  switch (kv_padded_dim(A.dim)) {
    case 32: return start<T, 32>(A, vec, (const T *)q, (T *)out, s);
    case 64: return start<T, 64>(A, vec, (const T *)q, (T *)out, s);
    case 96: return start<T, 96>(A, vec, (const T *)q, (T *)out, s);
    case 128: return start<T, 128>(A, vec, (const T *)q, (T *)out, s);
    case 192: return start<T, 192>(A, vec, (const T *)q, (T *)out, s);
    default:
      if constexpr (sizeof(T) == 2) return start<T, 256>(A, vec, (const T *)q, (T *)out, s);
      else return hipErrorInvalidValue;                                  // past kMostTileF32
  }
}

}  // namespace

hipError_t launch_tiles(const AttnArgs &A, bool vec, const void *q, int dtype, void *out, hipStream_t s) {
  if (dtype == BQM_F32) return by_dim<float>(A, vec, q, out, s);
  if (dtype == BQM_BF16) return by_dim<__bf16>(A, vec, q, out, s);
  return by_dim<_Float16>(A, vec, q, out, s);
}

}  // namespace attn
}  // namespace bqm
