// Appending to a paged K/V cache with the per-head RMSNorm and the NeoX
// rotation applied on the way, and reading cached rows back as values
// (include/qg.h, "Paged K/V cache", states both).
//
// Append. A CTA owns one block of 16 tokens of one sequence, the unit that
// shares a scale of an int8 page: whoever writes a row of it has to see all
// its new rows (for their maximum) and may have to bring the block's earlier
// rows to a larger scale. Its warps take (q, K or V; head) items, one warp
// for up to 8 new rows and two past that: a lane holds D/32 neighbouring
// values of each row in registers, so the norm's sum, the rotation's partner
// (D/2 away: another lane) and the block's maximum are warp shuffles, and
// each value is read once and written once. The cosines and sines of the
// block's tokens and the norms' weights are brought into shared memory once
// per CTA and serve all heads (the weights read for each head cost 4 of 36 us),
// while the first rows are under way.
//
// What bounds it: a few rows, the chain launch, lengths, table, rows, stores
// (32 sequences of one token, 16 + 2 x 8 heads of 128, with the read-back 6.4
// us); prompts, latency and issue, a lane's 8 rows in turn (16000 int8 rows of
// 8 users 90 us with the read-back, 3.6 TB/s).
//
// The mapping of CTAs to (sequence, block) needs no host knowledge of the
// lengths: n rows touch at most n/16 + 2 blocks, so slot ranges
// [row_start[b]/16 + 2b, row_start[b+1]/16 + 2(b+1)) are wide enough for
// every sequence and do not overlap.
#include "paged_kv.cuh"

#include "mma_sync.cuh"

#include <algorithm>
#include <cfloat>
#include <cmath>

namespace qg {
namespace pk {

constexpr int kWarps = 8;
constexpr int kMaxHalf = 128;  // rotated pairs of the widest head

struct AppendParams {
  uint8_t* kp;
  uint8_t* vp;
  float* ks;
  float* vs;
  const int32_t* table;
  const int32_t* kv_len;
  const int32_t* row_start;
  const uint8_t* q;
  const uint8_t* k;
  const uint8_t* v;
  long long q_ld, k_ld, v_ld;
  const uint16_t* qn;
  const uint16_t* kn;
  void* qo;
  int q_bf16;
  float eps;
  int half;  // rotated pairs
  int B, T, H, Hkv, page_size, max_pages, num_pages;
  double turns[kMaxHalf];  // angle of pair i at position 1, in units of pi
};

// EPL consecutive values of a row, fp32 or bf16, as they come from memory.
template <int EPL, bool XF32>
struct Raw {
  static constexpr int N = XF32 ? EPL : EPL / 2;
  uint32_t w[N];

  __device__ __forceinline__ void load(const uint8_t* p) {
    if constexpr (N == 1) {
      w[0] = __ldcg(reinterpret_cast<const uint32_t*>(p));
    } else if constexpr (N == 2) {
      const uint2 t = __ldcg(reinterpret_cast<const uint2*>(p));
      w[0] = t.x;
      w[1] = t.y;
    } else {
#pragma unroll
      for (int j = 0; j < N; j += 4) {
        const uint4 t = __ldcg(reinterpret_cast<const uint4*>(p) + j / 4);
        w[j] = t.x;
        w[j + 1] = t.y;
        w[j + 2] = t.z;
        w[j + 3] = t.w;
      }
    }
  }
  __device__ __forceinline__ void values(float (&x)[EPL]) const {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if constexpr (XF32) {
        x[j] = __uint_as_float(w[j]);
      } else {
        x[2 * j] = bf16_lo(w[j]);
        x[2 * j + 1] = bf16_hi(w[j]);
      }
    }
  }
};
template <int EPL>
__device__ __forceinline__ void store_bf16(uint16_t* p, const float (&x)[EPL]) {
  uint32_t w[EPL / 2];
#pragma unroll
  for (int j = 0; j < EPL / 2; ++j)
    w[j] = mm::pack_bf16(x[2 * j], x[2 * j + 1]);
  if constexpr (EPL == 2)
    *reinterpret_cast<uint32_t*>(p) = w[0];
  else if constexpr (EPL == 4)
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <int EPL>
__device__ __forceinline__ void store_f32(float* p, const float (&x)[EPL]) {
  if constexpr (EPL == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
  } else {
#pragma unroll
    for (int j = 0; j < EPL; j += 4)
      *reinterpret_cast<float4*>(p + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
  }
}

// EPL int8 codes as packed words (the last half unused for EPL = 2).
template <int EPL>
__device__ __forceinline__ void load_codes(const uint8_t* p, int (&c)[EPL]) {
  uint32_t w[2] = {0, 0};
  if constexpr (EPL == 2)
    w[0] = __ldcg(reinterpret_cast<const uint16_t*>(p));
  else if constexpr (EPL == 4)
    w[0] = __ldcg(reinterpret_cast<const uint32_t*>(p));
  else {
    const uint2 t = __ldcg(reinterpret_cast<const uint2*>(p));
    w[0] = t.x;
    w[1] = t.y;
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) c[j] = (int)(int8_t)(w[j >> 2] >> (8 * (j & 3)));
}

// The sum with 1.5 * 2^23 rounds a value to the nearest integer, ties to even;
// its low byte is the code.
__device__ __forceinline__ float rounded(float y) { return __fadd_rn(y, 12582912.f); }

// EPL codes rint(y) (y times the scales' ratio, rounded to fp32).
template <int EPL>
__device__ __forceinline__ void times_codes(const float (&y)[EPL], float ratio,
                                            uint32_t (&c)[EPL]) {
#pragma unroll
  for (int j = 0; j < EPL; ++j) c[j] = __float_as_uint(rounded(__fmul_rn(y[j], ratio)));
}
// EPL codes rint(x / s), the quotient rounded to fp32. |x| <= 127 s but for
// roundings, so nothing is clamped. below and above are 1 / s times 1 -+ 2^-22:
// with u = 2^-24, |x| above >= |x / s| (1 + 4u) (1 - u)^2 > |x / s| (1 + u), so the
// rounded quotient lies between x below and x above, and where these round to one
// integer it is the code. Only else, next to a tie, a value is divided (4099 int8
// prompt rows: 31.2 us with x * (1 / s), 34.7 with a division for each value, 32.4
// so). below = above = 0 (scale 0) gives 0; under a NaN scale any code.
template <int EPL>
__device__ __forceinline__ void quotient_codes(const float (&x)[EPL], float s, float below,
                                               float above, uint32_t (&c)[EPL]) {
  uint32_t tie = 0;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    c[j] = __float_as_uint(fmaf(x[j], below, 12582912.f));
    tie |= c[j] ^ __float_as_uint(fmaf(x[j], above, 12582912.f));
  }
  if (tie) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) c[j] = __float_as_uint(rounded(__fdiv_rn(x[j], s)));
  }
}
template <int EPL>
__device__ __forceinline__ void store_codes(uint8_t* p, const uint32_t (&c)[EPL]) {
  if constexpr (EPL == 2) {
    *reinterpret_cast<uint16_t*>(p) = (uint16_t)__byte_perm(c[0], c[1], 0x40);
  } else {
    uint32_t w[EPL / 4];
#pragma unroll
    for (int j = 0; j < EPL; j += 4)
      w[j / 4] = __byte_perm(__byte_perm(c[j], c[j + 1], 0x40), __byte_perm(c[j + 2], c[j + 3], 0x40),
                             0x5410);
    if constexpr (EPL == 4)
      *reinterpret_cast<uint32_t*>(p) = w[0];
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}

// EPL consecutive floats of shared memory.
template <int EPL>
__device__ __forceinline__ void lds(const float* p, float (&x)[EPL]) {
  if constexpr (EPL == 2) {
    const float2 t = *reinterpret_cast<const float2*>(p);
    x[0] = t.x;
    x[1] = t.y;
  } else {
#pragma unroll
    for (int j = 0; j < EPL; j += 4) {
      const float4 t = *reinterpret_cast<const float4*>(p + j);
      x[j] = t.x;
      x[j + 1] = t.y;
      x[j + 2] = t.z;
      x[j + 3] = t.w;
    }
  }
}

// RMSNorm of NR rows of one head across the warp (as qg_rmsnorm_perhead).
// For 8 rows the sums are scattered while they are reduced: after three
// exchanges a lane holds one row's (row lane / 4), so that its root and
// reciprocal are formed once, not on every lane, and 9 shuffles replace 40.
template <int D, int NR>
__device__ __forceinline__ void norm_rows(float (&x)[NR][D / 32], const float* w, float eps,
                                          int lane) {
  constexpr int EPL = D / 32;
  float nw[EPL], ss[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    ss[r] = 0.f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) ss[r] = fmaf(x[r][j], x[r][j], ss[r]);
  }
#pragma unroll
  for (int n = NR / 2, o = 16; n > 0; n >>= 1, o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int r = 0; r < n; ++r) {
      const float mine = up ? ss[n + r] : ss[r], other = up ? ss[r] : ss[n + r];
      ss[r] = mine + __shfl_xor_sync(0xffffffffu, other, o);
    }
  }
#pragma unroll
  for (int o = 16 / NR; o > 0; o >>= 1) ss[0] += __shfl_xor_sync(0xffffffffu, ss[0], o);
  const float inv = 1.0f / sqrtf(ss[0] / (float)D + eps);
  lds<EPL>(w + lane * EPL, nw);
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const float f = __shfl_sync(0xffffffffu, inv, r * (32 / NR));
#pragma unroll
    for (int j = 0; j < EPL; ++j) x[r][j] = x[r][j] * f * nw[j];
  }
}

// Rotation of NR rows of one head: dim d < half pairs with d + half, which
// the lane `half / EPL` further holds at the same place (half is a multiple
// of EPL). cs, sn: the rows' cosines and sines, `half` a row.
template <int D, int NR>
__device__ __forceinline__ void rotate_rows(float (&x)[NR][D / 32], const float* cs,
                                            const float* sn, int half, int lane) {
  constexpr int EPL = D / 32;
  const int hl = half / EPL;  // lanes per half
  const bool lo = lane < hl, hi = !lo && lane < 2 * hl;
  const int src = lo ? lane + hl : hi ? lane - hl : lane;
  const int i0 = (lo ? lane : hi ? lane - hl : 0) * EPL;
  const float sign = lo ? -1.f : 1.f;
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    float c[EPL], s[EPL];
    lds<EPL>(cs + r * half + i0, c);
    lds<EPL>(sn + r * half + i0, s);
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const float t = __shfl_sync(0xffffffffu, x[r][j], src) * s[j];
      const float y = fmaf(sign, t, x[r][j] * c[j]);
      if (lo || hi) x[r][j] = y;
    }
  }
}

template <int D, int NR>
__device__ __forceinline__ void put_query(const AppendParams& P, const float (&x)[NR][D / 32],
                                          int rows, long long at) {
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    if (r >= rows) break;
    if (P.q_bf16)
      store_bf16<D / 32>(reinterpret_cast<uint16_t*>(P.qo) + at + (long long)r * P.H * D, x[r]);
    else
      store_f32<D / 32>(reinterpret_cast<float*>(P.qo) + at + (long long)r * P.H * D, x[r]);
  }
}

// K or V rows of one head into a page. int8: `o` rows of the block lie before
// the block's new ones; `pair`: another warp has the block's other new rows
// (the block's maximum meets in smax, barrier `bar`).
template <int D, bool I8, int NR>
__device__ __forceinline__ void put_cache(const float (&x)[NR][D / 32], int rows, uint8_t* block,
                                          int first, float* scale, int o, bool pair, int half,
                                          unsigned* smax, int bar, int lane) {
  constexpr int EPL = D / 32;
  if constexpr (!I8) {
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      if (r >= rows) break;
      store_bf16<EPL>(reinterpret_cast<uint16_t*>(block) + (first + r) * D, x[r]);
    }
  } else {
    const float s_old = o > 0 ? __ldcg(scale) : 0.f;
    // the largest |x| by its bits, where infinities and NaN stand above all
    unsigned top = 0;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      unsigned m = 0;
#pragma unroll
      for (int j = 0; j < EPL; ++j) m = max(m, __float_as_uint(x[r][j]) & 0x7FFFFFFFu);
      top = max(top, r < rows ? m : 0u);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (pair) {
      if (lane == 0) smax[half] = top;
      asm volatile("bar.sync %0, 64;" ::"r"(bar) : "memory");
      top = max(smax[0], smax[1]);
      asm volatile("bar.sync %0, 64;" ::"r"(bar) : "memory");  // smax is used again
    }
    float s = fmaxf(s_old, __uint_as_float(top) / 127.0f);
    if (top >= 0x7F800000u || s_old != s_old) s = __int_as_float(0x7FC00000);
    if (s < FLT_MIN) s = 0.f;
    const float inv = s > 0.f ? 1.f / s : 0.f;  // (false for a NaN scale)
    const float below = inv * (1.f - 0x1p-22f), above = inv * (1.f + 0x1p-22f);
    if (half == 0 && o > 0 && s != s_old) {  // the block's earlier rows to the new scale
      const float ratio = s > 0.f ? s_old / s : 0.f;
      for (int r = 0; r < o; ++r) {
        int c[EPL];
        load_codes<EPL>(block + r * D + lane * EPL, c);
        float y[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) y[j] = (float)c[j];
        uint32_t w[EPL];
        times_codes<EPL>(y, ratio, w);
        store_codes<EPL>(block + r * D + lane * EPL, w);
      }
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      if (r >= rows) break;
      uint32_t w[EPL];
      quotient_codes<EPL>(x[r], s, below, above, w);
      store_codes<EPL>(block + (first + r) * D + lane * EPL, w);
    }
    if (half == 0) {
      __syncwarp();  // every lane has read s_old
      if (lane == 0) *scale = s;
    }
  }
}

// A CTA's block of 16 tokens: its new rows, lo .. lo + nr - 1 of the sequence
// (packed rows from `row`), the o rows of the block before them, its page.
struct NewRows {
  int first, lo, nr, o, page;
  long long row;
};

// The (q, K or V; head) items of a block, up to NR rows of a head a warp.
template <int D, bool I8, bool XF32, int NR>
__device__ __forceinline__ void append_rows(const AppendParams& P, const NewRows& B, float* cs,
                                            float* sn, float* norms, unsigned* smax) {
  constexpr int EPL = D / 32, XB = XF32 ? 4 : 2;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // past NR rows two neighbouring warps share the head's block
  const bool pair = B.nr > NR;
  const int half = pair ? warp & 1 : 0, base = half * NR, rows = min(NR, B.nr - base);
  const int items = 2 * P.Hkv + P.H, step = pair ? kWarps / 2 : kWarps;
  Raw<EPL, XF32> raw[NR];
  const auto fetch = [&](int it) {
    const bool isk = it < P.Hkv, isv = !isk && it < 2 * P.Hkv;
    const int h = isk ? it : isv ? it - P.Hkv : it - 2 * P.Hkv;
    const long long ld = isk ? P.k_ld : isv ? P.v_ld : P.q_ld;
    const uint8_t* const p =
        (isk ? P.k : isv ? P.v : P.q) + ((B.row + base) * ld + h * D + lane * EPL) * XB;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
#pragma unroll
      for (int j = 0; j < Raw<EPL, XF32>::N; ++j) raw[r].w[j] = 0;
      if (r < rows) raw[r].load(p + r * ld * XB);
    }
  };
  int it = blockIdx.y * step + (pair ? warp >> 1 : warp);
  if (it < items) fetch(it);  // under way while the angles are formed

  // cosines and sines of the new rows: the angle pos * theta^(-2i/rd) in units
  // of pi and its reduction to [-1, 1] in float64 (positions in the millions
  // keep the full fp32 accuracy), sincospi in fp32: within 2^-22 of the
  // exact values, at a fraction of the cost of a float64 sincos. A thread
  // keeps its pair, whose angle it reads once (each lane another one, which the
  // constant cache gives in turn).
  if (P.half) {
    const int f = tid % P.half, every = kWarps * 32 / P.half;
    const double turn = P.turns[f];
    for (int r = tid / P.half; r < B.nr && tid < every * P.half; r += every) {
      const double t = (double)(B.lo + r) * turn;
      sincospif((float)(t - 2.0 * rint(0.5 * t)), &sn[r * P.half + f], &cs[r * P.half + f]);
    }
  }
  for (int i = tid; i < 2 * D; i += kWarps * 32) {  // K's norm weights, then q's
    const uint16_t* const w = i < D ? P.kn : P.qn;
    if (w) norms[i] = bf16_bits_to_f32(__ldcg(w + i % D));
  }
  __syncthreads();

  const auto put = [&](const float (&x)[NR][EPL], bool isk, int h) {
    const long long hp = (long long)B.page * P.Hkv + h;
    const int in_page = B.first % P.page_size;
    uint8_t* block = (isk ? P.kp : P.vp) + (hp * P.page_size + in_page) * D * (I8 ? 1 : 2) +
                     (I8 ? 0 : lane * EPL * 2);
    float* scale =
        I8 ? (isk ? P.ks : P.vs) + hp * (P.page_size / kBlock) + in_page / kBlock : nullptr;
    put_cache<D, I8, NR>(x, rows, block, B.o + base, scale, B.o, pair, half, smax + (warp & ~1),
                         1 + (warp >> 1), lane);
  };
  // the next item's rows are under way while this one's are put away, where
  // registers hold both
  constexpr bool kAhead = NR == 1 || !XF32;
  for (; it < items; it += gridDim.y * step) {
    const bool isk = it < P.Hkv, isv = !isk && it < 2 * P.Hkv;
    const int h = isk ? it : isv ? it - P.Hkv : it - 2 * P.Hkv;
    float x[NR][EPL];
#pragma unroll
    for (int r = 0; r < NR; ++r) raw[r].values(x[r]);
    if (!isv && (isk ? P.kn : P.qn)) norm_rows<D, NR>(x, isk ? norms : norms + D, P.eps, lane);
    if (!isv && P.half) rotate_rows<D, NR>(x, cs + base * P.half, sn + base * P.half, P.half, lane);
    // (q_out may be q: every lane has the values of this item's rows, and the
    // next item's are another head's)
    __syncwarp();
    const int next = it + gridDim.y * step;
    if (kAhead && next < items) fetch(next);
    if (!isk && !isv)
      put_query<D, NR>(P, x, rows, (B.row + base) * P.H * D + h * D + lane * EPL);
    else if (B.page >= 0 && B.page < P.num_pages)
      put(x, isk, h);
    if (!kAhead && next < items) fetch(next);
  }
}

// CTAs an SM: bf16 rows of 128 take 80 registers with the next item's rows
// ahead (us with three CTAs so, three without, four: 16000 int8 rows of 8 users
// 90, 99, 121; 4099 rows 31.6, 32.4, 35.2; 600 rows 11.9, 12.0, 13.6); fp32 rows
// are a little faster as four at 64 (4099 rows 39.6 against 40.2).
constexpr int append_ctas(int D, bool xf32) { return D > 128 ? 2 : xf32 ? 4 : 3; }

template <int D, bool I8, bool XF32>
__global__ void __launch_bounds__(kWarps * 32, append_ctas(D, XF32))
append_kernel(const __grid_constant__ AppendParams P) {
  __shared__ __align__(16) float cs[kBlock * D / 2];
  __shared__ __align__(16) float sn[kBlock * D / 2];
  __shared__ __align__(16) float norms[2 * D];
  __shared__ unsigned smax[kWarps];
  __shared__ int s_b, s_r0, s_n, s_len;
  const int tid = threadIdx.x;
  pdl_wait();

  // the sequence whose slot range holds this CTA's slot
  const int u = blockIdx.x;
  int b = u, r0 = u, n = 1, len;
  if (P.row_start) {
    int found = 0;
    for (int i = tid; i < P.B; i += kWarps * 32) {
      const int from = row_begin(P.row_start, i, P.T), to = row_begin(P.row_start, i + 1, P.T);
      const int cached = __ldcg(P.kv_len + i);
      if (u >= from / kBlock + 2 * i && u < to / kBlock + 2 * (i + 1)) {
        found = 1;
        s_b = i;
        s_r0 = from;
        s_n = to - from;
        s_len = cached;
      }
    }
    // (two threads with a sequence: row starts that decrease, and what they
    // stored is a mix of both; the block is dropped)
    if (__syncthreads_count(found) != 1) return;
    b = s_b;
    r0 = s_r0;
    n = s_n;
    len = s_len;
  } else {
    len = __ldcg(P.kv_len + b);
  }
  if (n < 1 || len < n || len > P.max_pages * P.page_size) return;
  const int p0 = len - n;
  NewRows B;
  B.first = (p0 / kBlock + (P.row_start ? u - (r0 / kBlock + 2 * b) : 0)) * kBlock;
  if (B.first >= len) return;
  B.lo = max(p0, B.first);
  B.nr = min(len, B.first + kBlock) - B.lo;
  B.o = B.lo - B.first;
  B.row = r0 + (B.lo - p0);
  B.page = __ldcg(P.table + (long long)b * P.max_pages + B.first / P.page_size);
  if (B.nr == 1)
    append_rows<D, I8, XF32, 1>(P, B, cs, sn, norms, smax);
  else
    append_rows<D, I8, XF32, 8>(P, B, cs, sn, norms, smax);
}

struct GatherParams {
  const uint8_t* kp;
  const uint8_t* vp;
  const float* ks;
  const float* vs;
  const int32_t* table;
  const int32_t* first;
  const int32_t* row_start;
  void* ko;
  void* vo;
  int out_bf16;
  int B, T, Hkv, page_size, max_pages, num_pages;
};

// A CTA reads kGatherRows rows, a warp finding the page of each; a thread takes
// 8 neighbouring values of K or V, the same place in each row, so that its
// loads go out together.
constexpr int kGatherRows = kWarps;

template <int D, bool I8>
__global__ void __launch_bounds__(kWarps * 32) gather_kernel(const GatherParams P) {
  __shared__ int s_page[kGatherRows], s_off[kGatherRows];  // page -1: NaN, -2: no row
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  const int row0 = blockIdx.x * kGatherRows;
  {  // a warp finds a row's sequence and page
    const int row = row0 + warp;
    int b = row < P.T ? row : -1, from = row, first = 0;
    if (P.row_start) {
      b = -1;
      for (int i0 = 0; i0 < P.B && b < 0; i0 += 32) {
        const int i = i0 + lane;
        const int lo = i < P.B ? row_begin(P.row_start, i, P.T) : P.T;
        const int hi = i < P.B ? row_begin(P.row_start, i + 1, P.T) : 0;
        const int at = P.first && i < P.B ? __ldcg(P.first + i) : 0;
        const unsigned m = __ballot_sync(0xffffffffu, row < P.T && lo <= row && row < hi);
        if (m) {
          const int l = __ffs(m) - 1;
          b = i0 + l;
          from = __shfl_sync(0xffffffffu, lo, l);
          first = __shfl_sync(0xffffffffu, at, l);
        }
      }
    } else if (P.first && b >= 0) {
      first = __ldcg(P.first + b);
    }
    if (lane == 0) {
      int page = -2, off = 0;
      if (b >= 0) {
        const long long t = (long long)first + (row - from);
        page = -1;
        if (t >= 0 && t < (long long)P.max_pages * P.page_size) {
          const int pi = (int)t / P.page_size;
          off = (int)t - pi * P.page_size;
          page = __ldcg(P.table + (long long)b * P.max_pages + pi);
          if (page < 0 || page >= P.num_pages) page = -1;
        }
      }
      s_page[warp] = page;
      s_off[warp] = off;
    }
  }
  __syncthreads();
  const int half = P.Hkv * (D / 8);  // places per row of K, then as many of V
  for (int i = tid; i < 2 * half; i += kWarps * 32) {
    const bool isv = i >= half;
    const int at = isv ? i - half : i, h = at / (D / 8), d = at % (D / 8) * 8;
    void* out = isv ? P.vo : P.ko;
    if (!out) continue;
    const uint8_t* pages = isv ? P.vp : P.kp;
    const float* scales = isv ? P.vs : P.ks;
    Raw<I8 ? 4 : 8, false> raw[kGatherRows];  // 8 codes or values
    float scale[kGatherRows];
#pragma unroll
    for (int r = 0; r < kGatherRows; ++r) {
      const int page = s_page[r];
      scale[r] = __int_as_float(0x7FC00000);
#pragma unroll
      for (int j = 0; j < (I8 ? 2 : 4); ++j) raw[r].w[j] = I8 ? 0 : 0x7FC07FC0u;
      if (page < 0) continue;
      const long long hp = (long long)page * P.Hkv + h;
      raw[r].load(pages + ((hp * P.page_size + s_off[r]) * D + d) * (I8 ? 1 : 2));
      if (I8) scale[r] = __ldcg(scales + hp * (P.page_size / kBlock) + s_off[r] / kBlock);
    }
#pragma unroll
    for (int r = 0; r < kGatherRows; ++r) {
      if (s_page[r] == -2) continue;
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t w = raw[r].w[I8 ? j / 4 : j / 2];
        if constexpr (I8)
          x[j] = (float)(int8_t)(w >> (8 * (j & 3))) * scale[r];
        else
          x[j] = j & 1 ? bf16_hi(w) : bf16_lo(w);
      }
      const long long to = ((long long)(row0 + r) * P.Hkv + h) * D + d;
      if (P.out_bf16)
        store_bf16<8>(reinterpret_cast<uint16_t*>(out) + to, x);
      else
        store_f32<8>(reinterpret_cast<float*>(out) + to, x);
    }
  }
}

// Angles of the rotated pairs at position 1 in units of pi. A decode loop asks
// for the same ones each call, and 64 powers are 4 us of host time: the
// calling thread's last set is kept.
static void turns(double theta, int rotary_dim, double* out) {
  static thread_local double last_theta = 0.0, last[kMaxHalf];
  static thread_local int last_dim = -1;
  const int half = rotary_dim / 2;
  if (rotary_dim != last_dim || theta != last_theta) {
    for (int i = 0; i < half; ++i)
      last[i] = pow(theta, -2.0 * i / rotary_dim) / 3.14159265358979323846;
    last_theta = theta;
    last_dim = rotary_dim;
  }
  for (int i = 0; i < half; ++i) out[i] = last[i];
}

template <int D, bool I8>
cudaError_t launch_append(const AppendParams& P, bool xf32, dim3 grid, cudaStream_t st) {
  if (xf32)
    return launch_pdl(append_kernel<D, I8, true>, grid, dim3(kWarps * 32), 0, st, true, P);
  return launch_pdl(append_kernel<D, I8, false>, grid, dim3(kWarps * 32), 0, st, true, P);
}

template <int D>
cudaError_t launch_append(const AppendParams& P, bool i8, bool xf32, dim3 grid, cudaStream_t st) {
  return i8 ? launch_append<D, true>(P, xf32, grid, st) : launch_append<D, false>(P, xf32, grid, st);
}

template <int D>
cudaError_t launch_gather(const GatherParams& P, bool i8, dim3 grid, cudaStream_t st) {
  if (i8) return launch_pdl(gather_kernel<D, true>, grid, dim3(kWarps * 32), 0, st, true, P);
  return launch_pdl(gather_kernel<D, false>, grid, dim3(kWarps * 32), 0, st, true, P);
}

}  // namespace pk
}  // namespace qg

using namespace qg;

extern "C" qg_status qg_paged_kv_append(const qg_paged_kv* kv, const int32_t* page_table,
                                        int max_pages, const int32_t* kv_len,
                                        const int32_t* row_start, const void* q, long long q_ld,
                                        const void* k, long long k_ld, const void* v,
                                        long long v_ld, qg_dtype x_dtype, const uint16_t* q_norm,
                                        const uint16_t* k_norm, float eps, double theta,
                                        int rotary_dim, void* q_out, qg_dtype q_out_dtype, int B,
                                        int T, int H, void* stream) {
  clear_error();
  const char* who = "qg_paged_kv_append";
  if (qg_status s = pk::check_pool(who, kv, max_pages)) return s;
  const int D = kv->head_dim, Hkv = kv->kv_heads;
  QG_REQUIRE(B >= 0 && T >= 0 && H >= 0 && H <= 8192, QG_ERR_UNSUPPORTED_SHAPE,
             "%s: B=%d T=%d H=%d", who, B, T, H);
  QG_REQUIRE(B <= (1 << 16) && T <= (1 << 28), QG_ERR_UNSUPPORTED_SHAPE, "%s: B=%d T=%d too large",
             who, B, T);
  QG_REQUIRE(row_start || T == B, QG_ERR_UNSUPPORTED_SHAPE,
             "%s: T=%d rows without row_start must be B=%d", who, T, B);
  QG_REQUIRE((x_dtype == QG_F32 || x_dtype == QG_BF16) &&
                 (q_out_dtype == QG_F32 || q_out_dtype == QG_BF16),
             QG_ERR_INVALID_ARGUMENT, "%s: x_dtype=%d q_out_dtype=%d", who, (int)x_dtype,
             (int)q_out_dtype);
  QG_REQUIRE(rotary_dim >= 0 && rotary_dim <= D && rotary_dim % (D / 16) == 0,
             QG_ERR_UNSUPPORTED_SHAPE,
             "%s: rotary_dim=%d must be a multiple of %d in [0, head_dim=%d]", who, rotary_dim,
             D / 16, D);
  QG_REQUIRE(rotary_dim == 0 || theta > 0.0, QG_ERR_INVALID_ARGUMENT, "%s: theta=%g must be > 0",
             who, theta);
  if (B == 0 || T == 0) return QG_OK;
  if (qg_status s = pk::check_pool_pointers(who, kv)) return s;
  QG_REQUIRE(page_table && kv_len && k && v, QG_ERR_INVALID_ARGUMENT,
             "%s: null page_table, kv_len, k or v", who);
  QG_REQUIRE(H == 0 || (q && q_out), QG_ERR_INVALID_ARGUMENT, "%s: null q or q_out with H=%d", who,
             H);
  const int xb = x_dtype == QG_F32 ? 4 : 2;
  QG_REQUIRE(k_ld >= (long long)Hkv * D && v_ld >= (long long)Hkv * D &&
                 (H == 0 || q_ld >= (long long)H * D),
             QG_ERR_UNSUPPORTED_SHAPE, "%s: q_ld=%lld k_ld=%lld v_ld=%lld shorter than a row", who,
             q_ld, k_ld, v_ld);
  QG_REQUIRE(k_ld < (1LL << 40) && v_ld < (1LL << 40) && (H == 0 || q_ld < (1LL << 40)),
             QG_ERR_UNSUPPORTED_SHAPE, "%s: row stride too large", who);
  QG_REQUIRE(aligned(k, 16) && aligned(v, 16) && k_ld * xb % 16 == 0 && v_ld * xb % 16 == 0,
             QG_ERR_MISALIGNED, "%s: rows of k or v do not start on 16 bytes", who);
  QG_REQUIRE(H == 0 || (aligned(q, 16) && aligned(q_out, 16) && q_ld * xb % 16 == 0),
             QG_ERR_MISALIGNED, "%s: rows of q or q_out do not start on 16 bytes", who);
  QG_REQUIRE(aligned(page_table, 4) && aligned(kv_len, 4) && aligned(row_start, 4) &&
                 aligned(q_norm, 2) && aligned(k_norm, 2),
             QG_ERR_MISALIGNED, "%s: page_table, kv_len, row_start or a norm weight misaligned",
             who);
  pk::AppendParams P = {};
  P.kp = reinterpret_cast<uint8_t*>(kv->k_pages);
  P.vp = reinterpret_cast<uint8_t*>(kv->v_pages);
  P.ks = kv->k_scales;
  P.vs = kv->v_scales;
  P.table = page_table;
  P.kv_len = kv_len;
  P.row_start = row_start;
  P.q = reinterpret_cast<const uint8_t*>(q);
  P.k = reinterpret_cast<const uint8_t*>(k);
  P.v = reinterpret_cast<const uint8_t*>(v);
  P.q_ld = q_ld;
  P.k_ld = k_ld;
  P.v_ld = v_ld;
  P.qn = q_norm;
  P.kn = k_norm;
  P.qo = q_out;
  P.q_bf16 = q_out_dtype == QG_BF16;
  P.eps = eps;
  P.half = rotary_dim / 2;
  P.B = B;
  P.T = T;
  P.H = H;
  P.Hkv = Hkv;
  P.page_size = kv->page_size;
  P.max_pages = max_pages;
  P.num_pages = kv->num_pages;
  pk::turns(theta, rotary_dim, P.turns);
  const int slots = row_start ? T / pk::kBlock + 2 * B : B;
  // heads spread over CTAs until the grid fills the GPU four times (CTAs that
  // resident SMs hold) or each warp has one item
  const int most = (2 * Hkv + H + pk::kWarps - 1) / pk::kWarps;
  const int ny = std::max(1, std::min(most, 4 * num_sms() / std::max(slots, 1)));
  const dim3 grid(slots, ny);
  const bool i8 = kv->dtype == QG_KV_INT8, xf32 = x_dtype == QG_F32;
  cudaStream_t st = (cudaStream_t)stream;
  if (D == 64)
    pk::launch_append<64>(P, i8, xf32, grid, st);
  else if (D == 128)
    pk::launch_append<128>(P, i8, xf32, grid, st);
  else
    pk::launch_append<256>(P, i8, xf32, grid, st);
  return check_launch(who);
}

extern "C" qg_status qg_paged_kv_gather(const qg_paged_kv* kv, const int32_t* page_table,
                                        int max_pages, const int32_t* first,
                                        const int32_t* row_start, void* k_out, void* v_out,
                                        qg_dtype out_dtype, int B, int T, void* stream) {
  clear_error();
  const char* who = "qg_paged_kv_gather";
  if (qg_status s = pk::check_pool(who, kv, max_pages)) return s;
  QG_REQUIRE(B >= 0 && T >= 0 && B <= (1 << 16) && T <= (1 << 28), QG_ERR_UNSUPPORTED_SHAPE,
             "%s: B=%d T=%d", who, B, T);
  QG_REQUIRE(row_start || T == B, QG_ERR_UNSUPPORTED_SHAPE,
             "%s: T=%d rows without row_start must be B=%d", who, T, B);
  QG_REQUIRE(out_dtype == QG_F32 || out_dtype == QG_BF16, QG_ERR_INVALID_ARGUMENT,
             "%s: out_dtype=%d", who, (int)out_dtype);
  if (B == 0 || T == 0 || (!k_out && !v_out)) return QG_OK;
  if (qg_status s = pk::check_pool_pointers(who, kv)) return s;
  QG_REQUIRE(page_table, QG_ERR_INVALID_ARGUMENT, "%s: null page_table", who);
  QG_REQUIRE(aligned(k_out, 16) && aligned(v_out, 16), QG_ERR_MISALIGNED,
             "%s: k_out or v_out not 16-byte aligned", who);
  QG_REQUIRE(aligned(page_table, 4) && aligned(first, 4) && aligned(row_start, 4),
             QG_ERR_MISALIGNED, "%s: page_table, first or row_start misaligned", who);
  pk::GatherParams P = {};
  P.kp = reinterpret_cast<const uint8_t*>(kv->k_pages);
  P.vp = reinterpret_cast<const uint8_t*>(kv->v_pages);
  P.ks = kv->k_scales;
  P.vs = kv->v_scales;
  P.table = page_table;
  P.first = first;
  P.row_start = row_start;
  P.ko = k_out;
  P.vo = v_out;
  P.out_bf16 = out_dtype == QG_BF16;
  P.B = B;
  P.T = T;
  P.Hkv = kv->kv_heads;
  P.page_size = kv->page_size;
  P.max_pages = max_pages;
  P.num_pages = kv->num_pages;
  const dim3 grid((unsigned)((T + pk::kGatherRows - 1) / pk::kGatherRows));
  const bool i8 = kv->dtype == QG_KV_INT8;
  cudaStream_t st = (cudaStream_t)stream;
  if (kv->head_dim == 64)
    pk::launch_gather<64>(P, i8, grid, st);
  else if (kv->head_dim == 128)
    pk::launch_gather<128>(P, i8, grid, st);
  else
    pk::launch_gather<256>(P, i8, grid, st);
  return check_launch(who);
}
