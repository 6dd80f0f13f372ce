// Softmax attention over a paged K/V cache (include/qg.h, qg_paged_attention):
//
//   out[r][h] = sum_{t <= p(r)} softmax_t(scale q[r][h] . k[t][h/G]) v[t][h/G],
//   p(r) = kv_len[b] - n_b + (r - row_start[b]).
//
// What bounds it. A cached token of one KV head is 2 D codes (or bf16
// values) and meets G query heads of each row: 2 G flops a byte for a single
// row, so a decode is bound by reading the cache once. Long prompts are
// bound by the tensor cores.
//
// The tile. The unit is a block of 16 tokens, which never straddles a page
// and has one K and one V scale. Its "columns" are (row, head) pairs of one
// KV head. Scores are computed transposed, S^T = K Q^T, and the output as
// O^T = V^T P^T, with mma.sync m16n8k16: the 16 tokens (then 16 dims) are the
// M side and 8 columns the N side, so a decode's few query heads waste
// little, and the K and V operands go from global memory to registers in the
// order the fragments want: the contraction's order is free, so a lane takes
// 16 neighbouring bytes of two K rows, and 1/8 of the dims of four V rows,
// in whole 16-byte loads, with no shared memory and no barrier between them.
// P^T goes from the accumulator's layout to the operand's by movmatrix.
//
// int8 codes are exact in fp16 (1024 + q by a byte permute, minus 1152), so
// they are multiplied as they are; the K scale multiplies the scores, the V
// scale the weights. q is multiplied by a power of two before its rounding
// to fp16 (largest value in [2^13, 2^14)): bf16 q is exact down to 2^-28 of the
// largest, fp32 q takes two fp16 terms (22 bits). Weights times V's scale
// are brought into fp16's range by a running power of two r >= |scale| and
// 2^11: they keep 11 bits down to 2^-25 of the largest, where bf16 would
// keep 8. bf16 pages: bf16 operands, fp32 q in three bf16 terms, the weights in two
// (16 bits). With an fp32 output the weights take two terms (int8 pages) or three
// (bf16 pages); the denominator sums them unrounded. (One term for bf16 pages with a
// bf16 output: 7 x 1500 of 64 11.3 in place of 11.5 us, 32 x 2048 54.5 and 54.8, and
// errors of 2.3e-3 of the largest value in place of its rounding's 1.7e-3.)
//
// The softmax is online per column in fp32, with a lazy maximum: the
// reference only moves (and the accumulators are only rescaled) when a score
// passes it by 2^kMargin, one vote per tile instead of the shuffles of a
// maximum.
//
// Work split (decodes and short prompts). A CTA's 8 warps take its keys' tiles
// in turn and merge in shared memory. Kernel "cluster", where equal shares are
// good enough (see plan): an item, a (sequence, KV head, column tile), belongs
// to a cluster of up to 8 CTAs, whose results meet through distributed shared
// memory. Kernel "split": all items' key chunks form one line that is cut into
// equal pieces, one per CTA, from the lengths on the device: ragged batches are
// balanced, and the grid never depends on them. An item inside one piece is
// written out; the others' parts go to the workspace and a second small launch
// merges them in order. Results do not depend on scheduling in either.
// Larger prompts with a bf16 q and out go to the tcgen05 kernel of
// paged_attention_tc.cu.
#include <cuda_fp16.h>

#include "mma_sync.cuh"
#include "paged_attention.cuh"

#include <algorithm>
#include <cfloat>
#include <cmath>

namespace qg {
namespace pa {

constexpr int kWarps = 8;            // of the cluster and split kernels
constexpr int kCols = 8;             // (row, head) columns of a tile
constexpr int kChunk = kWarps * kBlock;
constexpr int kMergeThreads = 512;
constexpr int kItem = 2;             // chunks' worth of an item's other work (see SeqWork)
constexpr int kSlack = 2;            // chunks (see plan)
constexpr int kMaxPieces = 320;      // of the split kernel (two CTAs on each of 148 SMs)

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <bool I8>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (I8)
    mma_f16(c, a0, a1, a2, a3, b0, b1);
  else
    mm::mma_bf16(c, a0, a1, a2, a3, b0, b1);
}
// (lo, hi) rounded to the operand type; lo and hi become the rests.
template <bool I8>
__device__ __forceinline__ uint32_t take16(float& lo, float& hi) {
  if constexpr (I8) {
    const __half2 h = __floats2half2_rn(lo, hi);
    const float2 f = __half22float2(h);
    lo -= f.x;
    hi -= f.y;
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    lo -= __bfloat162float(h.x);
    hi -= __bfloat162float(h.y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// Four weights in PS bf16 terms, each but the last one cut off, not rounded, and
// at least 2^-126 where the weight is not 0: so a lower term is never 0 or of
// the other sign beside an infinite V value, whose sum would be NaN.
template <int PS>
__device__ __forceinline__ void split_weights(const float (&p)[4], uint32_t (&b)[PS][2]) {
  float rest[4], least[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    rest[i] = p[i];
    least[i] = fminf(p[i], FLT_MIN);
  }
#pragma unroll
  for (int e = 0; e < PS; ++e) {
    float h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = e + 1 < PS ? __uint_as_float(__float_as_uint(rest[i]) & 0xFFFF0000u) : rest[i];
      if (e > 0) h[i] = fmaxf(h[i], least[i]);
      rest[i] -= h[i];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      b[e][i] = e + 1 < PS ? __byte_perm(__float_as_uint(h[2 * i]), __float_as_uint(h[2 * i + 1]), 0x7632u)
                           : mm::pack_bf16(h[2 * i], h[2 * i + 1]);
  }
}

// Visible tokens of column c of the item's sequence. Columns past the last
// one (their q is zero, nothing is stored for them) see everything, so that
// they do not make a tile partly masked.
__device__ __forceinline__ int visible(const Params& P, const Item& it, int c) {
  const int i = c / P.G;
  return i < it.n ? it.len - it.n + i + 1 : 0x7FFFFFFF;
}

// The lane's D/32 neighbouring values of column c's query head.
template <int D>
__device__ __forceinline__ void load_q(const Params& P, const Item& it, int c, int lane,
                                       float (&x)[D / 32]) {
  constexpr int EPL = D / 32;
  const int i = c / P.G;
#pragma unroll
  for (int e = 0; e < EPL; ++e) x[e] = 0.f;
  if (i >= it.n) return;
  const long long at =
      ((long long)(it.r0 + i) * P.H + it.h * P.G + (c - i * P.G)) * D + lane * EPL;
  if (P.q_bf16) {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(P.q) + at;
#pragma unroll
    for (int e = 0; e < EPL; e += 2) {
      const uint32_t w = __ldcg(reinterpret_cast<const uint32_t*>(p + e));
      x[e] = bf16_lo(w);
      x[e + 1] = bf16_hi(w);
    }
  } else {
    const float* p = reinterpret_cast<const float*>(P.q) + at;
#pragma unroll
    for (int e = 0; e < EPL; e += 2) {
      const float2 w = __ldcg(reinterpret_cast<const float2*>(p + e));
      x[e] = w.x;
      x[e + 1] = w.y;
    }
  }
}

// Where element (column n, dim d) of Q lies in the fragments' order
// [k step][term][lane][4] of 16-bit values: a lane's 16 bytes
// of a K row are neighbouring dims, four per k step.
template <bool I8, int QS>
__device__ __forceinline__ int q_at(int n, int d, int term) {
  constexpr int PL = I8 ? 16 : 8;  // dims of a lane's 16 bytes
  const int t = d % (4 * PL) / PL, ks = d / (4 * PL) * (PL / 4) + d % PL / 4;
  return ((ks * QS + term) * 32 + (n % 8) * 4 + t) * 4 + d % 4;
}

// Stores a lane's neighbouring values of one column, split into QS terms.
template <int D, bool I8, int QS>
__device__ __forceinline__ void put_q(uint16_t* sq, int n, int lane, float (&x)[D / 32]) {
#pragma unroll
  for (int s = 0; s < QS; ++s)
#pragma unroll
    for (int e = 0; e < D / 32; e += 2)
      *reinterpret_cast<uint32_t*>(sq + q_at<I8, QS>(n, lane * (D / 32) + e, s)) =
          take16<I8>(x[e], x[e + 1]);
}

// A warp's running state over the columns of its item.
template <int D>
struct State {
  float m[2], l[2];        // columns 2 t (+ 1): reference, this lane's weights
  float o[D / 16][4];      // dims g D/8 + 2 i (+ 1), columns 2 t (+ 1)
  float r;                 // unit of o: the V scales seen are at most r

  __device__ __forceinline__ void clear() {
    m[0] = m[1] = -FLT_MAX;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    r = FLT_MIN;
  }
};

// A warp's walk over tiles first, first + step, ... < end of one sequence
// and KV head: page lookups 32 tiles at a time, K and V one tile ahead.
template <int D, bool I8, int QS, int PS>
struct Walk {
  static constexpr int ES = I8 ? 1 : 2;
  static constexpr int KC = D * ES / 64;        // 16-byte pieces of a lane per K row
  static constexpr int VB = D * ES / 8;         // bytes of a lane per V row
  static constexpr int VC = (VB + 15) / 16;
  const Params& P;
  const int lane, g, t;
  int lim[2];     // visible tokens of the lane's columns
  int min_lim, len;   // of all the item's columns; cached tokens
  float qf[2];    // scale_log2 / 2^e of the lane's columns
  const uint16_t* sq;
  uint4 kr[2][KC];
  uint4 vr[4][VC];
  float ks, vs;
  int blocks;         // lane i: block index in the pool of tile base + i step, -1: bad page
  int tile, step, end;

  __device__ __forceinline__ Walk(const Params& P_, int lane_)
      : P(P_), lane(lane_), g(lane_ >> 2), t(lane_ & 3) {}

  __device__ __forceinline__ void lookup(const Item& it, int first) {
    const long long at = (long long)first + (long long)lane * step;
    blocks = -1;
    if (at < end) {
      const int pi = (int)at / P.bpp;
      const int page = __ldcg(P.table + (long long)it.b * P.max_pages + pi);
      if (page >= 0 && page < P.num_pages)
        blocks = (page * P.Hkv + it.h) * P.bpp + ((int)at - pi * P.bpp);
    }
  }

  __device__ __forceinline__ void load_k(int blk) {
    const bool ok = blk >= 0;
    const uint8_t* p = P.kp + (long long)(ok ? blk : 0) * (kBlock * D * ES) + g * (D * ES) + t * 16;
#pragma unroll
    for (int c = 0; c < KC; ++c) {
      kr[0][c] = load16_if(p + c * 64, ok);
      kr[1][c] = load16_if(p + 8 * D * ES + c * 64, ok);
    }
    // a bad page: NaN scores for whoever sees its tokens
    ks = load_if(P.ks + blk, I8 && ok, ok ? 1.f : __int_as_float(0x7FC00000));
  }

  // Rows at or past the sequence's end hold anything: zero (0 * NaN).
  __device__ __forceinline__ void load_v(int blk) {
    const bool ok = blk >= 0;
    const int left = I8 ? kBlock : len - tile * kBlock;
    const uint8_t* p = P.vp + (long long)(ok ? blk : 0) * (kBlock * D * ES) + g * VB;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = 2 * t + (i & 1) + 8 * (i >> 1);
      const uint8_t* pi = p + key * (D * ES);
      const bool in = ok && key < left;
      if constexpr (VB >= 16) {
#pragma unroll
        for (int c = 0; c < VC; ++c) vr[i][c] = load16_if(pi + c * 16, in);
      } else {
        const uint2 w = load8_if(pi, in);
        vr[i][0] = make_uint4(w.x, w.y, 0, 0);
      }
    }
    vs = load_if(P.vs + blk, I8 && ok, 1.f);
  }

  static __device__ __forceinline__ uint32_t word(const uint4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
  }

  __device__ __forceinline__ void scores(float (&s)[4]) {
    float rest[4];  // of q's lower terms (see weigh)
    s[0] = s[1] = s[2] = s[3] = 0.f;
    if constexpr (QS > 1) rest[0] = rest[1] = rest[2] = rest[3] = 0.f;
#pragma unroll
    for (int c = 0; c < KC; ++c) {
#pragma unroll
      for (int u = 0; u < (I8 ? 4 : 2); ++u) {
        uint32_t a0, a1, a2, a3;
        if constexpr (I8) {
          const uint32_t lo = word(kr[0][c], u) ^ 0x80808080u, hi = word(kr[1][c], u) ^ 0x80808080u;
          a0 = codes01(lo);
          a1 = codes01(hi);
          a2 = codes23(lo);
          a3 = codes23(hi);
        } else {
          a0 = word(kr[0][c], 2 * u);
          a1 = word(kr[1][c], 2 * u);
          a2 = word(kr[0][c], 2 * u + 1);
          a3 = word(kr[1][c], 2 * u + 1);
        }
        const int step = c * (I8 ? 4 : 2) + u;
#pragma unroll
        for (int e = 0; e < QS; ++e) {
          const uint2 b =
              *reinterpret_cast<const uint2*>(sq + ((step * QS + e) * 32 + lane) * 4);
          mma<I8>(e ? rest : s, a0, a1, a2, a3, b.x, b.y);
        }
      }
    }
    // (bf16 pages: an infinite K value makes its term of q infinite in s, which
    // says it all; times a lower term of 0 or the other sign it is noise)
    if constexpr (QS > 1) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] += I8 ? rest[e] : fminf(fmaxf(rest[e], -FLT_MAX), FLT_MAX);
    }
  }

  // bf16 pages, a tile that some columns see in part, with V values that are
  // not finite: 0 * NaN must not reach the columns that do not see them, so
  // the products are formed one by one (never taken with finite values).
  static __device__ __forceinline__ void accumulate_seen(State<D>& S, const float (&p)[4],
                                                      const uint4 (&vr)[4][VC], int lane) {
    const int t = lane & 3;
#pragma unroll 1
    for (int key = 0; key < kBlock; ++key) {
      const int slot = (key & 1) + 2 * (key >> 3), src = (lane & ~3) | ((key & 7) >> 1);
      float w[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        w[e] = __shfl_sync(0xffffffffu, key < 8 ? p[e] : p[2 + e], (key & 7) * 4 + t);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint32_t mine = slot == 0   ? word(vr[0][i / 4], i % 4)
                              : slot == 1 ? word(vr[1][i / 4], i % 4)
                              : slot == 2 ? word(vr[2][i / 4], i % 4)
                                          : word(vr[3][i / 4], i % 4);
        const uint32_t x = __shfl_sync(0xffffffffu, mine, src);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (w[e] != 0.f) {
            S.o[i][e] = fmaf(w[e], bf16_lo(x), S.o[i][e]);
            S.o[i][2 + e] = fmaf(w[e], bf16_hi(x), S.o[i][2 + e]);
          }
      }
    }
  }

  __device__ __forceinline__ void weigh(State<D>& S, float (&p)[4], bool part) {
    if constexpr (!I8) {
      if (part) {
        // (0 * x is NaN for these alone: one instruction for two values)
        __nv_bfloat162 z = __floats2bfloat162_rn(0.f, 0.f);
        const __nv_bfloat162 zero = z;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < VC; ++c)
#pragma unroll
            for (int e = 0; e < (VB >= 16 ? 4 : 2); ++e) {
              const uint32_t x = word(vr[i][c], e);
              z = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x), zero, z);
            }
        const bool odd = (*reinterpret_cast<const uint32_t*>(&z) & 0x7FFF7FFFu) != 0;
        if (__any_sync(0xffffffffu, odd)) {
          accumulate_seen(S, p, vr, lane);
          return;
        }
      }
    }
    uint32_t b[PS][2];
    if constexpr (I8 || PS == 1) {
#pragma unroll
      for (int e = 0; e < PS; ++e) {
        b[e][0] = take16<I8>(p[0], p[1]);
        b[e][1] = take16<I8>(p[2], p[3]);
      }
    } else {
      split_weights<PS>(p, b);
    }
#pragma unroll
    for (int e = 0; e < PS; ++e) {
      b[e][0] = transpose8x8(b[e][0]);
      b[e][1] = transpose8x8(b[e][1]);
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      uint32_t a0, a1, a2, a3;
      if constexpr (I8) {
        // dims 2 i and 2 i + 1 of the lane's: bytes of word i / 2
        const int c = i / 8, e = i / 2 % 4;
        const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
        const uint32_t lo =
            __byte_perm(word(vr[0][c], e), word(vr[1][c], e), sel) ^ 0x80808080u;
        const uint32_t hi =
            __byte_perm(word(vr[2][c], e), word(vr[3][c], e), sel) ^ 0x80808080u;
        a0 = codes01(lo);
        a1 = codes23(lo);
        a2 = codes01(hi);
        a3 = codes23(hi);
      } else {
        const int c = i / 4, e = i % 4;
        a0 = __byte_perm(word(vr[0][c], e), word(vr[1][c], e), 0x5410u);
        a1 = __byte_perm(word(vr[0][c], e), word(vr[1][c], e), 0x7632u);
        a2 = __byte_perm(word(vr[2][c], e), word(vr[3][c], e), 0x5410u);
        a3 = __byte_perm(word(vr[2][c], e), word(vr[3][c], e), 0x7632u);
      }
      // The tensor core's adds truncate. Terms added to the running sum, 16 tokens an
      // add: what a bf16 result shows of that is nothing. For an fp32 one the tile's
      // sum is formed by itself, smallest term first, and added to the running one
      // with rounding, which keeps a long cache's sum at fp32's accuracy (32749
      // tokens: 1.3e-6 off with the terms added to the running sum).
      if constexpr (QS == 1) {
#pragma unroll
        for (int e = PS - 1; e >= 0; --e) mma<I8>(S.o[i], a0, a1, a2, a3, b[e][0], b[e][1]);
      } else {
        float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = PS - 1; e >= 0; --e) mma<I8>(t, a0, a1, a2, a3, b[e][0], b[e][1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) S.o[i][e] += t[e];
      }
    }
  }

  // The walk's tiles; the first one's loads go out.
  __device__ __forceinline__ void begin(const Item& it, int first, int step_, int end_) {
    tile = first;
    step = step_;
    end = end_;
    if (tile >= end) return;
    lookup(it, tile);
    const int blk = __shfl_sync(0xffffffffu, blocks, 0);
    load_k(blk);
    load_v(blk);
  }

  __device__ __forceinline__ void run(State<D>& S, const Item& it) {
    if (tile >= end) return;
    int at = 0;  // the tile's place in the batch of lookups
    for (;;) {
      const bool more = end - tile > step;
      if (more && ++at == 32) {
        at = 0;
        lookup(it, tile + step);
      }
      const int next = __shfl_sync(0xffffffffu, blocks, at);
      float p[4];
      scores(p);
      float f[2];
      f[0] = qf[0] * ks;
      f[1] = qf[1] * ks;
      if (more) load_k(next);
      // scores in log2 units, masked
      const int key0 = tile * kBlock + g;
      const bool part = tile * kBlock + kBlock > min_lim;
      bool over = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        p[e] *= f[e & 1];
        if (part && key0 + 8 * (e >> 1) >= lim[e & 1]) p[e] = -INFINITY;
        over |= p[e] > S.m[e & 1] + kMargin;
      }
      const bool wider = I8 && fabsf(vs) > S.r && fabsf(vs) <= FLT_MAX;  // the same in all lanes
      if (__any_sync(0xffffffffu, over) || wider) {
        float down = 1.f;
        if (wider) {
          const int ex = min(254, ((__float_as_int(vs) >> 23) & 255) + 1);
          const float r = __int_as_float(ex << 23);
          down = S.r / r;
          S.r = r;
        }
        float a[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(p[e], p[2 + e]);
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          x = fmaxf(x, S.m[e]);
          a[e] = ex2(S.m[e] - x);
          S.m[e] = x;
          S.l[e] *= a[e];
        }
        a[0] *= down;
        a[1] *= down;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          S.o[i][0] *= a[0];
          S.o[i][1] *= a[1];
          S.o[i][2] *= a[0];
          S.o[i][3] *= a[1];
        }
      }
      const float wv = I8 ? vs * (1.f / S.r) * 2048.f : 1.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = ex2(p[e] - S.m[e & 1]);
        S.l[e & 1] += x;
        // a token that the column does not see keeps weight 0 whatever the
        // block's scale is
        if constexpr (I8) p[e] = part && p[e] == -INFINITY ? 0.f : x * wv;
        else p[e] = x;
      }
      weigh(S, p, part);
      if (!more) break;
      tile += step;
      load_v(next);
    }
  }
};

// The unit of the accumulators of a state (2^11: the weights' own).
template <bool I8>
__device__ __forceinline__ float o_unit(float r) {
  return I8 ? r * (1.f / 2048.f) : 1.f;
}

// q of the item's column tile into shared memory, a column a warp, with the
// factor that turns a column's products into log2 units in sf. The loads go
// out first (take), so that they overlap the first keys' ones.
template <int D, bool I8, int QS>
struct StageQ {
  static_assert(kCols == kWarps, "a column a warp");
  float x[D / 32];
  __device__ __forceinline__ void take(const Params& P, const Item& it, int warp, int lane) {
    load_q<D>(P, it, it.ct * kCols + warp, lane, x);
  }
  __device__ __forceinline__ void put(const Params& P, uint16_t* sq, float* sf, int warp, int lane) {
    float unit = 1.f;
    if constexpr (I8) {
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) top = fmaxf(top, fabsf(x[e]));
      unit = q_unit(warp_max(top));
#pragma unroll
      for (int e = 0; e < D / 32; ++e) x[e] *= unit;
    }
    put_q<D, I8, QS>(sq, warp, lane, x);
    if (lane == 0) sf[warp] = P.scale_log2 / unit;
  }
};

template <class W>
__device__ __forceinline__ void set_limits(const Params& P, const Item& it, W& w) {
  int lo = 0x7FFFFFFF;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    w.lim[e] = visible(P, it, it.ct * kCols + 2 * w.t + e);
    lo = min(lo, w.lim[e]);
  }
  lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, 1));
  w.min_lim = min(lo, __shfl_xor_sync(0xffffffffu, lo, 2));
}

// Where column c of the item goes: its (row, query head) in out.
__device__ __forceinline__ int out_row(const Params& P, const Item& it, int c) {
  const int i = c / P.G;
  return (it.r0 + i) * P.H + it.h * P.G + (c - i * P.G);  // (below 2^30)
}
__device__ __forceinline__ void store_out(const Params& P, int row, int d, int D, float x) {
  const long long at = (long long)row * D + d;
  if (P.out_bf16)
    reinterpret_cast<uint16_t*>(P.out)[at] = f32_to_bf16_bits(x);
  else
    reinterpret_cast<float*>(P.out)[at] = x;
}

// A warp's state to shared memory: weights summed over the lanes that share a
// column, outputs in plain units.
template <int D, bool I8>
__device__ __forceinline__ void put_state(const State<D>& S, float* so, float* sm, float* sl,
                                          int cols, int warp, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const float u = o_unit<I8>(S.r);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float l = S.l[e];
    l += __shfl_xor_sync(0xffffffffu, l, 4);
    l += __shfl_xor_sync(0xffffffffu, l, 8);
    l += __shfl_xor_sync(0xffffffffu, l, 16);
    const int n = 2 * t + e;
    if (n < cols) {
      if (g == 0) {
        sm[warp * kCols + n] = S.m[e];
        sl[warp * kCols + n] = l;
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
        *reinterpret_cast<float2*>(so + (warp * kCols + n) * D + g * (D / 8) + 2 * i) =
            make_float2(S.o[i][e] * u, S.o[i][2 + e] * u);
    }
  }
}
// The CTA's reference M, weights' sum L and output O at column n, dim d.
template <int D>
__device__ __forceinline__ void join_warps(const float* so, const float* sm, const float* sl, int n,
                                           int d, float& M, float& L, float& O) {
  M = sm[n];
#pragma unroll
  for (int k = 1; k < kWarps; ++k) M = fmaxf(M, sm[k * kCols + n]);
  L = O = 0.f;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) {
    const float a = ex2(sm[k * kCols + n] - M);
    L = fmaf(a, sl[k * kCols + n], L);
    O = fmaf(a, so[(k * kCols + n) * D + d], O);
  }
}

// ------------------------------------------------------------ split kernel --

// A sequence's column tiles, the chunks of each of its items (at least one, so
// that empty ones are written), and an item's length on the line: its chunks
// behind kItem units for what it costs besides (q, the warps' join, the store):
// without them pieces of many short items took several times as long as the
// others (600 fp32 rows of 5 users over up to 2000 int8 tokens 164 us, with one
// unit 107, two 91, four 96). The host keeps a call's units below 2^31.
struct SeqWork {
  int tiles, chunks;
  __device__ __forceinline__ SeqWork(const Params& P, const Item& it) {
    tiles = (it.n * P.G + kCols - 1) / kCols;
    chunks = max(1, (it.len + kChunk - 1) / kChunk);
  }
  __device__ __forceinline__ int units() const { return chunks + kItem; }
  __device__ __forceinline__ unsigned total(int Hkv) const {
    return (unsigned)tiles * Hkv * units();
  }
};
// Blocks of 16 tokens that the item's last column sees.
__device__ __forceinline__ int seen_blocks(const Params& P, const Item& it) {
  const int rows = min(it.n, ((it.ct + 1) * kCols - 1) / P.G + 1);
  return (max(0, it.len - it.n + rows) + kBlock - 1) / kBlock;
}

// The line of N units cut into pieces: the first `rem` have q + 1 units,
// the others q.
struct Cut {
  unsigned q, rem;
  __device__ __forceinline__ Cut(unsigned N, unsigned pieces) {
    q = N / pieces;
    rem = N - q * pieces;
  }
  __device__ __forceinline__ unsigned begin(unsigned c) const { return q * c + min(c, rem); }
  __device__ __forceinline__ unsigned piece_of(unsigned x) const {
    const unsigned wide = (q + 1) * rem;
    return x < wide ? x / (q + 1) : rem + (x - wide) / q;
  }
};

// Running sums over the sequences, 32 at a time (every warp by itself): f
// gets a sequence (its item's n is 0 past the last one), its work, and the
// chunks before it; returns all chunks.
template <class F>
__device__ __forceinline__ unsigned each_seq(const Params& P, F f) {
  const int lane = threadIdx.x & 31;
  unsigned before = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < P.B; b0 += 32) {
    Item it = {0, 0, 0, 0, 0, 0};
    if (b0 + lane < P.B) set_seq(P, it, b0 + lane);
    const SeqWork w(P, it);
    const unsigned mine = w.total(P.Hkv);
    unsigned x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    f(it, w, before + x - mine, mine);
    before += __shfl_sync(0xffffffffu, x, 31);
  }
  return before;
}

// CTAs of the split kernel that an SM holds: two where a warp's keys, next
// keys and sums fit 128 registers. (bf16 pages of head size 128 at two CTAs
// spilled: 42.6 us against 37.8 for 32749 tokens in fp32.)
constexpr int split_ctas(int D, bool i8) { return D <= 64 || (i8 && D <= 128) ? 2 : 1; }

template <int D, bool I8, int QS, int PS>
__global__ void __launch_bounds__(kWarps * 32, split_ctas(D, I8))
split_kernel(const __grid_constant__ Params P) {
  extern __shared__ __align__(16) uint8_t smem[];
  float* so = reinterpret_cast<float*>(smem);            // [kWarps][kCols][D]
  float* sm = so + kWarps * kCols * D;                      // [kWarps][kCols]
  float* sl = sm + kWarps * kCols;                          // [kWarps][kCols]
  uint16_t* sq = reinterpret_cast<uint16_t*>(sl + kWarps * kCols);  // fragments of q
  __shared__ float sf[kCols];
  __shared__ int rows[2][kCols];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_trigger();  // the merge may find its items meanwhile

  // This CTA's piece [pos, stop) of the line, and the item where it begins.
  // Up to 32 sequences: one look at them tells both; more: a first look for
  // the line's length, a second for the place.
  Item it = {0, 0, 0, 0, 0, 0};
  unsigned pos = 0, stop = 0, rest = 0;
  const auto piece = [&](unsigned N) {
    const Cut cut(N, P.pieces);
    pos = cut.begin(blockIdx.x);
    stop = cut.begin(blockIdx.x + 1);
  };
  const auto settle = [&](const Item& mine, unsigned before, unsigned len) {
    const unsigned m = __ballot_sync(0xffffffffu, pos >= before && pos - before < len);
    if (!m) return;
    const int l = __ffs(m) - 1;
    it.b = __shfl_sync(0xffffffffu, mine.b, l);
    it.r0 = __shfl_sync(0xffffffffu, mine.r0, l);
    it.n = __shfl_sync(0xffffffffu, mine.n, l);
    it.len = __shfl_sync(0xffffffffu, mine.len, l);
    rest = pos - __shfl_sync(0xffffffffu, before, l);
  };
  if (P.B <= 32) {
    Item mine;
    unsigned before, len;
    piece(each_seq(P, [&](const Item& i, const SeqWork&, unsigned b, unsigned l) {
      mine = i;
      before = b;
      len = l;
    }));
    if (pos >= stop) return;
    settle(mine, before, len);
  } else {
    piece(each_seq(P, [](const Item&, const SeqWork&, unsigned, unsigned) {}));
    if (pos >= stop) return;
    each_seq(P, [&](const Item& i, const SeqWork&, unsigned b, unsigned l) {
      settle(i, b, l);
    });
  }
  SeqWork w(P, it);
  // (head, column tile) of the sequence, and the item's first chunk here
  int unit = (int)(rest / (unsigned)w.units());
  int c0 = (int)rest - unit * w.units();
  int left = c0 + (int)(stop - pos);  // units from the item's beginning to the piece's end
  // A cut before an item's first chunk moves to the item's beginning.
  if (c0 <= kItem) {
    c0 = 0;
    if (left <= kItem) return;
  }
  it.h = unit / w.tiles;
  it.ct = unit - it.h * w.tiles;

  Walk<D, I8, QS, PS> walk(P, lane);
  StageQ<D, I8, QS> qs;
  walk.sq = sq;
  State<D> S;
  const auto start = [&](const Item& i, int first, int last) {  // chunks [first, last)
    qs.take(P, i, warp, lane);
    walk.len = i.len;
    walk.begin(i, first * kWarps + warp, kWarps, min(last * kWarps, seen_blocks(P, i)));
  };
  int c1 = min(w.units(), left);
  start(it, max(0, c0 - kItem), max(0, c1 - kItem));
  int turn = 0;
  for (;;) {
    qs.put(P, sq, sf, warp, lane);
    turn ^= 1;  // (slower warps may still store the item before)
    if (tid < kCols) rows[turn][tid] = out_row(P, it, it.ct * kCols + tid);
    set_limits(P, it, walk);
    __syncthreads();
    walk.qf[0] = sf[2 * walk.t];
    walk.qf[1] = sf[2 * walk.t + 1];
    S.clear();
    walk.run(S, it);
    // the next item's first keys and q go out before this one is put away
    const Item cur = it;
    const bool first_part = c0 == 0, whole = c0 == 0 && c1 == w.units();
    left -= w.units();
    const bool more = left > kItem;
    if (more) {
      if (++unit == w.tiles * P.Hkv) {
        unit = 0;
        do {  // the next sequence with rows (one exists: chunks are left)
          if (it.b + 1 >= P.B) return;  // (unless row starts decrease)
          set_seq(P, it, it.b + 1);
        } while (it.n == 0);
        w = SeqWork(P, it);
      }
      it.h = unit / w.tiles;
      it.ct = unit - it.h * w.tiles;
      c0 = 0;
      c1 = min(w.units(), left);
      start(it, 0, max(0, c1 - kItem));
    }
    const int cols = min(kCols, cur.n * P.G - cur.ct * kCols);  // of the tile, real ones
    put_state<D, I8>(S, so, sm, sl, cols, warp, lane);
    __syncthreads();
    float* part = P.part + (long long)(2 * blockIdx.x + first_part) * kCols * (D + 2);
    for (int i = tid; i < cols * D; i += kWarps * 32) {
      const int n = i / D, d = i % D;
      float M, L, O;
      join_warps<D>(so, sm, sl, n, d, M, L, O);
      if (whole) {
        store_out(P, rows[turn][n], d, D, L != 0.f ? O / L : 0.f);
      } else {
        part[2 * kCols + i] = O;
        if (d == 0) {
          part[n] = M;
          part[kCols + n] = L;
        }
      }
    }
    if (!more) return;
  }
}

// ---------------------------------------------------------- cluster kernel --

__device__ __forceinline__ uint32_t remote(const float* p, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;"
      : "=r"(a)
      : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
  return a;
}
__device__ __forceinline__ float ld_remote(const float* p, int rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// An item a cluster: its Z CTAs take equal shares of the item's chunks and
// join their results through distributed shared memory, so one launch does.
// A column tile's slot: a sequence with x columns has at most x / kCols + 1 tiles,
// so slot ranges [begin G / kCols + b, end G / kCols + b + 1) do not overlap.
constexpr int kMaxZ = 8;
template <int D, bool I8, int QS, int PS>
__global__ void __launch_bounds__(kWarps * 32, split_ctas(D, I8))
cluster_kernel(const __grid_constant__ Params P) {
  extern __shared__ __align__(16) uint8_t smem[];
  float* so = reinterpret_cast<float*>(smem);            // [kWarps][kCols][D]
  float* sm = so + kWarps * kCols * D;                      // [kWarps][kCols]
  float* sl = sm + kWarps * kCols;                          // [kWarps][kCols]
  uint16_t* sq = reinterpret_cast<uint16_t*>(sl + kWarps * kCols);  // fragments of q
  __shared__ float sf[kCols];
  __shared__ int rows[kCols];
  __shared__ float pm[kCols], pl[kCols], po[kCols * D];           // the CTA's result
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int Z = P.pieces, z = blockIdx.x % Z, u = blockIdx.x / Z;
  pdl_wait();
  pdl_trigger();

  Item it = {-1, 0, 0, 0, 0, 0};
#pragma unroll 1
  for (int b0 = 0; b0 < P.B && it.b < 0; b0 += 32) {
    Item mine = {-1, 0, 0, 0, 0, 0};
    if (b0 + lane < P.B) set_seq(P, mine, b0 + lane);
    const int from = (int)((long long)mine.r0 * P.G / kCols) + b0 + lane;
    const int to = (int)((long long)(mine.r0 + mine.n) * P.G / kCols) + b0 + lane;
    const unsigned m = __ballot_sync(0xffffffffu, mine.n && u >= from && u <= to);
    if (m) {
      const int l = __ffs(m) - 1;
      it.b = __shfl_sync(0xffffffffu, mine.b, l);
      it.r0 = __shfl_sync(0xffffffffu, mine.r0, l);
      it.n = __shfl_sync(0xffffffffu, mine.n, l);
      it.len = __shfl_sync(0xffffffffu, mine.len, l);
      it.ct = __shfl_sync(0xffffffffu, u - from, l);
    }
  }
  if (it.b < 0) return;  // (the cluster's CTAs alike)
  const SeqWork w(P, it);
  if (it.ct >= w.tiles) return;
  it.h = blockIdx.y;

  Walk<D, I8, QS, PS> walk(P, lane);
  StageQ<D, I8, QS> qs;
  walk.sq = sq;
  State<D> S;
  const int c0 = (int)((long long)w.chunks * z / Z), c1 = (int)((long long)w.chunks * (z + 1) / Z);
  qs.take(P, it, warp, lane);
  walk.len = it.len;
  walk.begin(it, c0 * kWarps + warp, kWarps, min(c1 * kWarps, seen_blocks(P, it)));
  qs.put(P, sq, sf, warp, lane);
  if (tid < kCols) rows[tid] = out_row(P, it, it.ct * kCols + tid);
  set_limits(P, it, walk);
  __syncthreads();
  walk.qf[0] = sf[2 * walk.t];
  walk.qf[1] = sf[2 * walk.t + 1];
  S.clear();
  walk.run(S, it);
  const int cols = min(kCols, it.n * P.G - it.ct * kCols);
  put_state<D, I8>(S, so, sm, sl, cols, warp, lane);
  __syncthreads();
  for (int i = tid; i < cols * D; i += kWarps * 32) {
    const int n = i / D, d = i % D;
    float M, L, O;
    join_warps<D>(so, sm, sl, n, d, M, L, O);
    if (Z == 1) {
      store_out(P, rows[n], d, D, L != 0.f ? O / L : 0.f);
    } else {
      po[i] = O;
      if (d == 0) {
        pm[n] = M;
        pl[n] = L;
      }
    }
  }
  if (Z == 1) return;
  cluster_sync();
  // CTA z writes its share of the outputs; a thread's remote loads go out
  // together
  for (int i = z * kWarps * 32 + tid; i < cols * D; i += Z * kWarps * 32) {
    const int n = i / D, d = i % D;
    float m[kMaxZ], l[kMaxZ], o[kMaxZ];
#pragma unroll
    for (int k = 0; k < kMaxZ; ++k) {
      m[k] = k < Z ? ld_remote(&pm[n], k) : -FLT_MAX;
      l[k] = k < Z ? ld_remote(&pl[n], k) : 0.f;
      o[k] = k < Z ? ld_remote(&po[i], k) : 0.f;
    }
    float M = -FLT_MAX, L = 0.f, O = 0.f;
#pragma unroll
    for (int k = 0; k < kMaxZ; ++k) M = fmaxf(M, m[k]);
#pragma unroll
    for (int k = 0; k < kMaxZ; ++k) {
      const float a = ex2(m[k] - M);
      L = fmaf(a, l[k], L);
      O = fmaf(a, o[k], O);
    }
    store_out(P, rows[n], d, D, L != 0.f ? O / L : 0.f);
  }
  cluster_sync();  // nobody ends while its shared memory is read
}

// ------------------------------------------------------------ merge kernel --

// Items cut between pieces: one CTA per (column tile, head). A column tile's
// slot: a sequence with x columns has at most x / kCols + 1 tiles, so slot
// ranges [begin G / kCols + b, end G / kCols + b + 1) do not overlap.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const __grid_constant__ Params P) {
  __shared__ float acc[kMergeThreads];
  const int tid = threadIdx.x, lane = tid & 31;
  // (the split kernel's CTAs have passed their own wait, so what came before
  // it on the stream is complete: lengths and row starts may be read)
  const int u = blockIdx.x;
  Item it = {-1, 0, 0, 0, 0, 0};
  unsigned before = 0;
  const unsigned N = each_seq(P, [&](const Item& i, const SeqWork&, unsigned b, unsigned) {
    const int end = i.r0 + i.n;
    const bool in = i.n && u >= (int)((long long)i.r0 * P.G / kCols + i.b) &&
                    u <= (int)((long long)end * P.G / kCols + i.b);
    const unsigned m = __ballot_sync(0xffffffffu, in);
    if (!m) return;
    const int l = __ffs(m) - 1;
    it.b = __shfl_sync(0xffffffffu, i.b, l);
    it.r0 = __shfl_sync(0xffffffffu, i.r0, l);
    it.n = __shfl_sync(0xffffffffu, i.n, l);
    it.len = __shfl_sync(0xffffffffu, i.len, l);
    before = __shfl_sync(0xffffffffu, b, l);
  });
  // Every CTA waits before it ends: this grid must not complete before the
  // split kernel's, for which the next kernel waits only through this one.
  if (it.b < 0) {
    pdl_wait();
    return;
  }
  const SeqWork w(P, it);
  it.ct = u - (int)((long long)it.r0 * P.G / kCols + it.b);
  it.h = blockIdx.y;
  if (it.ct >= w.tiles) {
    pdl_wait();
    return;
  }
  const unsigned begin = before + (unsigned)(it.h * w.tiles + it.ct) * w.units();
  const Cut cut(N, P.pieces);
  // (within the workspace even if row starts decrease)
  const int last = P.pieces - 1;
  const int p0 = (int)min(cut.piece_of(begin + kItem), (unsigned)last);
  const int p1 = (int)min(cut.piece_of(begin + w.units() - 1), (unsigned)last);
  pdl_wait();
  if (p0 >= p1) return;  // written by its piece
  const int np = p1 - p0 + 1, cols = min(kCols, it.n * P.G - it.ct * kCols);
  // part of piece p0 + p: it begins the item in its second slot
  auto part = [&](int p) {
    return P.part + (long long)(2 * (p0 + p) + (p == 0)) * kCols * (D + 2);
  };
  // A thread an output, a warp within one column (of this CTA's share of the
  // dims); few outputs: several groups of warps share the pieces.
  const int dims = D / gridDim.z, outs = cols * dims;
  const int groups = max(1, min(np, kMergeThreads / outs));
  const int width = groups == 1 ? kMergeThreads : outs, grp = tid / width;
  for (int i = tid - grp * width; i < outs; i += width) {
    const int n = i / dims, d = blockIdx.z * dims + i % dims;
    float O = 0.f;
    if (grp < groups) {
      // lane p: piece p's factor
      const float m = lane < np ? __ldcg(part(lane) + n) : -FLT_MAX;
      const float l = lane < np ? __ldcg(part(lane) + kCols + n) : 0.f;
      float M = m;
      for (int p = 32 + lane; p < np; p += 32) M = fmaxf(M, __ldcg(part(p) + n));
      M = warp_max(M);
      float a = lane < np ? ex2(m - M) : 0.f, L = a * l;
      for (int p = 32 + lane; p < np; p += 32)
        L = fmaf(ex2(__ldcg(part(p) + n) - M), __ldcg(part(p) + kCols + n), L);
      L = warp_sum(L);
      for (int p = grp, from = 0; p < np; from += 32) {
        if (from) a = from + lane < np ? ex2(__ldcg(part(from + lane) + n) - M) : 0.f;
        const int to = min(np, from + 32);
#pragma unroll 8
        for (; p < to; p += groups)
          O = fmaf(__shfl_sync(0xffffffffu, a, p - from), __ldcg(part(p) + 2 * kCols + n * D + d), O);
      }
      O = L != 0.f ? O / L : 0.f;
    }
    if (groups > 1) {
      acc[tid] = O;
      __syncthreads();
      if (grp == 0)
        for (int g = 1; g < groups; ++g) O += acc[g * width + i];
    }
    if (grp == 0) store_out(P, out_row(P, it, it.ct * kCols + n), d, D, O);
  }
}

// ---------------------------------------------------------------- launches --

template <int D, bool I8, int QS, int PS>
cudaError_t launch_cluster(const Params& P, int z, cudaStream_t st) {
  const size_t smem = (size_t)kWarps * kCols * (D + 2) * 4 + (size_t)kCols * D * QS * 2;
  const auto kernel = cluster_kernel<D, I8, QS, PS>;
  ensure_smem((const void*)kernel, (int)smem);
  Params Q = P;
  Q.pieces = z;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((long long)P.T * P.G / kCols + P.B) * z), P.Hkv);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = z;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = z > 1 ? 2 : 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, kernel, Q);
}

template <int D, bool I8, int QS, int PS>
cudaError_t launch_split(const Params& P, cudaStream_t st) {
  const size_t smem = (size_t)kWarps * kCols * (D + 2) * 4 + (size_t)kCols * D * QS * 2;
  ensure_smem((const void*)split_kernel<D, I8, QS, PS>, (int)smem);
  cudaError_t e = launch_pdl(split_kernel<D, I8, QS, PS>, dim3(P.pieces), dim3(kWarps * 32),
                             smem, st, true, P);
  if (e != cudaSuccess || P.pieces == 1) return e;
  const long long slots = (long long)P.T * P.G / kCols + P.B;
  // few items: their dims over several CTAs, so that a thread has few pieces
  unsigned parts = 1;  // of the dims
  while (parts * 2 <= D / 64 && slots * P.Hkv * parts * 2 <= 2 * num_sms()) parts *= 2;
  return launch_pdl(merge_kernel<D>, dim3((unsigned)slots, P.Hkv, parts), dim3(kMergeThreads), 0,
                    st, true, P);
}

// How a call runs: by the prompt kernel, by z CTAs an item, or in pieces of the
// line (-1: it has over 31 bits).
struct Plan {
  bool prompt;
  int z, pieces;
};
inline Plan plan(int B, int T, int H, int Hkv, int D, bool i8, long long cap, bool exact) {
  const long long G = H / Hkv;
  // at most: a sequence of n rows has n G / 8 column tiles, rounded up
  const long long items = std::min(T * G / kCols + B, T * ((G + kCols - 1) / kCols)) * Hkv;
  const long long chunks = std::max(1LL, (cap + kChunk - 1) / kChunk);
  const long long most =
      std::min((long long)kMaxPieces, (long long)num_sms() * split_ctas(D, i8));
  const long long even = (items * chunks + most - 1) / most;  // chunks a piece
  // More than 8 columns a sequence: its keys are read once for each 8, or once
  // for 128 by the prompt kernel, which takes some 14 us before it has to stream.
  // The first where a piece has few chunks, and few items or long ones (8 KV
  // heads, int8 of 128 unless stated, this against that, us: 4 x 12 rows over 1000
  // tokens 14 / 17, 1 x 100 over 700 15 / 19, 16 x 6 over 2000 26 / 33, 12 rows each
  // 36 / 34; 4 x 12 rows of bf16 over 3000 19 / 30; 1 x 64 over 32768 179 / 135; 1 x
  // 300 over 300 27 / 15, 30 x 6 over 300 26 / 19). Two column tiles a warp in
  // place of one were slower than both (4 x 12 rows 19, 16 x 6 rows 50).
  if (D <= 128 && !exact && T * G > kCols * (long long)B &&
      !(even <= 21 && (items <= num_sms() || chunks >= 6)))
    return {true, 0, 0};
  if (items > 0x7FFFFFFFLL / (chunks + kItem)) return {false, 0, -1};
  // Clusters where an item's equal shares are little longer than the balanced
  // pieces would be (should the sequences fill their pages): up to two chunks
  // cost less than the second launch. Past 8 chunks a share only without a
  // cluster, whose CTAs wait for the slowest. Measured against the line and its
  // merge (us, 8 int8 KV heads of 128, 2 query heads each): 1 x 512 7.8 -> 6.5,
  // 4 x 2048 13.4 -> 10.3, 32 x 2048 33.6 -> 30.4; shares four chunks longer, 8 x
  // 8192, 29.1 -> 31; more CTAs than the GPU holds at once, 4 x 700 of 16 rows
  // in all, 11.2 -> 14.8.
  // (nor where most sequences are empty: each CTA looks through them)
  if (items <= most && B <= 4 * T) {
    // (one CTA an SM: clusters leave some of a GPC's SMs empty)
    const long long room = split_ctas(D, i8) == 1 ? most * 3 / 4 : most;
    int z = 1;
    while (z < kMaxZ && z < chunks && items * 2 * z <= room) z *= 2;
    const long long share = (chunks + z - 1) / z;
    if (share <= even + kSlack && (z == 1 || share <= 8)) return {false, z, 0};
  }
  return {false, 0, (int)std::max(1LL, std::min(most, items * chunks))};
}

template <int D, bool I8>
cudaError_t launch(const Params& P, const Plan& p, bool exact, cudaStream_t st) {
  constexpr int E = I8 ? 2 : 3, W = I8 ? 1 : 2;  // terms of fp32 q and weights; of the weights
  if (p.prompt) return launch_prompt(P, D, I8, st);
  if (exact)
    return p.z ? launch_cluster<D, I8, E, E>(P, p.z, st) : launch_split<D, I8, E, E>(P, st);
  return p.z ? launch_cluster<D, I8, 1, W>(P, p.z, st) : launch_split<D, I8, 1, W>(P, st);
}

// The largest number of pieces times columns any call of the head size uses.
inline size_t ws_bytes(int D) {
  return (size_t)2 * num_sms() * 2 * 8 * (D + 2) * 4;
}

}  // namespace pa
}  // namespace qg

using namespace qg;

extern "C" size_t qg_paged_attention_workspace_size(int head_dim) {
  if (head_dim <= 0 || head_dim > 256) return 0;
  return pa::ws_bytes(head_dim);
}

extern "C" qg_status qg_paged_attention(const qg_paged_kv* kv, const int32_t* page_table,
                                        int max_pages, const int32_t* kv_len,
                                        const int32_t* row_start, const void* q, qg_dtype q_dtype,
                                        void* out, qg_dtype out_dtype, int B, int T, int H,
                                        float scale, void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  const char* who = "qg_paged_attention";
  if (qg_status s = pk::check_pool(who, kv, max_pages)) return s;
  const int D = kv->head_dim, Hkv = kv->kv_heads;
  QG_REQUIRE(B >= 0 && T >= 0 && H >= 1 && H <= 8192, QG_ERR_UNSUPPORTED_SHAPE,
             "%s: B=%d T=%d H=%d", who, B, T, H);
  QG_REQUIRE(H % Hkv == 0, QG_ERR_UNSUPPORTED_SHAPE, "%s: H=%d must be a multiple of kv_heads=%d",
             who, H, Hkv);
  QG_REQUIRE(B <= (1 << 16) && (long long)T * H <= (1LL << 30), QG_ERR_UNSUPPORTED_SHAPE,
             "%s: B=%d T=%d H=%d too large", who, B, T, H);
  QG_REQUIRE(row_start || T == B, QG_ERR_UNSUPPORTED_SHAPE,
             "%s: T=%d rows without row_start must be B=%d", who, T, B);
  QG_REQUIRE((q_dtype == QG_F32 || q_dtype == QG_BF16) &&
                 (out_dtype == QG_F32 || out_dtype == QG_BF16),
             QG_ERR_INVALID_ARGUMENT, "%s: q_dtype=%d out_dtype=%d", who, (int)q_dtype,
             (int)out_dtype);
  QG_REQUIRE(scale > 0.f && scale <= 3.402823466e38f, QG_ERR_INVALID_ARGUMENT,
             "%s: scale must be positive and finite", who);
  QG_REQUIRE((long long)kv->num_pages * Hkv * (kv->page_size / pk::kBlock) <= 0x7FFFFFFFLL,
             QG_ERR_UNSUPPORTED_SHAPE, "%s: num_pages=%d: the pool is too large", who,
             kv->num_pages);
  if (B == 0 || T == 0) return QG_OK;
  const bool exact = q_dtype == QG_F32 || out_dtype == QG_F32;
  const pa::Plan plan =
      pa::plan(B, T, H, Hkv, D, kv->dtype == QG_KV_INT8, (long long)max_pages * kv->page_size, exact);
  QG_REQUIRE(plan.pieces >= 0, QG_ERR_UNSUPPORTED_SHAPE,
             "%s: T=%d rows of H=%d heads over max_pages=%d pages are too many for one call", who,
             T, H, max_pages);
  if (qg_status s = pk::check_pool_pointers(who, kv)) return s;
  QG_REQUIRE(page_table && kv_len && q && out, QG_ERR_INVALID_ARGUMENT,
             "%s: null page_table, kv_len, q or out", who);
  QG_REQUIRE(aligned(q, 16) && aligned(out, 16), QG_ERR_MISALIGNED,
             "%s: q or out not 16-byte aligned", who);
  QG_REQUIRE(aligned(page_table, 4) && aligned(kv_len, 4) && aligned(row_start, 4),
             QG_ERR_MISALIGNED, "%s: page_table, kv_len or row_start misaligned", who);
  const size_t need = pa::ws_bytes(D);
  QG_REQUIRE(ws && ws_bytes >= need, QG_ERR_WORKSPACE_TOO_SMALL,
             "%s: workspace of %zu bytes given, %zu needed", who, ws_bytes, need);
  QG_REQUIRE(aligned(ws, 256), QG_ERR_MISALIGNED, "%s: ws not 256-byte aligned", who);
  pa::Params P = {};
  P.q = q;
  P.out = out;
  P.kp = reinterpret_cast<const uint8_t*>(kv->k_pages);
  P.vp = reinterpret_cast<const uint8_t*>(kv->v_pages);
  P.ks = kv->k_scales;
  P.vs = kv->v_scales;
  P.table = page_table;
  P.kv_len = kv_len;
  P.row_start = row_start;
  P.part = reinterpret_cast<float*>(ws);
  P.q_bf16 = q_dtype == QG_BF16;
  P.out_bf16 = out_dtype == QG_BF16;
  P.B = B;
  P.T = T;
  P.H = H;
  P.Hkv = Hkv;
  P.G = H / Hkv;
  P.bpp = kv->page_size / pk::kBlock;
  P.max_pages = max_pages;
  P.num_pages = kv->num_pages;
  P.pieces = plan.pieces;
  P.scale_log2 = (float)((double)scale * 1.4426950408889634);
  const bool i8 = kv->dtype == QG_KV_INT8;
  cudaStream_t st = (cudaStream_t)stream;
  if (D == 64)
    i8 ? pa::launch<64, true>(P, plan, exact, st) : pa::launch<64, false>(P, plan, exact, st);
  else if (D == 128)
    i8 ? pa::launch<128, true>(P, plan, exact, st) : pa::launch<128, false>(P, plan, exact, st);
  else
    i8 ? pa::launch<256, true>(P, plan, exact, st) : pa::launch<256, false>(P, plan, exact, st);
  return check_launch(who);
}
