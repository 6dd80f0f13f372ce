// Filtered sampling (include/qg.h, qg_sample_filtered): temperature, top-k,
// top-p, min-p and a draw from a given uniform number, each row with
// parameters of its own, in one launch without a sort.
//
// All three filters keep a prefix of the candidates in descending order
// (equal values by index), and the draw is the place in that prefix where
// the running weight reaches u times the prefix's weight. So everything is
// one operation: find the candidate at which a running count, or a running
// weight, reaches a target. A histogram of (count, weight) over 2048 bins
// that are monotone in the value answers it up to one bin; the members of the
// few bins that can matter are collected in one more pass and sorted. With a small top-k only counts go into the histogram, and weights
// are formed for the members of the first bins alone.
//
// A row belongs to a cluster of CTAs, each holding a slice of it in shared
// memory: the row is read from HBM once, and the cluster's histograms and
// members meet in rank 0 through distributed shared memory.
//
// Weights are exp((l - max) / T) in float64, rounded to fixed point (2^-44
// of the largest for V near 152 thousand): integer sums do not depend on the
// order of the atomics, so results are the same each time, and a border is
// where float64 puts it up to 2^-45 a candidate. fp32 weights would move
// borders by 2^-24 of the total, more than a rare token's whole weight.
//
// What bounds it: one row, the chain of phases (151936 values over 16 CTAs, 46
// thousand cycles: reading 6, weights and histogram 11, its sums through
// distributed shared memory 7, border bins 5, collection 8, sort and search 6,
// the rest barriers); full batches, four shared-memory atomics and a float64 exp
// a value (32 rows of 151936 over 128 CTAs, 52 us: 20 of them). 24-29 us a row, by
// how many members the border bins have, 160 rows of 2048 13.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstddef>

#include "qg_internal.cuh"

namespace qg {
namespace sf {

constexpr int kBins = 2048;
constexpr int kFine = 1536;         // bins for the values whose weight is not 0
constexpr int kList = 512;          // members that rank 0 can hold at most (one a thread)
constexpr int kMaxCluster = 16;
constexpr int kResident = 37984;    // values of a slice that shared memory holds
constexpr int kSumRoom = 65536;     // 16-bit pieces whose sum 32 bits hold
constexpr int kSteps = 64;          // entries of the table of 2^(i / kSteps)

typedef unsigned long long u64;

struct Params {
  const float* logits;
  long long ld;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int32_t* out;
  int32_t* kept;
  float* logprob;
  int V, slice, resident, frac;  // frac: fraction bits of a fixed-point weight
  double pow2[kSteps];
};

enum Op { kDone, kCollect, kMinMax, kHist, kWeights };
struct Cmd {
  int op, bin, shift;
  u64 lo, hi;
};

// A place in the descending order: candidates before it, running weight with
// it, its key; or, for a bin: what lies before it, and what it holds.
struct Found {
  u64 rank, cum, key;
};
struct Bin {
  int at;
  u64 pc, pw, c, w;
};

struct Shared {
  u64 key_max[kMaxCluster], key_min[kMaxCluster];  // pushed by every rank
  unsigned count[kMaxCluster], above[kMaxCluster]; // candidates; weights >= min_p
  Cmd cmd;
  unsigned wanted[kBins / 32];  // bins to collect
  unsigned list_n;
  u64 red[32], red2[32];
  unsigned red3[32];
  double pow2[kSteps];
  u64 mine[kList];                       // this CTA's members of a collection
  unsigned mine_n, mine_at;              // how many, and where they go in rank 0's list
  int path;                              // rank 0: how the row goes on
  u64 list_key[kList], list_w[kList];    // rank 0's list: sorted keys, running weights
  // rank 0: the cluster's counts and weights by bin, and what lies before
  // each group of 32 bins (the whole at the end)
  u64 tot_w[kBins], sup_w[kBins / 32 + 1];
  unsigned tot_c[kBins], sup_c[kBins / 32 + 1];
  // this CTA's histogram: counts, and weights in pieces of 16, 16 and 12 bits,
  // whose sums over kSumRoom values fit 32 bits (see each_adding): atomics that
  // return nothing (a 64-bit one costs several, and two halves would need the
  // carry back)
  unsigned hist_c[kBins], hist_w0[kBins], hist_w1[kBins], hist_w2[kBins];
};
// Inside one bin (rank 0, rare): lies over the list.
constexpr int kSubBins = 512;
struct Sub {
  u64 w[kSubBins];
  unsigned c[kSubBins];
};
static_assert(sizeof(Shared) + kResident * 4 <= 227 * 1024, "a slice fits beside Shared");
static_assert(sizeof(Sub) <= 2 * kList * sizeof(u64), "Sub lies over list_key and list_w");

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
               "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote_at(uint32_t local, unsigned rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t remote(const void* p, unsigned rank) {
  return remote_at(static_cast<uint32_t>(__cvta_generic_to_shared(p)), rank);
}
__device__ __forceinline__ void st_u64(uint32_t a, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ void st_u32(uint32_t a, unsigned v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ u64 ld_u64(uint32_t a) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ unsigned ld_u32(uint32_t a) {
  unsigned v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ unsigned add_u32(uint32_t a, unsigned v) {
  unsigned r;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(r) : "r"(a), "r"(v) : "memory");
  return r;
}

// Order of the candidates as one integer: larger value first, then smaller
// index. 0 for a value that is no candidate (NaN, -inf).
__device__ __forceinline__ u64 key_of(float v, int i) {
  if (!(v > -INFINITY)) return 0;
  unsigned bits = __float_as_uint(v == 0.f ? 0.f : v);
  bits = (bits & 0x80000000u) ? ~bits : (bits | 0x80000000u);
  return ((u64)bits << 32) | (0xFFFFFFFFu - (unsigned)i);
}
__device__ __forceinline__ float value_of(u64 k) {
  const unsigned bits = (unsigned)(k >> 32);
  return __uint_as_float((bits & 0x80000000u) ? (bits & 0x7FFFFFFFu) : ~bits);
}
__device__ __forceinline__ int index_of(u64 k) { return (int)(0xFFFFFFFFu - (unsigned)k); }

__device__ __forceinline__ u64 warp_max64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ u64 warp_min64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = min(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Sum over the warp in three parts of 26, 26 and 12 bits (the parts' sums
// fit 32 bits).
__device__ __forceinline__ u64 warp_sum64(u64 v) {
  const u64 a = __reduce_add_sync(0xffffffffu, (unsigned)v & 0x3FFFFFFu);
  const u64 b = __reduce_add_sync(0xffffffffu, (unsigned)(v >> 26) & 0x3FFFFFFu);
  const u64 c = __reduce_add_sync(0xffffffffu, (unsigned)(v >> 52));
  return a + (b << 26) + (c << 52);
}

__device__ __forceinline__ void add_weight(Shared& S, int b, u64 w) {
  atomicAdd(&S.hist_w0[b], (unsigned)w & 0xFFFFu);
  if (w >> 16) atomicAdd(&S.hist_w1[b], (unsigned)(w >> 16) & 0xFFFFu);
  if (w >> 32) atomicAdd(&S.hist_w2[b], (unsigned)(w >> 32));
}

// The row's bins and weights.
struct Row {
  float top;       // the largest value
  double per_unit; // 64 / (ln2 T)
  int frac;        // fraction bits of a weight
  float reach;     // values further below the maximum have weight 0
  float fine, coarse, edge;  // bins: d * fine up to d = edge, then (d - edge) * coarse
  const double* pow2;

  // (l - max) / T in steps of ln2 / 64: 0 for the maximum itself (+inf too).
  __device__ __forceinline__ double steps(float v) const {
    const double x = ((double)v - (double)top) * per_unit;  // (the difference is exact)
    return v == top ? 0.0 : x;
  }
  // 2^(x / 64 + up) for x <= 0, the result above 2^-1022: table-driven (Tang, "Table-driven
  // implementation of the exponential function", 1989): x = n + f with n an
  // integer, 2^(n / 64) from the table of 64 and the exponent, e^(f ln2 / 64)
  // by its series up to the fifth power (the next term is below 2^-54).
  __device__ __forceinline__ double power(double x, int up) const {
    const double magic = 6755399441055744.0;  // 1.5 * 2^52: the sum rounds to an integer
    const double t = x + magic;
    const int k = __double2loint(t);
    const double f = x - (t - magic);
    constexpr double c = 0.010830424696249145;  // ln2 / 64
    double p = fma(f, c * c * c * c * c / 120, c * c * c * c / 24);
    p = fma(p, f, c * c * c / 6);
    p = fma(p, f, c * c / 2);
    p = fma(p, f, c) * f;
    const double s = pow2[k & (kSteps - 1)];
    const double y = fma(s, p, s);
    return __hiloint2double(__double2hiint(y) + (((k >> 6) + up) << 20), __double2loint(y));
  }
  // A candidate's weight for min-p, whose least positive value is 2^-149: as it
  // is down to 2^-1020, also where it is 0 in fixed point.
  __device__ __forceinline__ double weight(float v) const {
    return power(fmax(steps(v), -1020.0 * kSteps), 0);
  }
  // Whether v's weight can be more than 0.
  __device__ __forceinline__ bool weighs(float v) const {
    return v == top || (top - v <= reach && v > -INFINITY);
  }
  // power(x, frac) and the weight in units of 2^-frac: the sum with 2^52
  // rounds it.
  __device__ __forceinline__ u64 fixed_of(float v, double* y) const {
    const bool in = weighs(v);
    *y = power(in ? steps(v) : 0.0, frac);
    const u64 w = (u64)__double_as_longlong(*y + 4503599627370496.0) & 0xFFFFFFFFFFFFFull;
    return in ? w : 0;
  }
  __device__ __forceinline__ u64 fixed(float v) const {
    double y;
    return fixed_of(v, &y);
  }
  // Monotone in v: each step (difference, product, minimum, and the sum with
  // 2^23 that rounds to an integer) is.
  __device__ __forceinline__ int bin(float v) const {
    const float d = top - v;
    const float near = fminf(d * fine, (float)(kFine - 1));
    const float far = fminf((d - edge) * coarse, (float)(kBins - kFine - 1)) + (float)kFine;
    const int b = __float_as_int((d <= edge ? near : far) + 8388608.f) & (kBins - 1);
    return v == top ? 0 : b;
  }
};

// What a CTA of the cluster works on.
template <int NTHR>
struct Work {
  const Params& P;
  Shared& S;
  const Row row_;
  const float* data;
  const float* row;
  int begin, n;
  unsigned rank, C;

  // f(four values, index of the first) for places first .. last - 1 of the
  // slice, the indexes NTHR apart; -inf past them. Four at once, so that f can
  // form what it needs of all of them before it branches: their chains hide each
  // other's latency.
  template <class F>
  __device__ __forceinline__ void each(F f, int first, int last) const {
    const float* const from = P.resident ? data : row + begin;
    const int at = begin;  // (in registers, whatever f does to memory)
#pragma unroll 1
    for (int i = first + threadIdx.x; i < last; i += 4 * NTHR) {
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = i + e * NTHR < last ? from[i + e * NTHR] : -INFINITY;
      f(v, at + i);
    }
  }
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    each(f, 0, n);
  }

  // The whole slice for an f that adds weights to the histogram. A piece's sum
  // holds 65536 members of one bin; a slice of more (V past 2^20) goes in parts
  // of half as many, after each of which the sums' upper halves move up.
  template <class F>
  __device__ __forceinline__ void each_adding(F f) const {
    const int part = n <= kSumRoom ? kSumRoom : kSumRoom / 2;
#pragma unroll 1
    for (int at = 0; at < n; at += part) {
      each(f, at, min(n, at + part));
      if (n > part) {
        __syncthreads();
        for (int i = threadIdx.x; i < kBins; i += NTHR) {
          const unsigned lo = S.hist_w0[i], mid = S.hist_w1[i] + (lo >> 16);
          S.hist_w0[i] = lo & 0xFFFFu;
          S.hist_w1[i] = mid & 0xFFFFu;
          S.hist_w2[i] += mid >> 16;
        }
        __syncthreads();
      }
    }
  }

  __device__ __forceinline__ void sync() const {
    if (C == 1)
      __syncthreads();
    else
      cluster_sync();
  }

  __device__ __forceinline__ u64 own_weight(int b) const {
    return (u64)S.hist_w0[b] + ((u64)S.hist_w1[b] << 16) + ((u64)S.hist_w2[b] << 32);
  }

  // The cluster's sums of the CTAs' histograms into rank 0's (c, w), each rank
  // a share of the bins, and the sums of groups of 32 bins.
  __device__ __forceinline__ void sum_bins(int bins, unsigned* c, u64* w) const {
    const int per = bins / C;  // a multiple of 32
    for (int i = threadIdx.x; i < per; i += NTHR) {
      const int b = rank * per + i;
      unsigned nc = S.hist_c[b];
      u64 nw = w ? own_weight(b) : 0;
      if (C > 1) {
        nc = 0;
        nw = 0;
        const uint32_t ac = static_cast<uint32_t>(__cvta_generic_to_shared(&S.hist_c[b]));
        constexpr uint32_t next = kBins * 4;  // the four arrays follow each other
#pragma unroll 4
        for (unsigned r = 0; r < C; ++r) {
          const uint32_t a = remote_at(ac, r);
          nc += ld_u32(a);
          if (w)
            nw += (u64)ld_u32(a + next) + ((u64)ld_u32(a + 2 * next) << 16) +
                  ((u64)ld_u32(a + 3 * next) << 32);
        }
      }
      st_u32(remote(&c[b], 0), nc);
      if (w) st_u64(remote(&w[b], 0), nw);
      nc = __reduce_add_sync(0xffffffffu, nc);
      nw = warp_sum64(nw);
      if ((threadIdx.x & 31) == 0) {
        st_u32(remote(&S.sup_c[b / 32], 0), nc);
        if (w) st_u64(remote(&S.sup_w[b / 32], 0), nw);
      }
    }
  }

  // This thread's candidates with a weight of at least min_p: the CTA's sum to
  // rank 0.
  __device__ __forceinline__ void push_above(unsigned above) const {
    above = __reduce_add_sync(0xffffffffu, above);
    if ((threadIdx.x & 31) == 0) S.red3[threadIdx.x >> 5] = above;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < NTHR / 32; ++i) above += S.red3[i];
      st_u32(remote(&S.above[rank], 0), above);
    }
  }

  // The slice's weights (and, with `count`, counts) into the histogram.
  __device__ __forceinline__ void weigh(const Row& R, double min_p, bool count) const {
    unsigned above = 0;
    // (a weight of at least this is not 0 in fixed point)
    const double least = __hiloint2double((1023 - R.frac) << 20, 0);
    each_adding([&](const float (&v)[4], int) {
      int b[4];
      u64 w[4];
      double y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        b[e] = R.bin(v[e]);
        w[e] = R.fixed_of(v[e], &y[e]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (count && v[e] > -INFINITY) atomicAdd(&S.hist_c[b[e]], 1u);
        if (w[e]) add_weight(S, b[e], w[e]);
      }
      if (min_p >= least) {  // (scaling by 2^frac is exact: this is power(x, 0) >= min_p)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          above += w[e] && __hiloint2double(__double2hiint(y[e]) - (R.frac << 20),
                                            __double2loint(y[e])) >= min_p;
      } else if (min_p > 0.0) {
#pragma unroll 1
        for (int e = 0; e < 4; ++e) {
          const float x = e == 0 ? v[0] : e == 1 ? v[1] : e == 2 ? v[2] : v[3];
          above += x > -INFINITY && R.weight(x) >= min_p;
        }
      }
    });
    if (min_p > 0.0) push_above(above);
  }

  // One collective step of the cluster.
  __device__ __noinline__ void serve(double min_p) const {
    const Row R = row_;
    const Cmd c = S.cmd;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (c.op == kCollect) {  // members of the wanted bins whose keys lie in [lo, hi]
      // the CTA's own first, then all of them at once to rank 0
      if (tid == 0) S.mine_n = 0;
      __syncthreads();
      each([&](const float (&v)[4], int i) {
        unsigned hit = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int b = R.bin(v[e]);
          hit |= (S.wanted[b >> 5] >> (b & 31) & 1) << e;
        }
        if (!hit) return;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const u64 k = key_of(v[e], i + e * NTHR);
          if ((hit >> e & 1) && k != 0 && k >= c.lo && k <= c.hi) {
            const unsigned at = atomicAdd(&S.mine_n, 1u);
            if (at < NTHR) S.mine[at] = k;
          }
        }
      });
      __syncthreads();
      const unsigned m = S.mine_n;
      if (tid == 0) S.mine_at = add_u32(remote(&S.list_n, 0), m);
      __syncthreads();
      const unsigned at = S.mine_at + tid;
      if (tid < (int)min(m, (unsigned)NTHR) && at < NTHR)
        st_u64(remote(&S.list_key[at], 0), S.mine[tid]);
    } else if (c.op == kMinMax) {  // of the bin's keys
      u64 lo = ~0ull, hi = 0;
      each([&](const float (&v)[4], int i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (!(v[e] > -INFINITY) || R.bin(v[e]) != c.bin) continue;
          const u64 k = key_of(v[e], i + e * NTHR);
          lo = min(lo, k);
          hi = max(hi, k);
        }
      });
      lo = warp_min64(lo);
      hi = warp_max64(hi);
      if (lane == 0) {
        S.red[warp] = lo;
        S.red2[warp] = hi;
      }
      __syncthreads();
      if (tid == 0) {
        for (int i = 1; i < NTHR / 32; ++i) {
          lo = min(lo, S.red[i]);
          hi = max(hi, S.red2[i]);
        }
        st_u64(remote(&S.key_min[rank], 0), lo);
        st_u64(remote(&S.key_max[rank], 0), hi);
      }
    } else if (c.op == kWeights) {  // the whole row's weights by bin
      weigh(R, min_p, false);
      sync();
      sum_bins(kBins, S.tot_c, S.tot_w);
    } else {  // kHist: the bin's keys in [lo, hi] by their distance to hi
      for (int i = tid; i < kSubBins; i += NTHR) {
        S.hist_c[i] = 0;
        S.hist_w0[i] = S.hist_w1[i] = S.hist_w2[i] = 0;
      }
      __syncthreads();
      each_adding([&](const float (&v)[4], int i) {
#pragma unroll 1
        for (int e = 0; e < 4; ++e) {
          const float x = e == 0 ? v[0] : e == 1 ? v[1] : e == 2 ? v[2] : v[3];
          const u64 k = key_of(x, i + e * NTHR);
          if (!(x > -INFINITY) || R.bin(x) != c.bin || k < c.lo || k > c.hi) continue;
          const int b = (int)((c.hi - k) >> c.shift);
          atomicAdd(&S.hist_c[b], 1u);
          const u64 w = R.fixed(x);
          if (w) add_weight(S, b, w);
        }
      });
      sync();
      Sub& sub = *reinterpret_cast<Sub*>(S.list_key);
      sum_bins(kSubBins, sub.c, sub.w);
    }
    sync();
  }

  // Rank 0: one collective step (every thread calls it).
  __device__ __forceinline__ void ask(const Cmd& c, double min_p) const {
    __syncthreads();
    if (threadIdx.x == 0) S.list_n = 0;
    if (threadIdx.x < C) {
      const uint32_t a = remote(&S.cmd, threadIdx.x);
      st_u32(a + offsetof(Cmd, op), c.op);
      st_u32(a + offsetof(Cmd, bin), c.bin);
      st_u32(a + offsetof(Cmd, shift), c.shift);
      st_u64(a + offsetof(Cmd, lo), c.lo);
      st_u64(a + offsetof(Cmd, hi), c.hi);
    }
    if (c.op == kCollect)
      for (unsigned i = threadIdx.x; i < (C - 1) * (kBins / 32); i += NTHR)
        st_u32(remote(&S.wanted[i % (kBins / 32)], 1 + i / (kBins / 32)),
               S.wanted[i % (kBins / 32)]);
    sync();
    if (c.op != kDone) serve(min_p);
  }

  // Warp 0 of rank 0: the groups' sums into what lies before each.
  __device__ __forceinline__ void scan_groups(int bins) const {
    const int lane = threadIdx.x & 31, groups = bins / 32;  // at most 64: two a lane
    const unsigned c0 = 2 * lane < groups ? S.sup_c[2 * lane] : 0;
    const unsigned c1 = 2 * lane < groups ? S.sup_c[2 * lane + 1] : 0;
    const u64 w0 = 2 * lane < groups ? S.sup_w[2 * lane] : 0;
    const u64 w1 = 2 * lane < groups ? S.sup_w[2 * lane + 1] : 0;
    unsigned xc = c0 + c1;
    u64 xw = w0 + w1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned yc = __shfl_up_sync(0xffffffffu, xc, o);
      const u64 yw = __shfl_up_sync(0xffffffffu, xw, o);
      if (lane >= o) {
        xc += yc;
        xw += yw;
      }
    }
    if (2 * lane < groups) {
      S.sup_c[2 * lane + 1] = xc - c1;
      S.sup_c[2 * lane + 2] = xc;
      S.sup_w[2 * lane + 1] = xw - w1;
      S.sup_w[2 * lane + 2] = xw;
    }
    __syncwarp();
    if (lane == 0) {
      S.sup_c[0] = 0;
      S.sup_w[0] = 0;
    }
    __syncwarp();
  }

  // Warp 0 of rank 0: the bin where the running count passes the target
  // (by_weight: where the running weight reaches it).
  __device__ __noinline__ Bin find_bin(int bins, const unsigned* c, const u64* w, bool by_weight,
                                       u64 target) const {
    const int lane = threadIdx.x & 31, groups = bins / 32;
    const u64 t = by_weight ? target - 1 : target;
    // groups that begin at or before t: the last one holds it
    const int g0 = lane, g1 = lane + 32;
    const bool in0 = g0 < groups && (by_weight ? S.sup_w[g0] : S.sup_c[g0]) <= t;
    const bool in1 = g1 < groups && (by_weight ? S.sup_w[g1] : S.sup_c[g1]) <= t;
    int g = __popc(__ballot_sync(0xffffffffu, in0)) + __popc(__ballot_sync(0xffffffffu, in1)) - 1;
    // (empty groups share their start with the next one, and come before it)
    const unsigned mc = c[g * 32 + lane];
    const u64 mw = w[g * 32 + lane];
    unsigned xc = mc;
    u64 xw = mw;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned yc = __shfl_up_sync(0xffffffffu, xc, o);
      const u64 yw = __shfl_up_sync(0xffffffffu, xw, o);
      if (lane >= o) {
        xc += yc;
        xw += yw;
      }
    }
    const u64 ic = S.sup_c[g] + xc, iw = S.sup_w[g] + xw;
    const unsigned m = __ballot_sync(0xffffffffu, (by_weight ? iw : ic) > t);
    const int l = m ? __ffs(m) - 1 : 31;
    Bin b;
    b.at = g * 32 + l;
    b.pc = __shfl_sync(0xffffffffu, ic - mc, l);
    b.pw = __shfl_sync(0xffffffffu, iw - mw, l);
    b.c = __shfl_sync(0xffffffffu, mc, l);
    b.w = __shfl_sync(0xffffffffu, mw, l);
    return b;
  }

  // Warp 0: the first of n places for which f holds (n if none; f changes once).
  template <class F>
  __device__ __forceinline__ unsigned first_of(unsigned n, F f) const {
    const unsigned lane = threadIdx.x & 31;
    unsigned base = 0;
    if (n == 0) return 0;
    if (n > 32) {  // groups of 32 (at most 32 of them) by their last place
      const unsigned m = __ballot_sync(0xffffffffu, f(min(lane * 32 + 31, n - 1)));
      base = m ? 32 * (__ffs(m) - 1) : n - 1;
    }
    const unsigned q = min(base + lane, n - 1);
    const unsigned m = __ballot_sync(0xffffffffu, f(q));
    return m ? min(base + __ffs(m) - 1, n - 1) : n;
  }

  // A place in the list's part of a bin.
  __device__ __forceinline__ Found in_list(const Bin& b, unsigned start, unsigned n, bool by_weight,
                                           u64 target) const {
    const u64 base = start ? S.list_w[start - 1] : 0;
    const unsigned q =
        start + (by_weight ? first_of(n - start,
                                      [&](unsigned i) {
                                        return S.list_w[start + i] - base + b.pw >= target;
                                      })
                           : (unsigned)(target - b.pc));
    const unsigned at = min(q, max(n, 1u) - 1);
    return Found{b.pc + (at - start), S.list_w[at] - base + b.pw, S.list_key[at]};
  }

  // Sorts the list's n keys, largest first, one a thread (bitonic; strides
  // below a warp by shuffles, the others through the list's two arrays in
  // turn), and forms the running weights.
  __device__ __noinline__ void sort_list(unsigned n) const {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Row R = row_;
    u64 k = tid < (int)n ? S.list_key[tid] : 0;
    u64* buf[2] = {S.list_w, S.list_key};
    int turn = 0;
    if (n > 32 || warp == 0) {
#pragma unroll 1
      for (unsigned size = 2; size < 2 * n; size <<= 1) {
#pragma unroll 1
        for (unsigned stride = size >> 1; stride > 0; stride >>= 1) {
          u64 o;
          if (stride < 32) {
            o = __shfl_xor_sync(0xffffffffu, k, stride);
          } else {
            buf[turn][tid] = k;
            __syncthreads();
            o = buf[turn][tid ^ stride];
            turn ^= 1;
          }
          const bool larger = ((tid & stride) == 0) == ((tid & size) == 0);
          k = larger ? max(k, o) : min(k, o);
        }
      }
    }
    u64 x = k ? R.fixed(value_of(k)) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) S.red[warp] = x;
    __syncthreads();
    const u64 before = warp_sum64(lane < warp ? S.red[lane] : 0);
    S.list_key[tid] = k;
    S.list_w[tid] = x + before;
    __syncthreads();
  }
};

// f of a weight, at least 1, at most all of it.
__device__ __noinline__ u64 share(double f, u64 total) {
  const double t = ceil(fmin(fmax(f, 0.0), 1.0) * (double)total);
  return max((u64)1, min(total, __double2ull_rn(t)));
}

template <int NTHR>
__global__ void __launch_bounds__(NTHR, 512 / NTHR) sample_kernel(const __grid_constant__ Params P) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& S = *reinterpret_cast<Shared*>(smem);
  float* data = reinterpret_cast<float*>(smem + sizeof(Shared));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned C = gridDim.x, rank = cluster_rank();
  const int b = blockIdx.y;
  const int begin = min(P.V, (int)rank * P.slice), n = min(P.slice, P.V - begin);
  const float* row = P.logits + (long long)b * P.ld;
  for (int i = tid; i < kBins; i += NTHR) {
    S.hist_c[i] = 0;
    S.hist_w0[i] = S.hist_w1[i] = S.hist_w2[i] = 0;
  }
  if (tid < kSteps) S.pow2[tid] = P.pow2[tid];
  // the other CTAs run, before anything is written into their shared memory
  if (C > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  pdl_wait();
  const float T = P.temperature ? __ldcg(P.temperature + b) : 1.f;
  const int top_k = P.top_k ? __ldcg(P.top_k + b) : 0;
  const float top_p = P.top_p ? __ldcg(P.top_p + b) : 1.f;
  const float min_p = P.min_p ? __ldcg(P.min_p + b) : 0.f;

  // ---- the row's candidates: largest (the first of equal ones), smallest,
  // how many
  float fhi = -INFINITY, flo = INFINITY;
  int ihi = 0;
  unsigned cnt = 0;
  auto note = [&](float v, int i) {
    if (v > -INFINITY) {
      if (v > fhi) {
        fhi = v;
        ihi = i;
      }
      flo = fminf(flo, v);
      ++cnt;
    }
  };
  int i = tid;
  for (; i + 7 * NTHR < n; i += 8 * NTHR) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __ldcg(row + begin + i + e * NTHR);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (P.resident) data[i + e * NTHR] = v[e];
      note(v[e], begin + i + e * NTHR);
    }
  }
  for (; i < n; i += NTHR) {
    const float v = __ldcg(row + begin + i);
    if (P.resident) data[i] = v;
    note(v, begin + i);
  }
  u64 hi = warp_max64(cnt ? key_of(fhi, ihi) : 0);
  u64 lo = warp_min64(cnt ? key_of(flo, 0) : ~0ull);
  cnt = __reduce_add_sync(0xffffffffu, cnt);
  if (lane == 0) {
    S.red[warp] = hi;
    S.red2[warp] = lo;
    S.red3[warp] = cnt;
  }
  if (C > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  __syncthreads();
  if (warp == 0) {  // to every rank
    hi = warp_max64(lane < NTHR / 32 ? S.red[lane] : 0);
    lo = warp_min64(lane < NTHR / 32 ? S.red2[lane] : ~0ull);
    cnt = __reduce_add_sync(0xffffffffu, lane < NTHR / 32 ? S.red3[lane] : 0);
    if (lane < (int)C) {
      st_u64(remote(&S.key_max[rank], lane), hi);
      st_u64(remote(&S.key_min[rank], lane), lo);
      st_u32(remote(&S.count[rank], lane), cnt);
    }
  }
  if (C == 1)
    __syncthreads();
  else
    cluster_sync();
  hi = 0;
  lo = ~0ull;
  cnt = 0;
  for (unsigned r = 0; r < C; ++r) {
    hi = max(hi, S.key_max[r]);
    lo = min(lo, S.key_min[r]);
    cnt += S.count[r];
  }
  if (cnt == 0 || !(T > 0.f) || top_k == 1) {  // no candidate, or the first one
    if (rank == 0 && tid == 0) {
      P.out[b] = cnt ? index_of(hi) : 0;
      if (P.kept) P.kept[b] = cnt ? 1 : 0;
      if (P.logprob) P.logprob[b] = cnt ? 0.f : __int_as_float(0x7FC00000);
    }
    return;  // (nobody reads another CTA's shared memory any more)
  }
  Row R;
  R.pow2 = S.pow2;
  R.top = value_of(hi);
  R.per_unit = 92.33248261689366 / (double)T;
  R.frac = P.frac;
  // fine bins up to the last value with a weight, coarse ones beyond
  const float span = R.top - value_of(lo);
  R.reach = fminf(span, (float)(0.6931471805599453 * (P.frac + 1) * (double)T));
  R.edge = fminf(R.reach, FLT_MAX);
  if (!(R.top <= FLT_MAX)) R.reach = -1.f;  // +inf leaves the others nothing
  R.fine = R.edge > 0.f ? (float)kFine / R.edge : 0.f;
  const float rest = fminf(span, 32.f * R.edge + 64.f) - R.edge;
  R.coarse = rest > 0.f ? (float)(kBins - kFine) / rest : 0.f;
  const Work<NTHR> W = {P, S, R, data, row, begin, n, rank, C};

  // ---- histogram of counts and, unless a small top-k will do without, of
  // weights
  const double mp = min_p > 0.f ? fmin(1.0, (double)min_p) : 0.0;
  const bool few = top_k > 0 && top_k <= NTHR / 2 && (unsigned)top_k < cnt;
  if (few)
    W.each([&](const float (&v)[4], int) {
      int b[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e] = R.bin(v[e]);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (v[e] > -INFINITY) atomicAdd(&S.hist_c[b[e]], 1u);
    });
  else
    W.weigh(R, mp, true);
  W.sync();
  W.sum_bins(kBins, S.tot_c, few ? nullptr : S.tot_w);
  W.sync();

  if (rank != 0) {  // rank 0 leads from here
    for (;;) {
      W.sync();
      if (S.cmd.op == kDone) return;
      W.serve(mp);
    }
  }
  // ---- rank 0. Decisions are warp 0's; the other warps help with collections
  // and sorting.
  const float ub = P.u ? __ldcg(P.u + b) : 0.f;
  u64 kept = cnt, sum = 0;
  Bin kb = {-1, 0, 0, 0, 0};
  Found pick = {0, 0, 0};
  if (top_k > 0 && (u64)top_k < kept) kept = top_k;
  const bool by_k = kept < cnt;
  auto want = [&](int from, int to) {  // bins from .. to (warp 0)
#pragma unroll
    for (int e = 0; e < kBins / 32; e += 32) {
      const int q = e + lane, l = max(0, from - 32 * q), h = min(31, to - 32 * q);
      if (l <= h) S.wanted[q] |= (0xFFFFFFFFu >> (31 - h)) & (0xFFFFFFFFu << l);
    }
  };
  auto bin_at = [&](bool by_weight, u64 target) {
    return W.find_bin(kBins, S.tot_c, S.tot_w, by_weight, target);
  };
  auto go_on = [&](int path) {  // warp 0's decision, known to all
    __syncthreads();
    if (tid == 0) S.path = path;
    __syncthreads();
    return S.path;
  };
  enum { kPathFew, kPathList, kPathSlow, kPathWeigh, kPathEnd };

  int path = 0;
  if (warp == 0) {
    for (int q = lane; q < kBins / 32; q += 32) S.wanted[q] = 0;
    if (few)
      for (int q = lane; q < kBins / 32; q += 32) S.sup_w[q] = 0;
    __syncwarp();
    W.scan_groups(kBins);
    if (few) {
      kb = bin_at(false, kept - 1);
      path = kb.pc + kb.c <= NTHR ? kPathFew : kPathWeigh;
      if (path == kPathFew) want(0, kb.at);
    } else {
      path = kPathSlow;
    }
  }
  if (few) path = go_on(path);
  if (few && path == kPathFew) {
    // ---- the members of the first bins, sorted; the filters shorten the list
    W.ask(Cmd{kCollect, 0, 0, 0, ~0ull}, mp);
    W.sort_list(S.list_n);
    if (warp == 0) {
      auto first_at = [&](unsigned len, u64 target) {  // whose running weight reaches it
        return min(len - 1, W.first_of(len, [&](unsigned q) { return S.list_w[q] >= target; }));
      };
      unsigned len = (unsigned)kept;
      if (top_p < 1.f) len = first_at(len, share(top_p, S.list_w[len - 1])) + 1;
      if (mp > 0.0)
        len = W.first_of(len, [&](unsigned q) { return R.weight(value_of(S.list_key[q])) < mp; });
      kept = len;
      sum = S.list_w[len - 1];
      pick.key = S.list_key[first_at(len, share(ub, sum))];
    }
  } else {
    if (few) {  // too many share the first bins: weights after all
      W.ask(Cmd{kWeights, 0, 0, 0, 0}, mp);
      if (warp == 0) W.scan_groups(kBins);
    }
    u64 total = 0, above = cnt;
    if (warp == 0) {
      // ---- the bins that can hold a filter's end or the draw, from what the
      // histogram bounds; their members in one collection
      total = S.sup_w[kBins / 32];
      if (mp > 0.0) above = __reduce_add_sync(0xffffffffu, lane < (int)C ? S.above[lane] : 0);
      u64 z0 = total, z1 = total;    // bounds of the weight that top-k keeps
      u64 s0 = total, s1 = total;    // of the kept weight
      u64 many = 0;
      if (by_k) {
        kb = bin_at(false, kept - 1);
        z1 = kb.pw + kb.w;
        z0 = kept == kb.pc + kb.c ? z1 : min(z1, kb.pw + 1);
        s0 = z0;
        s1 = z1;
        want(kb.at, kb.at);
        many += kb.c;
      }
      if (top_p < 1.f) {
        const Bin p0 = bin_at(true, share(top_p, z0));
        const Bin p1 = z1 == z0 ? p0 : bin_at(true, share(top_p, z1));
        s0 = min(s0, p0.pw + 1);
        s1 = min(s1, p1.pw + p1.w);
        want(p0.at, p1.at);
        many += p1.pc + p1.c - p0.pc;
      }
      if (above < kept) {
        const Bin m = bin_at(false, above - 1);
        s0 = min(s0, m.pw + 1);
        s1 = min(s1, m.pw + m.w);
        want(m.at, m.at);
        many += m.c;
      }
      const Bin d0 = bin_at(true, share(ub, min(s0, total)));
      const Bin d1 = bin_at(true, share(ub, max(s1, (u64)1)));
      want(d0.at, d1.at);
      many += d1.pc + d1.c - d0.pc;
      path = many <= NTHR ? kPathList : kPathSlow;
    }
    path = go_on(path);
    if (path == kPathList) {
      W.ask(Cmd{kCollect, 0, 0, 0, ~0ull}, mp);
      const unsigned n_list = S.list_n;
      W.sort_list(n_list);
      if (warp == 0) {
        bool lost = false;  // a bin outside the collection: the bounds did not hold
        auto search = [&](bool by_weight, u64 target) {
          const Bin q = bin_at(by_weight, target);
          if (!(S.wanted[q.at >> 5] >> (q.at & 31) & 1)) {
            lost = true;
            return Found{0, 1, 0};
          }
          const unsigned start = W.first_of(
              n_list, [&](unsigned i) { return R.bin(value_of(S.list_key[i])) >= q.at; });
          return W.in_list(q, start, min(n_list, start + (unsigned)q.c), by_weight, target);
        };
        u64 k = kept, run = total;
        if (by_k) run = search(false, k - 1).cum;
        if (top_p < 1.f) {
          const Found f = search(true, share(top_p, run));
          k = min(k, f.rank + 1);
          run = f.cum;
        }
        if (above < k) {
          k = above;
          run = search(false, k - 1).cum;
        }
        pick = search(true, share(ub, run));
        path = lost ? kPathSlow : kPathEnd;
        if (!lost) {
          kept = k;
          sum = run;
        }
      }
      path = go_on(path);
    }
    if (path == kPathSlow) {
      // ---- one bin after another: those with many members (equal or crowded
      // values) are narrowed down by the keys first. `kept`, `sum` and `pick`
      // are the same in all threads here
      total = S.sup_w[kBins / 32];
      above = cnt;
      if (mp > 0.0) {
        above = 0;
        for (unsigned r = 0; r < C; ++r) above += S.above[r];
      }
      auto search = [&](bool by_weight, u64 target) {
        Sub& sub = *reinterpret_cast<Sub*>(S.list_key);
        __syncthreads();
        Bin q = W.find_bin(kBins, S.tot_c, S.tot_w, by_weight, target);  // (every warp)
        const int bin = q.at;
        Cmd cmd = {kCollect, bin, 0, 0, ~0ull};
        if (q.c > NTHR) {
          W.ask(Cmd{kMinMax, bin, 0, 0, 0}, mp);
          cmd.lo = ~0ull;
          cmd.hi = 0;
          for (unsigned r = 0; r < C; ++r) {
            cmd.lo = min(cmd.lo, S.key_min[r]);
            cmd.hi = max(cmd.hi, S.key_max[r]);
          }
          // the row's groups make way for the bin's and come back after it
          const unsigned keep_c = tid <= kBins / 32 ? S.sup_c[tid] : 0;
          const u64 keep_w = tid <= kBins / 32 ? S.sup_w[tid] : 0;
          while (q.c > NTHR) {
            const u64 width = cmd.hi - cmd.lo;  // keys differ: at least q.c - 1
            const int bits = 64 - __clzll((long long)width);
            const Cmd h = {kHist, bin, max(0, bits - 9), cmd.lo, cmd.hi};
            W.ask(h, mp);
            if (warp == 0) W.scan_groups(kSubBins);
            __syncthreads();
            const Bin s = W.find_bin(kSubBins, sub.c, sub.w, by_weight,
                                     by_weight ? target - q.pw : target - q.pc);
            q.pc += s.pc;
            q.pw += s.pw;
            q.c = s.c;
            q.w = s.w;
            const u64 top = cmd.hi - ((u64)s.at << h.shift);
            const u64 low = top - (((u64)1 << h.shift) - 1);
            cmd.lo = low > top || low < cmd.lo ? cmd.lo : low;
            cmd.hi = top;
          }
          __syncthreads();
          if (tid <= kBins / 32) {
            S.sup_c[tid] = keep_c;
            S.sup_w[tid] = keep_w;
          }
        }
        __syncthreads();
        if (tid < kBins / 32) S.wanted[tid] = tid == bin >> 5 ? 1u << (bin & 31) : 0;
        W.ask(cmd, mp);
        W.sort_list(S.list_n);
        return W.in_list(q, 0, (unsigned)q.c, by_weight, target);  // (every warp)
      };
      sum = total;
      if (by_k) sum = search(false, kept - 1).cum;
      if (top_p < 1.f) {
        const Found f = search(true, share(top_p, sum));
        kept = min(kept, f.rank + 1);
        sum = f.cum;
      }
      if (above < kept) {
        kept = above;
        sum = search(false, kept - 1).cum;
      }
      pick = search(true, share(ub, sum));
    }
  }
  W.ask(Cmd{kDone, 0, 0, 0, 0}, mp);
  if (tid == 0) {
    P.out[b] = index_of(pick.key);
    if (P.kept) P.kept[b] = (int32_t)kept;
    if (P.logprob)
      P.logprob[b] = (float)log(R.power(R.steps(value_of(pick.key)), R.frac) / (double)sum);
  }
}

// CTAs per row: as many as leave each a slice worth a CTA (2048 values: with
// 4096, 16 rows of 16000 took 23.5 us in place of 20.9; with 1024, 4 rows of 4000
// 16.7 in place of 13.1) and fit the GPU at once
// for the whole batch; more where a slice would not fit shared memory. Clusters
// of 8 and 16 leave some of a GPC's SMs empty (rows of 151936: 6 with 16 CTAs
// each 34 us, with 8 41, 8 with 16 51, with 8 41; 18 with 8 54, with 4 50).
inline int cluster_for(int B, int V) {
  int c = 1;
  const auto fits = [&](int n) {
    return (long long)B * n <= num_sms() * (n == 16 ? 6 : n == 8 ? 7 : 8) / 8;
  };
  while (c < kMaxCluster && V / (2 * c) >= 2048 && fits(2 * c)) c *= 2;
  while (c < kMaxCluster && (V + c - 1) / c > kResident) c *= 2;
  return c;
}

template <int NTHR>
cudaError_t launch(const Params& P, int C, int B, cudaStream_t st) {
  const void* f = (const void*)sample_kernel<NTHR>;
  ensure_smem(f, (int)(sizeof(Shared) + kResident * 4));
  if (C > 8) {
    cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C, B);
  cfg.blockDim = dim3(NTHR);
  cfg.dynamicSmemBytes = sizeof(Shared) + (P.resident ? (size_t)P.slice * 4 : 0);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  count_launch();
  return cudaLaunchKernelEx(&cfg, sample_kernel<NTHR>, P);
}

struct Pow2 {
  double v[kSteps];
  Pow2() {
    for (int i = 0; i < kSteps; ++i) v[i] = exp2((double)i / kSteps);
  }
};

}  // namespace sf
}  // namespace qg

using namespace qg;

extern "C" qg_status qg_sample_filtered(const float* logits, long long ld, int B, int V,
                                        const float* temperature, const int32_t* top_k,
                                        const float* top_p, const float* min_p, const float* u,
                                        int32_t* out, int32_t* kept, float* logprob,
                                        void* stream) {
  clear_error();
  const char* who = "qg_sample_filtered";
  QG_REQUIRE(B >= 0 && V >= 1 && V <= (1 << 22), QG_ERR_UNSUPPORTED_SHAPE,
             "%s: B=%d V=%d (V in [1, 2^22])", who, B, V);
  QG_REQUIRE(B <= 65535, QG_ERR_UNSUPPORTED_SHAPE, "%s: B=%d above 65535", who, B);
  QG_REQUIRE(ld >= V && ld < (1LL << 40), QG_ERR_UNSUPPORTED_SHAPE,
             "%s: ld=%lld shorter than a row of V=%d", who, ld, V);
  if (B == 0) return QG_OK;
  QG_REQUIRE(logits && out && u, QG_ERR_INVALID_ARGUMENT, "%s: null logits, u or out", who);
  QG_REQUIRE(aligned(logits, 4) && aligned(temperature, 4) && aligned(top_k, 4) &&
                 aligned(top_p, 4) && aligned(min_p, 4) && aligned(u, 4) && aligned(out, 4) &&
                 aligned(kept, 4) && aligned(logprob, 4),
             QG_ERR_MISALIGNED, "%s: a pointer is not 4-byte aligned", who);
  static const sf::Pow2 pow2;
  const int C = sf::cluster_for(B, V);
  sf::Params P = {};
  P.logits = logits;
  P.ld = ld;
  P.temperature = temperature;
  P.top_k = top_k;
  P.top_p = top_p;
  P.min_p = min_p;
  P.u = u;
  P.out = out;
  P.kept = kept;
  P.logprob = logprob;
  P.V = V;
  P.slice = (V + C - 1) / C;
  P.resident = P.slice <= sf::kResident;
  P.frac = 44;
  while (((unsigned long long)V << P.frac) > (1ull << 62)) --P.frac;
  for (int i = 0; i < sf::kSteps; ++i) P.pow2[i] = pow2.v[i];
  cudaStream_t st = (cudaStream_t)stream;
  // Short slices, and more CTAs than SMs: fewer threads, whose barriers cost less
  // and of which an SM takes two blocks (512 and 256 threads, us: 160 rows of 2048
  // 21.4, 12.9; 250 rows of 6000 32.1, 26.2; one CTA an SM, 64 rows of 8000, 20.0,
  // 22.9).
  const bool few = P.slice <= 4096 || (P.slice <= 8192 && (long long)B * C > num_sms());
  const cudaError_t e = few ? sf::launch<256>(P, C, B, st) : sf::launch<512>(P, C, B, st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    set_error("%s: CUDA launch failed: %s", who, cudaGetErrorString(e));
    return QG_ERR_CUDA;
  }
  return check_launch(who);
}
