// Filtered sampling (include/qg.h, qg_sample_filtered): temperature, top-k,
// top-p, min-p and a draw from a given uniform number, each row with
// parameters of its own, in one launch without a sort.
//
// All three filters keep a prefix of the candidates in descending order
// (equal values by index), and the draw is the place in that prefix where
// the running weight reaches u times the prefix's weight. So everything is
// one operation: find the candidate at which a running count, or a running
// weight, reaches a target. A histogram of (count, weight) over 1024 bins
// that are monotone in the value answers it up to one bin; the bin's members
// (a handful) are then collected and ranked against each other.
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
#include <algorithm>
#include <cfloat>
#include <cstddef>

#include "qg_internal.cuh"

namespace qg {
namespace sf {

constexpr int kThreads = 512;
constexpr int kBins = 1024;
constexpr int kFine = 768;          // bins for the values whose weight is not 0
constexpr int kList = 1024;         // members of a bin that rank 0 ranks directly
constexpr int kMaxCluster = 16;
constexpr int kResident = 38016;    // values of a slice that shared memory holds

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
};

enum Op { kDone, kCollect, kMinMax, kHist };
struct Cmd {
  int op, bin, shift;
  u64 lo, hi;
};

struct Shared {
  u64 key_max[kMaxCluster], key_min[kMaxCluster];  // pushed by every rank
  unsigned count[kMaxCluster], above[kMaxCluster]; // candidates; weights >= min_p
  Cmd cmd;
  unsigned list_n;
  u64 red[kThreads / 32], red2[kThreads / 32];
  unsigned red3[kThreads / 32];
  // a search's answer (rank 0)
  int s_bin;
  u64 a_rank, a_cum, a_key;
  u64 list_key[kList];
  u64 list_w[kList];
  u64 hist_w[kBins];      // this CTA's
  u64 tot_w[kBins], sub_w[kBins];        // the cluster's (rank 0): row, and inside a bin
  u64 tot_pw[kBins], sub_pw[kBins];      // exclusive prefixes
  unsigned hist_c[kBins], tot_c[kBins], sub_c[kBins], tot_pc[kBins], sub_pc[kBins];
};

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
               "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void* p, unsigned rank) {
  const uint32_t local = static_cast<uint32_t>(__cvta_generic_to_shared(p));
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_u64(uint32_t a, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ void st_u32(uint32_t a, unsigned v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ u64 ld_u64(uint32_t a) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ unsigned ld_u32(uint32_t a) {
  unsigned v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
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

// The row's bins and weights.
struct Row {
  float top;       // the largest value
  double inv_t;    // 1 / temperature
  double unit;     // 2^frac
  double floor_;   // (l - max) / T below this has weight 0
  float fine, coarse, edge;  // bins: d * fine up to d = edge, then (d - edge) * coarse

  __device__ __forceinline__ double weight(float v) const {
    if (v == top) return 1.0;  // (also +inf; below it everything is then 0)
    const double x = ((double)v - (double)top) * inv_t;
    return x > -INFINITY ? exp(x) : 0.0;
  }
  __device__ __forceinline__ u64 fixed(float v) const {
    if (v == top) return (u64)unit;
    const double x = ((double)v - (double)top) * inv_t;
    return x > floor_ ? __double2ull_rn(exp(x) * unit) : 0;
  }
  // Monotone in v: each step (difference, product, conversion) is.
  __device__ __forceinline__ int bin(float v) const {
    if (v == top) return 0;
    const float d = top - v;
    if (d <= edge) return (int)fminf(d * fine, (float)(kFine - 1));
    return kFine + (int)fminf((d - edge) * coarse, (float)(kBins - kFine - 1));
  }
};

template <class F>
__device__ __forceinline__ void each(const Params& P, const float* data, const float* row,
                                     int begin, int n, F f) {
  for (int i = threadIdx.x; i < n; i += kThreads)
    f(P.resident ? data[i] : __ldcg(row + begin + i), begin + i);
}

// Exclusive prefixes of the cluster's counts and weights over the bins
// (rank 0, all threads): two neighbouring bins a thread.
__device__ __forceinline__ void prefixes(Shared& S, const unsigned* c, const u64* w, unsigned* pc,
                                         u64* pw) {
  static_assert(kBins == 2 * kThreads, "two bins a thread");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned c0 = c[2 * tid], c1 = c[2 * tid + 1];
  const u64 w0 = w[2 * tid], w1 = w[2 * tid + 1];
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
  if (lane == 31) {
    S.red3[warp] = xc;
    S.red[warp] = xw;
  }
  __syncthreads();
  unsigned bc = xc - c0 - c1;
  u64 bw = xw - w0 - w1;
  for (int i = 0; i < warp; ++i) {
    bc += S.red3[i];
    bw += S.red[i];
  }
  pc[2 * tid] = bc;
  pc[2 * tid + 1] = bc + c0;
  pw[2 * tid] = bw;
  pw[2 * tid + 1] = bw + w0;
  __syncthreads();
}

// The cluster's sums of the CTAs' histograms into rank 0's (c, w): each rank
// sums a share of the bins.
__device__ __forceinline__ void sum_bins(Shared& S, unsigned rank, unsigned C, unsigned* c,
                                         u64* w) {
  const int per = kBins / C;
  for (int i = threadIdx.x; i < per; i += kThreads) {
    const int b = rank * per + i;
    unsigned nc = 0;
    u64 nw = 0;
    for (unsigned r = 0; r < C; ++r) {
      nc += ld_u32(remote(&S.hist_c[b], r));
      nw += ld_u64(remote(&S.hist_w[b], r));
    }
    st_u32(remote(&c[b], 0), nc);
    st_u64(remote(&w[b], 0), nw);
  }
}

// One collective step of the cluster on the members of a bin whose keys lie
// in [lo, hi].
__device__ __forceinline__ void serve(const Params& P, Shared& S, const Row& R, const float* data,
                                      const float* row, int begin, int n, unsigned rank,
                                      unsigned C) {
  const Cmd c = S.cmd;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (c.op == kCollect) {
    const uint32_t cnt = remote(&S.list_n, 0);
    each(P, data, row, begin, n, [&](float v, int i) {
      const u64 k = key_of(v, i);
      if (k && R.bin(v) == c.bin && k >= c.lo && k <= c.hi) {
        const unsigned at = add_u32(cnt, 1);
        if (at < kList) {
          st_u64(remote(&S.list_key[at], 0), k);
          st_u64(remote(&S.list_w[at], 0), R.fixed(v));
        }
      }
    });
  } else if (c.op == kMinMax) {
    u64 lo = ~0ull, hi = 0;
    each(P, data, row, begin, n, [&](float v, int i) {
      const u64 k = key_of(v, i);
      if (k && R.bin(v) == c.bin) {
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
      for (int i = 1; i < kThreads / 32; ++i) {
        lo = min(lo, S.red[i]);
        hi = max(hi, S.red2[i]);
      }
      st_u64(remote(&S.key_min[rank], 0), lo);
      st_u64(remote(&S.key_max[rank], 0), hi);
    }
  } else {
    for (int i = tid; i < kBins; i += kThreads) {
      S.hist_c[i] = 0;
      S.hist_w[i] = 0;
    }
    __syncthreads();
    each(P, data, row, begin, n, [&](float v, int i) {
      const u64 k = key_of(v, i);
      if (k && R.bin(v) == c.bin && k >= c.lo && k <= c.hi) {
        const int b = (int)((c.hi - k) >> c.shift);
        atomicAdd(&S.hist_c[b], 1u);
        const u64 w = R.fixed(v);
        if (w) atomicAdd(&S.hist_w[b], w);
      }
    });
    cluster_sync();
    sum_bins(S, rank, C, S.sub_c, S.sub_w);
  }
  cluster_sync();
}

// Rank 0: one collective step (every thread calls it).
__device__ __forceinline__ void ask(const Params& P, Shared& S, const Row& R, const float* data,
                                    const float* row, int begin, int n, unsigned C, const Cmd& c) {
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
  cluster_sync();
  if (c.op != kDone) serve(P, S, R, data, row, begin, n, 0, C);
}

// The bin where the running count passes `target` (by_weight: where the
// running weight reaches it).
__device__ __forceinline__ int find_bin(Shared& S, const unsigned* c, const u64* w,
                                        const unsigned* pc, const u64* pw, bool by_weight,
                                        u64 target) {
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += kThreads) {
    const bool in = by_weight ? pw[i] < target && target <= pw[i] + w[i]
                              : pc[i] <= target && target < (u64)pc[i] + c[i];
    if (in) S.s_bin = i;
  }
  __syncthreads();
  return S.s_bin;
}

__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const __grid_constant__ Params P) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& S = *reinterpret_cast<Shared*>(smem);
  float* data = reinterpret_cast<float*>(smem + sizeof(Shared));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned C = gridDim.x, rank = cluster_rank();
  const int b = blockIdx.y;
  const int begin = min(P.V, (int)rank * P.slice), n = min(P.slice, P.V - begin);
  const float* row = P.logits + (long long)b * P.ld;
  for (int i = tid; i < kBins; i += kThreads) {
    S.hist_c[i] = 0;
    S.hist_w[i] = 0;
  }
  pdl_wait();

  // ---- the row's candidates: largest, smallest, how many
  u64 hi = 0, lo = ~0ull;
  unsigned cnt = 0;
#pragma unroll 8
  for (int i = tid; i < n; i += kThreads) {
    const float v = __ldcg(row + begin + i);
    if (P.resident) data[i] = v;
    const u64 k = key_of(v, begin + i);
    hi = max(hi, k);
    lo = min(lo, k ? k : ~0ull);
    cnt += k != 0;
  }
  hi = warp_max64(hi);
  lo = warp_min64(lo);
  cnt = __reduce_add_sync(0xffffffffu, cnt);
  if (lane == 0) {
    S.red[warp] = hi;
    S.red2[warp] = lo;
    S.red3[warp] = cnt;
  }
  __syncthreads();
  if (tid < (int)C) {  // to every rank
    hi = S.red[0];
    lo = S.red2[0];
    cnt = S.red3[0];
    for (int i = 1; i < kThreads / 32; ++i) {
      hi = max(hi, S.red[i]);
      lo = min(lo, S.red2[i]);
      cnt += S.red3[i];
    }
    st_u64(remote(&S.key_max[rank], tid), hi);
    st_u64(remote(&S.key_min[rank], tid), lo);
    st_u32(remote(&S.count[rank], tid), cnt);
  }
  cluster_sync();
  hi = 0;
  lo = ~0ull;
  cnt = 0;
  for (unsigned r = 0; r < C; ++r) {
    hi = max(hi, S.key_max[r]);
    lo = min(lo, S.key_min[r]);
    cnt += S.count[r];
  }

  // ---- the row's parameters
  const float T = P.temperature ? __ldcg(P.temperature + b) : 1.f;
  const int top_k = P.top_k ? __ldcg(P.top_k + b) : 0;
  const float top_p = P.top_p ? __ldcg(P.top_p + b) : 1.f;
  const float min_p = P.min_p ? __ldcg(P.min_p + b) : 0.f;
  if (cnt == 0 || !(T > 0.f) || top_k == 1) {  // no candidate, or the first one
    if (rank == 0 && tid == 0) {
      P.out[b] = cnt ? index_of(hi) : 0;
      if (P.kept) P.kept[b] = cnt ? 1 : 0;
      if (P.logprob) P.logprob[b] = cnt ? 0.f : __int_as_float(0x7FC00000);
    }
    return;  // (nobody reads another CTA's shared memory any more)
  }
  Row R;
  R.top = value_of(hi);
  R.inv_t = 1.0 / (double)T;
  R.unit = (double)(1ull << P.frac);
  R.floor_ = -0.6931471805599453 * (P.frac + 1);
  // fine bins up to the last value with a weight, coarse ones beyond
  const float span = R.top - value_of(lo);
  R.edge = fminf(fminf(span, (float)(-R.floor_ * (double)T)), FLT_MAX);
  R.fine = R.edge > 0.f ? (float)kFine / R.edge : 0.f;
  const float rest = fminf(span, 32.f * R.edge + 64.f) - R.edge;
  R.coarse = rest > 0.f ? (float)(kBins - kFine) / rest : 0.f;

  // ---- histogram of counts and weights
  const bool use_m = min_p > 0.f;
  const double mp = fmin(1.0, (double)min_p);
  unsigned above = 0;
  each(P, data, row, begin, n, [&](float v, int i) {
    if (!(v > -INFINITY)) return;
    const int k = R.bin(v);
    atomicAdd(&S.hist_c[k], 1u);
    const u64 w = R.fixed(v);
    if (w) atomicAdd(&S.hist_w[k], w);
    if (use_m) above += R.weight(v) >= mp;
  });
  above = __reduce_add_sync(0xffffffffu, above);
  if (lane == 0) S.red3[warp] = above;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < kThreads / 32; ++i) above += S.red3[i];
    st_u32(remote(&S.above[rank], 0), above);
  }
  cluster_sync();
  sum_bins(S, rank, C, S.tot_c, S.tot_w);
  cluster_sync();

  if (rank != 0) {  // rank 0 leads from here
    for (;;) {
      cluster_sync();
      if (S.cmd.op == kDone) return;
      serve(P, S, R, data, row, begin, n, rank, C);
    }
  }
  prefixes(S, S.tot_c, S.tot_w, S.tot_pc, S.tot_pw);

  int listed = -1;  // the bin whose members are in the list, all of them
  unsigned list_n = 0;
  u64 list_pc = 0, list_pw = 0;  // candidates and weight before the list

  // The candidate where the running count passes `target`, or the running
  // weight reaches it: a_rank (candidates before it), a_cum (running weight
  // with it) and, if `want_key`, a_key.
  auto search = [&](bool by_weight, u64 target, bool want_key) {
    const int bin = find_bin(S, S.tot_c, S.tot_w, S.tot_pc, S.tot_pw, by_weight, target);
    const u64 pc = S.tot_pc[bin], pw = S.tot_pw[bin];
    const unsigned c = S.tot_c[bin];
    if (!want_key && (c == 1 || (!by_weight && target == pc + c - 1))) {
      __syncthreads();
      if (tid == 0) {
        S.a_rank = pc + c - 1;
        S.a_cum = pw + S.tot_w[bin];
      }
      __syncthreads();
      return;
    }
    if (listed != bin) {
      Cmd cmd = {kCollect, bin, 0, 0, ~0ull};
      list_n = c;
      list_pc = pc;
      list_pw = pw;
      listed = bin;
      if (c > kList) {  // narrow the bin down by its keys
        listed = -1;
        ask(P, S, R, data, row, begin, n, C, Cmd{kMinMax, bin, 0, 0, 0});
        cmd.lo = ~0ull;
        cmd.hi = 0;
        for (unsigned r = 0; r < C; ++r) {
          cmd.lo = min(cmd.lo, S.key_min[r]);
          cmd.hi = max(cmd.hi, S.key_max[r]);
        }
        while (list_n > kList) {
          const u64 width = cmd.hi - cmd.lo;  // keys differ, so it is at least list_n - 1
          const int bits = 64 - __clzll((long long)width);
          Cmd h = {kHist, bin, max(0, bits - 10), cmd.lo, cmd.hi};
          ask(P, S, R, data, row, begin, n, C, h);
          prefixes(S, S.sub_c, S.sub_w, S.sub_pc, S.sub_pw);
          const int s = find_bin(S, S.sub_c, S.sub_w, S.sub_pc, S.sub_pw, by_weight,
                                 by_weight ? target - list_pw : target - list_pc);
          list_n = S.sub_c[s];
          list_pc += S.sub_pc[s];
          list_pw += S.sub_pw[s];
          const u64 top = cmd.hi - ((u64)s << h.shift);
          const u64 low = top - (((u64)1 << h.shift) - 1);
          cmd.lo = low > top || low < cmd.lo ? cmd.lo : low;
          cmd.hi = top;
        }
      }
      ask(P, S, R, data, row, begin, n, C, cmd);
    }
    // rank the members against each other
    for (unsigned i = tid; i < list_n; i += kThreads) {
      const u64 k = S.list_key[i];
      u64 before = list_pc, sum = list_pw;
      for (unsigned j = 0; j < list_n; ++j) {
        const bool ahead = S.list_key[j] > k;
        before += ahead;
        sum += ahead ? S.list_w[j] : 0;
      }
      const u64 w = S.list_w[i];
      if (by_weight ? sum < target && target <= sum + w : before == target) {
        S.a_rank = before;
        S.a_cum = sum + w;
        S.a_key = k;
      }
    }
    __syncthreads();
  };
  auto share = [&](double f, u64 total) {  // f of a weight, at least 1, at most all of it
    const double t = ceil(fmin(fmax(f, 0.0), 1.0) * (double)total);
    return max((u64)1, min(total, __double2ull_rn(t)));
  };

  u64 kept = cnt, sum = S.tot_pw[kBins - 1] + S.tot_w[kBins - 1];
  if (top_k > 0 && (u64)top_k < kept) {
    kept = top_k;
    search(false, kept - 1, false);
    sum = S.a_cum;
  }
  if (top_p < 1.f) {
    search(true, share(top_p, sum), false);
    kept = min(kept, S.a_rank + 1);
    sum = S.a_cum;
  }
  if (use_m) {
    u64 m = 0;
    for (unsigned r = 0; r < C; ++r) m += S.above[r];
    if (m < kept) {
      kept = m;
      search(false, kept - 1, false);
      sum = S.a_cum;
    }
  }
  search(true, share(P.u ? (double)__ldcg(P.u + b) : 0.0, sum), true);
  const u64 pick = S.a_key;
  ask(P, S, R, data, row, begin, n, C, Cmd{kDone, 0, 0, 0, 0});
  if (tid == 0) {
    P.out[b] = index_of(pick);
    if (P.kept) P.kept[b] = (int32_t)kept;
    if (P.logprob) P.logprob[b] = (float)log(R.weight(value_of(pick)) / ((double)sum / R.unit));
  }
}

// CTAs per row: as many as leave each a slice worth a CTA, and fit the GPU
// for the whole batch; more where a slice would not fit shared memory.
inline int cluster_for(int B, int V) {
  int c = 1;
  while (c < kMaxCluster && V / (2 * c) >= 4096 && (long long)B * 2 * c <= num_sms()) c *= 2;
  while (c < kMaxCluster && (V + c - 1) / c > kResident) c *= 2;
  return c;
}

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
  const size_t smem = sizeof(sf::Shared) + (P.resident ? (size_t)P.slice * 4 : 0);
  ensure_smem((const void*)sf::sample_kernel, (int)(sizeof(sf::Shared) + sf::kResident * 4));
  if (C > 8) {
    cudaError_t e = cudaFuncSetAttribute((const void*)sf::sample_kernel,
                                         cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    QG_REQUIRE(e == cudaSuccess, QG_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C, B);
  cfg.blockDim = dim3(sf::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = (cudaStream_t)stream;
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
  cudaLaunchKernelEx(&cfg, sf::sample_kernel, P);
  return check_launch(who);
}
