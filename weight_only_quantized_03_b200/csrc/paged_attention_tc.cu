// Prompt rows over a paged K/V cache on the tcgen05 tensor cores
// (include/qg.h, qg_paged_attention; the other kernels and the units of the
// int8 operands: paged_attention.cu).
//
// A CTA takes 128 (row, query head) pairs of one KV head of one sequence and
// walks their keys 64 at a time: S = Q K^T and O += P V are tcgen05.mma with
// M = 128, accumulators in tensor memory (O: head_dim columns, S: two buffers
// of 64). Warps 4-7 bring K and V from the pages in the 128-byte swizzled
// layout, K as the K-major operand and V, in the same [token][dim] order, as
// the MN-major one: int8 codes become fp16 (exact) on the way through
// registers, bf16 values come by asynchronous copies. Warps 0-3 own a row a
// thread: no maximum or sum crosses threads. They read S, form the weights
// with the lazy maximum of the decode kernel and write them as 16-bit pairs
// over S, where the second product reads them as its A operand. One thread of
// warp 8 issues the products; S of the next keys is in flight while the rows
// work on the current ones.
//
// 99 KB of shared memory and 256 tensor-memory columns at head size 128, so
// that an SM holds two CTAs and one's softmax meets the other's products.
// What bounds it: a 64-key step takes a lone CTA 1900 cycles, of which the
// rows' 64 weights a thread are 1400 and their way back to tensor memory 200;
// two CTAs on an SM take about 2900 for a step each. The step's products are
// 640 cycles of tensor core (S reads both operands from shared memory), and a
// scheduler issues every other cycle. 4096 rows over 4096 tokens (16 query, 8
// KV heads of 128): 113 us, 607 TFLOP/s. Measured and slower: eight row warps with
// half of a step's keys each (2053 rows of five users: 69 against 60 us), 256
// pairs a CTA (80), and the line of all steps cut into equal pieces with a
// merge behind (108: a step's scheduling and the pieces' parts cost more than
// the balance gave).
//
// Balance: long tiles start first, and where the tiles do not fill the GPU a
// cluster of up to eight CTAs shares a tile's keys; their results meet through
// distributed shared memory (128 rows over 32768 tokens: 698 us with one CTA a
// tile, 119 with eight).
//
// A value of V that is infinite or NaN at a token that some of the rows do
// not see must not reach them as 0 * inf: it is left out of the operand, and
// in the end the rows that see such values read them again and add them (bf16
// pages; under an int8 block's NaN scale the weights of rows that do not see
// it are exact zeros and the codes are finite).
//
// Every wait is bounded (1 s). One that gives up ends the CTA's work; its
// rows are then NaN.
#include <cuda_fp16.h>

#include <climits>
#include <type_traits>

#include "mma_sync.cuh"
#include "paged_attention.cuh"
#include "tcgen05_util.cuh"

namespace qg {
namespace pa {

using namespace tc;

constexpr int kRows = 128;         // rows of a CTA
constexpr int kKeys = 64;          // keys of a step
constexpr int kPThreads = 288;     // 4 softmax warps, 4 loading warps, the issuing warp
constexpr int kTmemCols = 256;
constexpr int kScol = 128;         // S buffers at columns 128 and 192; O at 0

template <int D>
struct PromptSmem {
  static constexpr int kQ = kRows * D * 2, kKV = kKeys * D * 2;
  static constexpr int kTail = 2560;  // PromptShared
  static constexpr int kBytes = 1024 + kQ + 4 * kKV + kTail;
};

struct PromptShared {  // behind the operands
  uint64_t q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_full, drain;
  float scale[4][8];   // ring: a step's K and V scales (4 blocks of 16 tokens each)
  float unit[kRows];   // of each pair's q
  float m[kRows], l[kRows];  // what a pair's keys gave (clusters)
  float factor[kRows];       // of each CTA's part of the pairs written here
  uint32_t tmem;
  int abort;
  int odd;             // values of V that are not finite were left out
};

#define QG_R8(a, i) "r"((a)[i]), "r"((a)[i + 1]), "r"((a)[i + 2]), "r"((a)[i + 3]), \
                    "r"((a)[i + 4]), "r"((a)[i + 5]), "r"((a)[i + 6]), "r"((a)[i + 7])
#define QG_W8(a, i) "=r"((a)[i]), "=r"((a)[i + 1]), "=r"((a)[i + 2]), "=r"((a)[i + 3]), \
                    "=r"((a)[i + 4]), "=r"((a)[i + 5]), "=r"((a)[i + 6]), "=r"((a)[i + 7])

// 32 columns of the warp's 32 lanes, a register each. The load and the wait
// for it are one statement: the compiler may move or spill the registers
// of a load that has not been waited for.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31},"
      " [%32];\n\ttcgen05.wait::ld.sync.aligned;"
      : QG_W8(v, 0), QG_W8(v, 8), QG_W8(v, 16), QG_W8(v, 24)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      QG_R8(v, 0), QG_R8(v, 8), QG_R8(v, 16), QG_R8(v, 24)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(one));
  return one != 0;
}
// Shared-memory writes visible to the tensor core.
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// MN-major operand, 128-byte swizzle: 64 neighbouring dims of a token are a
// 128-byte row, 8 tokens a 1024-byte group (SBO between groups), the next 64
// dims a panel further (LBO).
__device__ __forceinline__ uint64_t mn_desc(uint32_t addr, uint32_t panel) {
  uint64_t d = 0;
  d |= (uint64_t)((addr >> 4) & 0x3FFFu);
  d |= (uint64_t)(panel >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}
constexpr uint32_t kBisMnMajor = 1u << 16;  // instruction descriptor: B is MN-major

// Clusters: another CTA's shared memory at the address of `p`.
__device__ __forceinline__ uint32_t remote(const void* p, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ float remote_f32(const float* p, int rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float4 remote_f32x4(const uint8_t* p, int rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(remote(p, rank))
               : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// Byte offset of 16-byte chunk c (8 dims) of a row in panels of 64 dims.
template <int ROWS>
__device__ __forceinline__ int at_chunk(int row, int c) {
  return (c >> 3) * (ROWS * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
}

// Byte offset of 4 dims (chunk c) of a pair's result: pairs 512 (256) bytes
// apart, chunks exchanged by the pair so that neighbours' stores meet other
// banks.
template <int D>
__device__ __forceinline__ int part_at(int pair, int c) {
  return pair * (D * 4) + ((c ^ (pair & (D / 4 - 1))) << 4);
}

// A cluster's results of its tile: CTA z takes 128 / Z pairs from all of them
// (a softmax's parts: each has its reference m, its weights' sum l, and its
// output divided by l) and writes them out. Loads from the others' shared
// memory take several hundred cycles: a thread's go out together. Returns
// whether any CTA left V values out.
template <int D, int Z, class F>
__device__ __forceinline__ int join(PromptShared& S, const uint8_t* parts, int z, int first,
                                    int cols, F out_at) {
  constexpr int N = kRows / Z, C = D / 8;  // pairs, chunks of 8 dims
  const int tid = threadIdx.x;
  int odd = 0;
  if (tid < N) {  // the pair's factors
    float m[Z], l[Z], M = -FLT_MAX, L = 0.f;
#pragma unroll
    for (int k = 0; k < Z; ++k) {
      m[k] = remote_f32(&S.m[z * N + tid], k);
      l[k] = remote_f32(&S.l[z * N + tid], k);
    }
#pragma unroll
    for (int k = 0; k < Z; ++k) M = fmaxf(M, m[k]);
#pragma unroll
    for (int k = 0; k < Z; ++k) {
      l[k] *= ex2(m[k] - M);
      L += l[k];
    }
    const float f = L != 0.f ? 1.f / L : 0.f;
#pragma unroll
    for (int k = 0; k < Z; ++k) S.factor[k * N + tid] = l[k] * f;
  }
  {
    int o[Z];
#pragma unroll
    for (int k = 0; k < Z; ++k) o[k] = __float_as_int(remote_f32((const float*)&S.odd, k));
#pragma unroll
    for (int k = 0; k < Z; ++k) odd |= o[k];
  }
  __syncthreads();
#pragma unroll 2
  for (int i = tid; i < N * C; i += kPThreads) {
    const int pair = i / C, d = i % C;
    float4 y[Z][2];
#pragma unroll
    for (int k = 0; k < Z; ++k)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        y[k][e] = remote_f32x4(parts + part_at<D>(z * N + pair, 2 * d + e), k);
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < Z; ++k) {
      const float a = S.factor[k * N + pair];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        x[4 * e] = fmaf(a, y[k][e].x, x[4 * e]);
        x[4 * e + 1] = fmaf(a, y[k][e].y, x[4 * e + 1]);
        x[4 * e + 2] = fmaf(a, y[k][e].z, x[4 * e + 2]);
        x[4 * e + 3] = fmaf(a, y[k][e].w, x[4 * e + 3]);
      }
    }
    if (first + z * N + pair < cols)
      *reinterpret_cast<uint4*>(out_at(z * N + pair) + 8 * d) =
          make_uint4(mm::pack_bf16(x[0], x[1]), mm::pack_bf16(x[2], x[3]),
                     mm::pack_bf16(x[4], x[5]), mm::pack_bf16(x[6], x[7]));
  }
  return odd;
}

template <int D, bool I8>
__global__ void __launch_bounds__(kPThreads, 2) prompt_kernel(const __grid_constant__ Params P) {
  using L = PromptSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sq = smem;
  uint8_t* sk = sq + L::kQ;        // [2]
  uint8_t* sv = sk + 2 * L::kKV;   // [2]
  PromptShared& S = *reinterpret_cast<PromptShared*>(sv + 2 * L::kKV);
  volatile int* abort = &S.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();

  // The tile: long ones first, so that short ones fill the gaps at the end.
  // The sequences (32 at a time) go by their length, a sequence's tiles from
  // the last one back, heads side by side.
  int slot = (int)(blockIdx.x / (unsigned)P.Hkv);
  Item it = {-1, (int)blockIdx.x - slot * P.Hkv, 0, 0, 0, 0};
#pragma unroll 1
  for (int b0 = 0; b0 < P.B && it.b < 0; b0 += 32) {
    Item mine = {-1, 0, 0, 0, 0, 0};
    if (b0 + lane < P.B) set_seq(P, mine, b0 + lane);
    const int tiles = (mine.n * P.G + kRows - 1) / kRows;
    int before = 0, all = 0;
#pragma unroll 8
    for (int o = 0; o < 32; ++o) {
      const int ol = __shfl_sync(0xffffffffu, mine.len, o);
      const int ot = __shfl_sync(0xffffffffu, tiles, o);
      all += ot;
      before += ol > mine.len || (ol == mine.len && o < lane) ? ot : 0;
    }
    const unsigned m = __ballot_sync(0xffffffffu, slot >= before && slot - before < tiles);
    if (m) {
      const int l = __ffs(m) - 1;
      it.b = __shfl_sync(0xffffffffu, mine.b, l);
      it.r0 = __shfl_sync(0xffffffffu, mine.r0, l);
      it.n = __shfl_sync(0xffffffffu, mine.n, l);
      it.len = __shfl_sync(0xffffffffu, mine.len, l);
      it.ct = __shfl_sync(0xffffffffu, tiles - 1 - (slot - before), l);
    }
    slot -= all;
  }
  if (it.b < 0) return;
  const int first = it.ct * kRows, cols = it.n * P.G;  // (row, head) pairs of the sequence
  const int before = it.len - it.n;  // tokens cached before the rows
  // tokens that the last pair sees, and that all pairs see
  const int keys = it.len ? before + (min(first + kRows, cols) - 1) / P.G + 1 : 0;
  const int common = before + first / P.G + 1;
  const int all = (keys + kKeys - 1) / kKeys;
  // the steps of this CTA of the cluster: key0 / 64 of them lie before
  const int Z = gridDim.z, z = blockIdx.z;
  const int j0 = (int)((long long)all * z / Z), steps = (int)((long long)all * (z + 1) / Z) - j0;
  const int key0 = j0 * kKeys;

  // softmax threads: their pair's place in q and out
  const int c = first + tid, ri = c / P.G;
  const bool real = tid < kRows && c < cols;
  const int at = real ? (it.r0 + ri) * P.H + it.h * P.G + (c - ri * P.G) : -1;  // (below 2^30)
  uint16_t* out = reinterpret_cast<uint16_t*>(P.out) + (long long)(real ? at : 0) * D;
  if (all == 0) {
    if (real && z == 0)
      for (int d = 0; d < D; d += 8) *reinterpret_cast<uint4*>(out + d) = make_uint4(0, 0, 0, 0);
    return;
  }

  // A softmax warp brings its own 32 pairs of q, whole rows at a time; the
  // loads are under way while the barriers and tensor memory are set up.
  constexpr int LPR = D / 8, RPI = 32 / LPR;  // lanes of a row, rows of a load
  const int cc = lane % LPR;
  uint4 x[LPR];
  if (warp < 4 && steps) {
#pragma unroll
    for (int i = 0; i < LPR; ++i) {
      const int from = __shfl_sync(0xffffffffu, at, i * RPI + lane / LPR);
      x[i] = load16_if(reinterpret_cast<const uint8_t*>(P.q) + ((long long)from * D + cc * 8) * 2,
                       from >= 0);
    }
  }

  if (tid == 0) {
    mbar_init(&S.q_full, kRows);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.k_full[i], 64);
      mbar_init(&S.v_full[i], 64);
      mbar_init(&S.k_empty[i], 1);
      mbar_init(&S.v_empty[i], 1);
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_full[i], kRows);
    }
    mbar_init(&S.o_full, 1);
    mbar_init(&S.drain, 1);
    S.abort = 0;
    S.odd = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&S.tmem)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  // Not before tensor memory is allocated: the next kernel's CTAs may take
  // theirs before they wait for this grid, and hold it until they have.
  pdl_trigger();
  const uint32_t tmem = S.tmem;
  bool ok = true;

  if (warp < 4) {
    // ------------------------------------------------------------ the rows
    const int lim = real ? before + ri + 1 : INT_MAX;  // tokens the pair sees
    float qf = P.scale_log2;
    if (steps) {
      // q into shared memory, for int8 pages times a power of two, as fp16
      if constexpr (I8) {
        // two 16-bit maxima a word: magnitudes order as integers. Rows side by
        // side, so that their exchanges overlap
        uint32_t top[LPR];
#pragma unroll
        for (int i = 0; i < LPR; ++i)
          top[i] = __vmaxu2(__vmaxu2(x[i].x & 0x7FFF7FFFu, x[i].y & 0x7FFF7FFFu),
                            __vmaxu2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu));
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1)
#pragma unroll
          for (int i = 0; i < LPR; ++i)
            top[i] = __vmaxu2(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
#pragma unroll
        for (int i = 0; i < LPR; ++i) {
          const float unit = q_unit(fmaxf(bf16_lo(top[i]), bf16_hi(top[i])));
          uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __half2 h = __floats2half2_rn(bf16_lo(w[e]) * unit, bf16_hi(w[e]) * unit);
            w[e] = *reinterpret_cast<const uint32_t*>(&h);
          }
          x[i] = make_uint4(w[0], w[1], w[2], w[3]);
          if (cc == 0) S.unit[32 * warp + i * RPI + lane / LPR] = unit;
        }
      }
#pragma unroll
      for (int i = 0; i < LPR; ++i)
        *reinterpret_cast<uint4*>(
            sq + at_chunk<kRows>(32 * warp + i * RPI + lane / LPR, cc)) = x[i];
      __syncwarp();
      if constexpr (I8) qf /= S.unit[tid];
    }
    fence_async();
    mbar_arrive(&S.q_full);

    const uint32_t lanes = tmem + ((uint32_t)(32 * warp) << 16);
    // V's unit: 2048 / r is finite from 2^-115 on (at a scale of 2^-126 weights keep
    // their 11 bits down to 2^-14 of the largest, not 2^-25)
    float m = -FLT_MAX, l = 0.f, r = 0x1p-115f;
    for (int j = 0; j < steps; ++j) {
      const int b = j & 1;
      if (!wait_bar(&S.s_full[b], (uint32_t)(j >> 1) & 1u, abort)) {
        ok = false;
        break;
      }
      fence_after();
      const uint32_t sc = lanes + kScol + 64 * b;
      float ks[4], vs[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ks[i] = S.scale[j & 3][i] * qf;
        vs[i] = I8 ? S.scale[j & 3][4 + i] : 1.f;
      }
      const bool part = key0 + j * kKeys + kKeys > common;
      const int left = lim - key0 - j * kKeys;  // visible tokens of this step (or more, or none)
      // The row's largest score. A negative scale turns the order round. Blocks
      // that the row does not see at all stay out: under a scale of 0 (zeros
      // appended) or near it the least score would become one near 0.
      auto largest = [&]() {
        float top = -FLT_MAX;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t s[32];
          tmem_ld32(sc + 32 * h, s);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float k = ks[2 * h + q];
            const uint32_t flip = __float_as_uint(k) & 0x80000000u;
            float x[4] = {-FLT_MAX, -FLT_MAX, -FLT_MAX, -FLT_MAX};
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float y = __uint_as_float(s[16 * q + i] ^ flip);
              if (32 * h + 16 * q + i >= left) y = -FLT_MAX;
              x[i & 3] = fmaxf(x[i & 3], y);
            }
            const float y = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * fabsf(k);
            if (32 * h + 16 * q < left) top = fmaxf(top, y);
          }
        }
        return top;
      };
      // The weights relative to m as 16-bit pairs, their sum, the largest.
      uint32_t p[32];
      float sum, most;
      auto weights = [&](auto masked, float inv) {
        float t[4] = {0.f, 0.f, 0.f, 0.f}, x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t s[32];
          tmem_ld32(sc + 32 * h, s);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float k = ks[2 * h + q], w = I8 ? vs[2 * h + q] * inv : 1.f;
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              float y[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                y[e] = ex2(fmaf(__uint_as_float(s[16 * q + i + e]), k, -m));
                const bool hid = masked && 32 * h + 16 * q + i + e >= left;
                if (hid) y[e] = 0.f;
                t[(i + e) & 3] += y[e];
                x[(i + e) & 3] = fmaxf(x[(i + e) & 3], y[e]);
                if constexpr (I8) {
                  y[e] *= w;
                  if (hid) y[e] = 0.f;  // (whatever the block's scale is)
                }
              }
              if constexpr (I8) {
                const __half2 z = __floats2half2_rn(y[0], y[1]);
                p[16 * h + 8 * q + i / 2] = *reinterpret_cast<const uint32_t*>(&z);
              } else {
                p[16 * h + 8 * q + i / 2] = mm::pack_bf16(y[0], y[1]);
              }
            }
          }
        }
        sum = (t[0] + t[1]) + (t[2] + t[3]);
        most = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      };
      auto form = [&]() {
        const float inv = I8 ? 2048.f / r : 1.f;
        if (part)
          weights(std::true_type(), inv);
        else
          weights(std::false_type(), inv);
      };
      // V's largest scale among the blocks that the row sees: a later block's
      // must not cost it bits
      float vtop = 0.f;
      if constexpr (I8) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (16 * i < left && fabsf(vs[i]) <= FLT_MAX) vtop = fmaxf(vtop, fabsf(vs[i]));
      }
      const bool wider = I8 && vtop > r;
      // Every warp waits for every product once, in order (a parity tells a
      // phase only from its neighbours): here if O has to be rescaled, else at
      // the end of the step, when it has long been done.
      bool waited = j == 0;
      // The weights are formed with the reference as it is; only if one of a
      // warp's rows has outgrown it (or V's unit grows, or there is none yet)
      // the largest scores are looked for, and the weights formed again.
      bool again = j == 0 || (I8 && __any_sync(0xffffffffu, wider));
      if (!again) {
        form();
        again = __any_sync(0xffffffffu, most > (float)(1 << (int)kMargin));
      }
      if (again) {
        const float top = largest();
        float a = 1.f;
        if (wider) {
          const float n =
              __int_as_float(min(254, ((__float_as_int(vtop) >> 23) & 255) + 1) << 23);
          a = r / n;
          r = n;
        }
        const float x = fmaxf(m, top), e = ex2(m - x);
        m = x;
        l *= e;
        a *= e;
        if (j > 0) {  // O is whole up to the step before: rescale it
          if (!wait_bar(&S.o_full, (uint32_t)(j - 1) & 1u, abort)) {
            ok = false;
            break;
          }
          waited = true;
          fence_after();
#pragma unroll 1
          for (int d = 0; d < D; d += 32) {
            uint32_t o[32];
            tmem_ld32(lanes + d, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
            tmem_st32(lanes + d, o);
          }
        }
        form();
      }
      l += sum;
      tmem_st32(sc, p);
      if (!waited && !wait_bar(&S.o_full, (uint32_t)(j - 1) & 1u, abort)) {
        ok = false;
        break;
      }
      tmem_wait_st();
      fence_before();
      mbar_arrive(&S.p_full[b]);
    }
    if (ok && steps && !wait_bar(&S.o_full, (uint32_t)(steps - 1) & 1u, abort)) ok = false;
    if (!ok) *abort = 1;
    fence_after();
    // (V's unit apart from 1 / l: as one factor they would lose bits below 2^-126)
    const float f = l != 0.f ? 1.f / l : 0.f, unit = I8 ? r * (1.f / 2048.f) : 1.f;
    const float lost = __int_as_float(0x7FC00000);
    S.m[tid] = m;
    S.l[tid] = ok ? l : lost;
#pragma unroll 1
    for (int d = 0; d < D; d += 32) {
      uint32_t o[32];
      if (steps)
        tmem_ld32(lanes + d, o);
      else
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = 0;
#pragma unroll
      for (int i = 0; i < 32; ++i)
        o[i] = __float_as_uint(ok ? __uint_as_float(o[i]) * f * unit : lost);
      if (Z > 1) {  // to where Q and K were: every product is done
#pragma unroll
        for (int i = 0; i < 32; i += 4)
          *reinterpret_cast<uint4*>(smem + part_at<D>(tid, (d + i) / 4)) =
              make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
      } else if (real) {
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          uint4 w;
          w.x = mm::pack_bf16(__uint_as_float(o[i]), __uint_as_float(o[i + 1]));
          w.y = mm::pack_bf16(__uint_as_float(o[i + 2]), __uint_as_float(o[i + 3]));
          w.z = mm::pack_bf16(__uint_as_float(o[i + 4]), __uint_as_float(o[i + 5]));
          w.w = mm::pack_bf16(__uint_as_float(o[i + 6]), __uint_as_float(o[i + 7]));
          *reinterpret_cast<uint4*>(out + d + i) = w;
        }
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ the pages
    // Warps 4 and 5 bring K, 6 and 7 V, each a step ahead in registers and two
    // in page numbers.
    constexpr int ES = I8 ? 1 : 2, CPR = D * ES / 16;  // 16-byte chunks of a row
    constexpr int R = kKeys * CPR / 64;                // chunks of a thread
    const bool isv = warp >= 6;
    const int t = tid - (isv ? 192 : 128);
    const uint8_t* const pool = isv ? P.vp : P.kp;
    uint8_t* const buf = isv ? sv : sk;
    uint64_t* const full = isv ? S.v_full : S.k_full;
    uint64_t* const empty = isv ? S.v_empty : S.k_empty;
    // Block base + lane's page, 32 blocks (8 steps) at a time, loaded a step
    // before it is looked at; from it the block's place in the pool, -1 for a
    // bad page, -2 past the keys.
    auto page_of = [&](int base) {
      const int blk = key0 / kBlock + base + lane;
      return blk * kBlock < keys ? __ldcg(P.table + (long long)it.b * P.max_pages + blk / P.bpp)
                                 : -1;
    };
    auto place_of = [&](int base, int page) {
      const int blk = key0 / kBlock + base + lane;
      if (blk * kBlock >= keys) return -2;
      return page >= 0 && page < P.num_pages
                 ? (page * P.Hkv + it.h) * P.bpp + (blk - blk / P.bpp * P.bpp)
                 : -1;
    };
    // Thread t's chunk i: 64 / CPR rows further than chunk i - 1, the same
    // place in the row; 64 chunks never pass a block of 16 rows.
    const int row0 = t / CPR, cc = t % CPR;
    const auto wait_empty = [&](int j) {
      return j < 2 || wait_bar(&empty[j & 1], (uint32_t)((j >> 1) + 1) & 1u, abort);
    };
    int page = page_of(0), places = place_of(0, page);
    const auto look = [&](int j) {  // before step j's loads
      if (j % 8 == 7) page = page_of(4 * (j + 1));
      if (j % 8 == 0) places = place_of(4 * j, page);
    };
    if constexpr (I8) {
      uint4 x[R];
      float scale = 1.f, vscale = 1.f;  // lanes 0-3 of warp 4; a bad page gives NaN scores
      auto load = [&](int j) {
        const int from = j * 4 % 32;  // the step's blocks: lanes from .. from + 3
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int blk = __shfl_sync(0xffffffffu, places, from + i * 64 / (kBlock * CPR));
          x[i] = load16_if(pool + (long long)blk * (kBlock * D) + (i * 64 % (kBlock * CPR) + t) * 16,
                           blk >= 0);
        }
        const int id = __shfl_sync(0xffffffffu, places, from + (lane & 3));
        const bool scaled = warp == 4 && id >= 0;
        scale = load_if(P.ks + id, scaled, id == -1 ? __int_as_float(0x7FC00000) : 1.f);
        vscale = load_if(P.vs + id, scaled, 0.f);  // (no block: nothing sets the unit of V)
      };
      if (steps) load(0);
      for (int j = 0; j < steps; ++j) {
        const int b = j & 1;
        if (!wait_empty(j)) {
          ok = false;
          break;
        }
        uint8_t* const dst = buf + b * L::kKV;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int row = i * (64 / CPR) + row0;
          const uint32_t w[4] = {x[i].x ^ 0x80808080u, x[i].y ^ 0x80808080u, x[i].z ^ 0x80808080u,
                                 x[i].w ^ 0x80808080u};
          *reinterpret_cast<uint4*>(dst + at_chunk<kKeys>(row, 2 * cc)) =
              make_uint4(codes01(w[0]), codes23(w[0]), codes01(w[1]), codes23(w[1]));
          *reinterpret_cast<uint4*>(dst + at_chunk<kKeys>(row, 2 * cc + 1)) =
              make_uint4(codes01(w[2]), codes23(w[2]), codes01(w[3]), codes23(w[3]));
        }
        // A ring of four steps. The rows read a step's scales once its S is full,
        // before V need be there, so K's warps bring V's scales too.
        if (!isv && t < 4) {
          S.scale[j & 3][t] = scale;
          S.scale[j & 3][4 + t] = vscale;
        }
        fence_async();
        mbar_arrive(&full[b]);
        if (j + 1 < steps) {
          look(j + 1);
          load(j + 1);
        }
      }
    } else {
      // bf16 values go to shared memory as they are, by asynchronous copies a
      // step ahead (through registers the two steps in flight took 64 of them).
      const uint32_t to = smem_u32(buf);
      auto send = [&](int j) {
        if (!wait_empty(j)) return false;
        const int from = j * 4 % 32;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int blk = __shfl_sync(0xffffffffu, places, from + i * 64 / (kBlock * CPR));
          const int row = i * (64 / CPR) + row0;
          const bool in = blk >= 0 && (!isv || key0 + j * kKeys + row < it.len);
          const uint8_t* p = pool + (long long)(in ? blk : 0) * (kBlock * D * ES) +
                             (i * 64 % (kBlock * CPR) + t) * 16;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                           to + (uint32_t)((j & 1) * L::kKV + at_chunk<kKeys>(row, cc))),
                       "l"(p), "r"(in ? 16 : 0)
                       : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        // (the ring's place of step j - 4: its rows are done, or S of step j - 2
        // would not have been issued)
        const int id = __shfl_sync(0xffffffffu, places, from + (lane & 3));
        if (!isv && t < 4) S.scale[j & 3][t] = id == -1 ? __int_as_float(0x7FC00000) : 1.f;
        return true;
      };
      // values of V that are not finite out of the operand, each thread its own
      auto leave_out = [&](uint8_t* dst) {
#pragma unroll 1
        for (int i = 0; i < R; ++i) {
          uint4* const at =
              reinterpret_cast<uint4*>(dst + at_chunk<kKeys>(i * (64 / CPR) + row0, cc));
          const uint4 x = *at;
          uint32_t w[4] = {x.x, x.y, x.z, x.w};
          bool odd = false;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool hi = (w[e] & 0x7F800000u) == 0x7F800000u, lo = (w[e] & 0x7F80u) == 0x7F80u;
            odd |= hi || lo;
            if (hi) w[e] &= 0xFFFFu;
            if (lo) w[e] &= 0xFFFF0000u;
          }
          if (!odd) continue;
          *at = make_uint4(w[0], w[1], w[2], w[3]);
          S.odd = 1;
        }
      };
      if (steps) ok = send(0);
      for (int j = 0; ok && j < steps; ++j) {
        if (j + 1 < steps) {
          look(j + 1);
          if (!send(j + 1)) {
            ok = false;
            break;
          }
          asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
          asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        // (some rows do not see all of a partly masked step's tokens)
        if (isv && key0 + j * kKeys + kKeys > common) leave_out(buf + (j & 1) * L::kKV);
        fence_async();
        mbar_arrive(&full[j & 1]);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
    if (!ok) *abort = 1;
  } else {
    // --------------------------------------------------------- the products
    // The whole warp walks the loop and one elected lane issues, so that
    // addresses and descriptors stay in uniform registers (a branch on the lane
    // number cost 160 cycles a product in place of about 70).
    const uint32_t base = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t is = I8 ? instr_desc_f16<kKeys>() : instr_desc<kKeys>();
    const uint32_t ip = (I8 ? instr_desc_f16<D>() : instr_desc<D>()) | kBisMnMajor;
    // (addresses in a descriptor are in units of 16 bytes; 16 dims are 32
    // bytes of a K-major row, 16 tokens two groups of an MN-major panel)
    const uint64_t dq = smem_desc(smem_u32(sq)), dk = smem_desc(smem_u32(sk));
    const uint64_t dv = mn_desc(smem_u32(sv), kKeys * 128);
    auto wait = [&](uint64_t* bar, int parity) {
      ok = __all_sync(0xffffffffu, wait_bar(bar, (uint32_t)parity & 1u, abort));
      fence_after();
      return ok;
    };
    auto issue_s = [&](int j) {
      const int b = j & 1;
      if (!wait(&S.k_full[b], j >> 1)) return;
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t da = dq + (uint64_t)((k / 4) * (kRows * 8) + 2 * (k % 4));
          const uint64_t db =
              dk + (uint64_t)(b * (L::kKV / 16) + (k / 4) * (kKeys * 8) + 2 * (k % 4));
          asm volatile(
              "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
              " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(
                  base + (uint32_t)(kScol + 64 * b)),
              "l"(da), "l"(db), "r"(is), "r"(k > 0 ? 1u : 0u)
              : "memory");
        }
        commit(&S.s_full[b]);
        commit(&S.k_empty[b]);
      }
      __syncwarp();
    };
    if (wait(&S.q_full, 0) && steps) issue_s(0);
    for (int j = 0; ok && j < steps; ++j) {
      const int b = j & 1;
      if (j + 1 < steps) issue_s(j + 1);
      if (!ok || !wait(&S.p_full[b], j >> 1) || !wait(&S.v_full[b], j >> 1)) break;
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k) {
          const uint64_t db = dv + (uint64_t)(b * (L::kKV / 16) + k * 128);
          asm volatile(
              "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
              " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(base),
              "r"(base + (uint32_t)(kScol + 64 * b + 8 * k)), "l"(db), "r"(ip),
              "r"(j > 0 || k > 0 ? 1u : 0u)
              : "memory");
        }
        commit(&S.v_empty[b]);
        commit(&S.o_full);
      }
      __syncwarp();
    }
    if (!ok) {  // products in flight end before tensor memory is given back
      *abort = 1;
      if (elect_one()) commit(&S.drain);
      __syncwarp();
      const unsigned long long t0 = now_ns();
      while (!mbar_try_wait(&S.drain, 0))
        if (now_ns() - t0 > kWaitNs) break;
    }
  }
  fence_before();
  if (Z > 1)
    cluster_sync();
  else
    __syncthreads();
  if (warp == 8) {
    __syncwarp();
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
  }
  // place of one of the tile's pairs in out
  const auto out_at = [&](int pair) {
    const int cp = first + pair, rp = cp / P.G;
    return reinterpret_cast<uint16_t*>(P.out) +
           ((long long)(it.r0 + rp) * P.H + it.h * P.G + (cp - rp * P.G)) * D;
  };
  int odd = S.odd;
  const int mine = kRows / Z;  // pairs that this CTA writes
  if (Z > 1) {
    if (Z == 2)
      odd = join<D, 2>(S, smem, z, first, cols, out_at);
    else if (Z == 4)
      odd = join<D, 4>(S, smem, z, first, cols, out_at);
    else
      odd = join<D, 8>(S, smem, z, first, cols, out_at);
    cluster_sync();  // nobody ends while its shared memory is read
  }
  if (!I8 && odd) {  // (rare) V values that were left out, to the rows that see them
    __syncthreads();
    const int pair = z * mine + tid, seen = before + (first + pair) / P.G + 1;
    if (tid >= mine || first + pair >= cols) return;
    uint16_t* const o = out_at(pair);
#pragma unroll 1
    for (int d = 0; d < D; d += 8) {
      float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int key = common / kKeys * kKeys; key < seen; ++key) {
        const int blk = key / kBlock, pi = blk / P.bpp;
        const int page = __ldcg(P.table + (long long)it.b * P.max_pages + pi);
        if (page < 0 || page >= P.num_pages) continue;
        const long long row =
            ((long long)(page * P.Hkv + it.h) * P.bpp + (blk - pi * P.bpp)) * kBlock + key % kBlock;
        const uint4 w = __ldcg(reinterpret_cast<const uint4*>(P.vp + (row * D + d) * 2));
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t bits = e & 1 ? x[e / 2] & 0xFFFF0000u : x[e / 2] << 16;
          if ((bits & 0x7F800000u) == 0x7F800000u) sum[e] += __uint_as_float(bits);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (sum[e] != 0.f)
          o[d + e] = f32_to_bf16_bits(bf16_bits_to_f32(o[d + e]) + sum[e]);
    }
  }
}

// CTAs of a cluster that share a tile's keys: as many as fit the GPU at once
// (two an SM) with four steps each, should the sequences fill their pages.
// Measured with 1, 2, 4 and 8 (us): 128 rows over 32768 tokens 698, 310, 182,
// 119; 512 over 8192 148, 82, 67, 95; 2053 rows of five users 50, 55, 100, 208;
// 300 rows over themselves 14, 15, 20, 37. (Page tables far wider than the
// sequences get the larger ones: 300 rows with room for 32768 tokens 20.)
static int prompt_cluster(const Params& P) {
  const long long tiles = ((long long)P.T * P.G / kRows + P.B / 2 + 1) * P.Hkv;
  const long long steps = (long long)P.max_pages * P.bpp * kBlock / kKeys;
  int z = 1;
  while (z < 8 && tiles * 2 * z <= 2 * num_sms() && steps >= 8 * z) z *= 2;
  return z;
}

template <int D, bool I8>
static cudaError_t launch_prompt_kernel(const Params& P, cudaStream_t st) {
  const size_t smem = PromptSmem<D>::kBytes;
  static_assert(sizeof(PromptShared) <= PromptSmem<D>::kTail, "PromptShared fits behind the operands");
  ensure_smem((const void*)prompt_kernel<D, I8>, (int)smem);
  const long long slots = (long long)P.T * P.G / kRows + P.B;
  const int Z = prompt_cluster(P);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(slots * P.Hkv), 1, Z);
  cfg.blockDim = dim3(kPThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = Z;
  cfg.attrs = attr;
  cfg.numAttrs = Z > 1 ? 2 : 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, prompt_kernel<D, I8>, P);
}

cudaError_t launch_prompt(const Params& P, int D, bool i8, cudaStream_t st) {
  if (D == 64)
    return i8 ? launch_prompt_kernel<64, true>(P, st) : launch_prompt_kernel<64, false>(P, st);
  return i8 ? launch_prompt_kernel<128, true>(P, st) : launch_prompt_kernel<128, false>(P, st);
}

}  // namespace pa
}  // namespace qg
