// What the paged attention kernels share: parameters, the rows of a sequence,
// the units of int8 operands.
#pragma once

#include <cfloat>

#include "paged_kv.cuh"

namespace qg {
namespace pa {

using pk::kBlock;
using pk::row_begin;

constexpr float kMargin = 4.f;  // log2 of how far a weight may pass 1

struct Params {
  const void* q;
  void* out;
  const uint8_t* kp;
  const uint8_t* vp;
  const float* ks;
  const float* vs;
  const int32_t* table;
  const int32_t* kv_len;
  const int32_t* row_start;
  float* part;  // [2 * pieces][NC * (D + 2)]
  int q_bf16, out_bf16;
  int B, T, H, Hkv, G, bpp, max_pages, num_pages;  // bpp: blocks of 16 tokens per page
  int pieces;
  float scale_log2;
};

// Prompts on the tcgen05 tensor cores (paged_attention_tc.cu): bf16 q and
// out, head size 64 or 128.
cudaError_t launch_prompt(const Params& P, int D, bool i8, cudaStream_t st);

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 (8) bytes through L2, or zeros: a predicated load, since a choice made
// after the load would wait for it.
__device__ __forceinline__ uint4 load16_if(const uint8_t* p, bool in) {
  uint4 v;
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %5, 0;\n"
      " mov.b32 %0, 0;\n mov.b32 %1, 0;\n mov.b32 %2, 0;\n mov.b32 %3, 0;\n"
      " @p ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];\n}\n"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"((int)in));
  return v;
}
__device__ __forceinline__ uint2 load8_if(const uint8_t* p, bool in) {
  uint2 v;
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %3, 0;\n"
      " mov.b32 %0, 0;\n mov.b32 %1, 0;\n"
      " @p ld.global.cg.v2.u32 {%0, %1}, [%2];\n}\n"
      : "=&r"(v.x), "=&r"(v.y)
      : "l"(p), "r"((int)in));
  return v;
}
// A float through L2, or `other`.
__device__ __forceinline__ float load_if(const float* p, bool in, float other) {
  float v;
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %2, 0;\n mov.b32 %0, %3;\n"
      " @p ld.global.cg.f32 %0, [%1];\n}\n"
      : "=&f"(v)
      : "l"(p), "r"((int)in), "f"(other));
  return v;
}

// One (sequence, KV head, column tile) item.
struct Item {
  int b, h, ct;   // sequence, KV head, column tile
  int r0, n;      // the sequence's first packed row and rows
  int len;        // cached tokens, 0 for a length out of range
};

__device__ __forceinline__ void set_seq(const Params& P, Item& it, int b) {
  it.b = b;
  it.r0 = row_begin(P.row_start, b, P.T);
  it.n = max(0, row_begin(P.row_start, b + 1, P.T) - it.r0);
  const int len = __ldcg(P.kv_len + b);
  it.len = len >= it.n && (long long)len <= (long long)P.max_pages * P.bpp * kBlock ? len : 0;
}

// 2^e that brings the largest |q| into [2^13, 2^14) (int8 pages).
__device__ __forceinline__ float q_unit(float top) {
  const int ex = (__float_as_int(top) >> 23) & 255;  // 0: zero or subnormal, 255: not finite
  if (ex == 0 || ex == 255) return 1.f;
  return __int_as_float(min(254, max(1, 127 + 13 - (ex - 127))) << 23);
}

}  // namespace pa
}  // namespace qg
