// The paged K/V cache shared by qg_paged_kv_append, qg_paged_kv_gather and
// qg_paged_attention: host-side checks of a qg_paged_kv and the device
// helpers that map packed rows to sequences.
#pragma once

#include "qg_internal.cuh"

namespace qg {
namespace pk {

constexpr int kBlock = QG_KV_BLOCK;  // tokens that share one scale of an int8 page

// `who` names the entry point. Checks the pool and the page table's extent.
inline qg_status check_pool(const char* who, const qg_paged_kv* kv, int max_pages) {
  QG_REQUIRE(kv, QG_ERR_INVALID_ARGUMENT, "%s: null kv", who);
  QG_REQUIRE(kv->dtype == QG_KV_BF16 || kv->dtype == QG_KV_INT8, QG_ERR_INVALID_ARGUMENT,
             "%s: kv dtype=%d is neither QG_KV_BF16 nor QG_KV_INT8", who, (int)kv->dtype);
  QG_REQUIRE(kv->head_dim == 64 || kv->head_dim == 128 || kv->head_dim == 256,
             QG_ERR_UNSUPPORTED_SHAPE, "%s: head_dim=%d must be 64, 128 or 256", who,
             kv->head_dim);
  QG_REQUIRE(kv->kv_heads >= 1 && kv->kv_heads <= 1024, QG_ERR_UNSUPPORTED_SHAPE,
             "%s: kv_heads=%d must be in [1, 1024]", who, kv->kv_heads);
  QG_REQUIRE(kv->page_size >= kBlock && kv->page_size % kBlock == 0 && kv->page_size <= 65536,
             QG_ERR_UNSUPPORTED_SHAPE,
             "%s: page_size=%d must be a multiple of %d in [%d, 65536]", who, kv->page_size,
             kBlock, kBlock);
  QG_REQUIRE(kv->num_pages >= 0 && max_pages >= 0, QG_ERR_UNSUPPORTED_SHAPE,
             "%s: num_pages=%d max_pages=%d must be >= 0", who, kv->num_pages, max_pages);
  QG_REQUIRE((long long)max_pages * kv->page_size <= 0x7FFFFFFFLL - 65536,
             QG_ERR_UNSUPPORTED_SHAPE, "%s: max_pages=%d x page_size=%d tokens is too large", who,
             max_pages, kv->page_size);
  return QG_OK;
}

// The pool's pointers; needed as soon as a call has work.
inline qg_status check_pool_pointers(const char* who, const qg_paged_kv* kv) {
  QG_REQUIRE(kv->k_pages && kv->v_pages, QG_ERR_INVALID_ARGUMENT, "%s: null k_pages or v_pages",
             who);
  QG_REQUIRE(aligned(kv->k_pages, 16) && aligned(kv->v_pages, 16), QG_ERR_MISALIGNED,
             "%s: k_pages or v_pages not 16-byte aligned", who);
  if (kv->dtype == QG_KV_INT8) {
    QG_REQUIRE(kv->k_scales && kv->v_scales, QG_ERR_INVALID_ARGUMENT,
               "%s: null k_scales or v_scales with int8 pages", who);
    QG_REQUIRE(aligned(kv->k_scales, 4) && aligned(kv->v_scales, 4), QG_ERR_MISALIGNED,
               "%s: k_scales or v_scales not 4-byte aligned", who);
  }
  return QG_OK;
}

// Inputs may come from the kernel just before on the stream, so everything
// is read after pdl_wait() and through L2 (__ldcg), never as read-only data
// that the compiler may load earlier.

// First row of sequence b (b in [0, B]) of the packed batch of T rows. Row
// starts come from device memory, so they are clamped to [0, T]: a wrong one
// gives wrong rows, never an access out of bounds.
__device__ __forceinline__ int row_begin(const int32_t* row_start, int b, int T) {
  if (!row_start) return b;
  const int r = __ldcg(row_start + b);
  return r < 0 ? 0 : r > T ? T : r;
}

}  // namespace pk
}  // namespace qg
