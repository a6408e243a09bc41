// abi_common.h -- host-side helpers shared by the C-ABI translation units
// (abi.cu, abi_tree.cu): error text, argument checks, workspace carving.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "../../include/dflash.h"
#include "common.cuh"
#include "trace.h"

namespace dfl {

// Sets the thread-local error text (printf-style) and returns `code`.
int fail(int code, const char* fmt, ...);

#define DF_CHECK(cond, ...)                                 \
  do {                                                      \
    if (!(cond)) return fail(DFLASH_ERR_INVALID_ARG, __VA_ARGS__); \
  } while (0)

#define DF_CUDA(call)                                                                       \
  do {                                                                                      \
    cudaError_t e_ = (call);                                                                \
    if (e_ != cudaSuccess) return fail(DFLASH_ERR_CUDA, "%s: %s", #call, cudaGetErrorString(e_)); \
  } while (0)

// Launch with optional tracing (family, algorithmic bytes).
#define DF_LAUNCH(st, fam, bytes, call)                                                     \
  do {                                                                                      \
    trace_pre((st), (fam));                                                                 \
    cudaError_t e_ = (call);                                                                \
    trace_post((st), (double)(bytes));                                                      \
    if (e_ != cudaSuccess) return fail(DFLASH_ERR_CUDA, "%s: %s", #call, cudaGetErrorString(e_)); \
  } while (0)

inline size_t elem_size(int dtype) { return dtype == DFLASH_BF16 ? 2 : 4; }

// Device pointers that the kernels read with 16-byte accesses.
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Carves a workspace into 256-byte aligned pieces; with base == nullptr it
// only measures.
struct Bump {
  char* base;
  size_t off = 0;
  explicit Bump(void* b) : base(static_cast<char*>(b)) {}
  void* take(size_t bytes) {
    off = (off + 255) & ~size_t(255);
    void* p = base ? base + off : nullptr;
    off += bytes;
    return p;
  }
};

inline int num_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
  return n;
}

inline int check_dims(const dflash_dims& d, const char* who) {
  DF_CHECK(d.dtype == DFLASH_F32 || d.dtype == DFLASH_BF16, "%s: dtype %d not F32/BF16", who, d.dtype);
  DF_CHECK(d.hidden > 0 && d.hidden % 8 == 0, "%s: hidden %d must be a positive multiple of 8", who, d.hidden);
  DF_CHECK(d.head_dim == 64 || d.head_dim == 128, "%s: head_dim %d must be 64 or 128", who, d.head_dim);
  DF_CHECK(d.n_q_heads > 0 && d.n_kv_heads > 0 && d.n_q_heads % d.n_kv_heads == 0,
           "%s: n_q_heads %d must be a positive multiple of n_kv_heads %d", who, d.n_q_heads, d.n_kv_heads);
  DF_CHECK(d.intermediate > 0 && d.intermediate % 8 == 0, "%s: intermediate %d must be a multiple of 8", who,
           d.intermediate);
  DF_CHECK((d.n_q_heads * d.head_dim) % 8 == 0, "%s: n_q_heads*head_dim must be a multiple of 8", who);
  DF_CHECK(d.vocab > 0, "%s: vocab must be positive", who);
  DF_CHECK(d.rms_eps >= 0.f && d.rope_theta > 0.f, "%s: rms_eps >= 0 and rope_theta > 0 required", who);
  return DFLASH_OK;
}

struct Ctx {
  uint32_t* status;
  uint32_t* counters;
};

inline Ctx header(void* ws) {
  Ctx c;
  c.status = static_cast<uint32_t*>(ws);
  c.counters = reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + kHeaderBytes);
  return c;
}

inline int check_ws(void* ws, size_t ws_bytes, size_t need, const char* who) {
  if (!ws) return fail(DFLASH_ERR_INVALID_ARG, "%s: workspace is NULL", who);
  if (ws_bytes < need)
    return fail(DFLASH_ERR_WORKSPACE, "%s: workspace %zu bytes, %zu required", who, ws_bytes, need);
  if ((reinterpret_cast<uintptr_t>(ws) & 255) != 0)
    return fail(DFLASH_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
  return DFLASH_OK;
}

// A paged cache: page size a multiple of the 128-key attention chunk,
// capacity == max_pages * page_size.
inline int check_kv_pages(const dflash_kv& kv, const char* who) {
  if (!kv.pages) return DFLASH_OK;
  DF_CHECK(kv.page_size > 0 && kv.page_size % 128 == 0, "%s: page_size must be a positive multiple of 128", who);
  DF_CHECK(kv.max_pages > 0 && kv.pool_pages > 0, "%s: max_pages and pool_pages must be positive", who);
  DF_CHECK((long)kv.max_pages * kv.page_size == kv.capacity, "%s: capacity must equal max_pages * page_size", who);
  DF_CHECK((long)kv.pool_pages * kv.page_size <= (1L << 30), "%s: page pool too large", who);
  return DFLASH_OK;
}

}  // namespace dfl
