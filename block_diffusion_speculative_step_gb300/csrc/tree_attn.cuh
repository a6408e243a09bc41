// tree_attn.cuh -- device helpers of the tree attention kernels.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace dfl {

// The rows a tree row sees: bit j of w for itself and every ancestor.  par:
// the parents (shared memory), null for the chain.  False: a padding row;
// *bad: a parent that is neither a row before it, -1 nor padding.
__device__ __forceinline__ bool tree_row_mask(const int* par, int row, uint32_t (&w)[4], bool* bad) {
  if (par == nullptr) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = row + 1 - 32 * i;
      w[i] = n >= 32 ? 0xffffffffu : n > 0 ? (1u << n) - 1u : 0u;
    }
    return true;
  }
  int j = row;
  for (;;) {  // parents strictly decrease: at most row + 1 steps
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if ((j >> 5) == i) w[i] |= 1u << (j & 31);
    const int p = par[j];
    if (p == -1) return true;
    if (p < 0 || p >= j) {
      *bad = p != DFLASH_TREE_PAD;
      return false;
    }
    j = p;
  }
}

// Eight elements e .. e+7 of 8-bit cache row `row`.
__device__ __forceinline__ void load8_e4m3(const void* codes, const uint8_t* ex, size_t row, int d, int e,
                                           float (&v)[8]) {
  const uint2 c = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(codes) + row * d + e);
  const float sc = __int_as_float((int)__ldg(ex + row) << 23);  // 2^(exp - 127)
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((w[j >> 1] >> (16 * (j & 1))) & 0xFFFFu), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    v[2 * j] = f.x * sc;
    v[2 * j + 1] = f.y * sc;
  }
}

}  // namespace dfl
