// prompt_attn.cuh -- device helper of the prompt attention kernels.
#pragma once
#include "common.cuh"
#include "internal.h"

namespace dfl {

// What a layer asks for besides the attention, done by every thread of the
// grid (thread i of n): positions outside the RoPE table are reported; rows of
// no sequence get an output of 0.  good: row_start is in order.
template <typename T>
__device__ __forceinline__ void prompt_layer_rows(const PromptAttnDesc& a, bool good, long long i, long long n) {
  if (a.pos)
    for (long long m = i; m < a.M; m += n)
      if ((uint32_t)__ldg(a.pos + m) >= (uint32_t)a.pos_end) raise_status(a.status, ST_RANGE);
  if (!a.zero_pad) return;
  const long long r0 = good ? __ldg(a.row_start) : 0, r1 = good ? __ldg(a.row_start + a.n_seqs) : 0;
  const long long per = (long long)a.nq * a.d * (int)sizeof(T) / 16, out = a.M - (r1 - r0);
  for (long long k = i; k < out * per; k += n) {
    const long long m = k / per < r0 ? k / per : k / per + (r1 - r0);
    if (!DFL_CHECK(m >= 0 && m < a.M, a.status)) continue;
    reinterpret_cast<uint4*>(a.out)[m * per + k % per] = make_uint4(0, 0, 0, 0);
  }
}

}  // namespace dfl
