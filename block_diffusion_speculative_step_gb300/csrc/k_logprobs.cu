// k_logprobs.cu -- log probabilities of given tokens, entropies and the best
// alternatives of rows of logits (see dflash_token_logprobs).
//
// A row is cut into contiguous slices, one per CTA of a cluster; a slice is
// read once.  Each thread keeps a running maximum m, z = sum 2^d and s = sum d
// 2^d over d = c (x - m), c = log2(e) / T, from which
//   log p(t) = (x_t - m) / T - ln z,   H = ln z - ln 2 * s / z.
// The alternatives need no second pass over the row: a thread also keeps the
// maxima of four quarters of its elements (units).  The topk-th largest of the
// threads' maxima bounds the topk-th largest element from below, so only the
// units that reach it, about topk of them, hold candidates; warps read those
// again (L2) and insert them into sorted lists of 32, one entry per lane.
// Ties, sorted rows and rows of equal logits only make more units qualify, up
// to a second pass over the row.
#include <cooperative_groups.h>
#include <float.h>
#include <math.h>

#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "launch.cuh"

namespace cg = cooperative_groups;

namespace dfl {

namespace {

constexpr int kLpThreads = 512;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpUnits = 4;        // quarters of a thread's elements
constexpr int kLpMaxCluster = 8;

struct LpShared {
  float m[kLpWarps], z[kLpWarps], s[kLpWarps];
  float row[3];                    // the slice's m, z, s (read by the cluster's first CTA)
  uint64_t list[kLpWarps][32];     // sorted lists; list[0]: the slice's (read by the cluster's first CTA)
  uint32_t best[kLpWarps][32];     // threads' maxima, sorted
  uint32_t bound;
  int n_units;
  uint16_t unit[kLpThreads * kLpUnits];
};

// Order of logits as unsigned numbers (-0 equals +0).
__device__ __forceinline__ uint32_t lp_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float lp_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) - 1u | 0x80000000u));
}

// One bitonic step: lanes with bit `o` clear keep the larger of the pair (desc) or the smaller.
template <typename K>
__device__ __forceinline__ K lp_step(K v, int o, bool desc) {
  const K w = __shfl_xor_sync(0xffffffffu, v, o);
  const bool low = (threadIdx.x & o) == 0;
  return (low == desc) == (v > w) ? v : w;
}
// A warp's 32 values in descending order.
template <typename K>
__device__ __forceinline__ K lp_sort(K v) {
#pragma unroll
  for (int n = 2; n <= 32; n *= 2)
#pragma unroll
    for (int o = n / 2; o > 0; o >>= 1) v = lp_step(v, o, n == 32 || (threadIdx.x & n) == 0);
  return v;
}
// The 32 largest of two descending lists, descending (w: the second list, lane i its entry 31 - i).
template <typename K>
__device__ __forceinline__ K lp_merge(K v, K w) {
  v = v > w ? v : w;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = lp_step(v, o, true);
  return v;
}
// The warps' descending lists merged into the first one's, in shared memory.
template <typename K>
__device__ __forceinline__ void lp_join(K (*list)[32], K mine) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  list[warp][lane] = mine;
#pragma unroll
  for (int n = kLpWarps / 2; n > 0; n >>= 1) {
    __syncthreads();
    if (warp < n) list[warp][lane] = mine = lp_merge(mine, list[warp + n][31 - lane]);
  }
  __syncthreads();
}

__device__ __forceinline__ float lp_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// (z, s) moved from reference m to n >= m.
__device__ __forceinline__ void lp_move(float m, float n, float c, float& z, float& s) {
  const float d = fmaxf((m - n) * c, -256.f), f = lp_ex2(d);  // (2^-256 is 0; d * z must not become inf * 0)
  s = f * fmaf(d, z, s);
  z *= f;
}

// A row's logits in 16-byte pieces from its first aligned address on; what lies
// outside the row is -inf.
struct LpRow {
  const float* p;  // 16-byte aligned, `lead` elements before the row
  int lead, V;
  __device__ __forceinline__ int pieces() const { return (lead + V + 3) >> 2; }
  __device__ __forceinline__ float4 load(int v) const {
    const int e = 4 * v - lead;
    if (e >= 0 && e + 4 <= V) return __ldg(reinterpret_cast<const float4*>(p) + v);
    float x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = e + k >= 0 && e + k < V ? __ldg(p + 4 * v + k) : -INFINITY;
    return make_float4(x[0], x[1], x[2], x[3]);
  }
};

__global__ void __launch_bounds__(kLpThreads) logprob_kernel(const __grid_constant__ LogprobDesc d) {
  __shared__ LpShared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int nc = cl.num_blocks(), rank = cl.block_rank(), m_row = blockIdx.x / nc;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_launch_dependents();
  LpRow row;
  {
    const float* base = d.logits + (size_t)m_row * d.V;
    row.lead = (int)((reinterpret_cast<uintptr_t>(base) & 15) >> 2);
    row.p = base - row.lead;
    row.V = d.V;
  }
  const float c = d.invT * 1.4426950408889634f;
  const int per = (row.pieces() + nc - 1) / nc;
  const int v0 = min(rank * per, row.pieces()), n = min(per, row.pieces() - v0);
  const int q = ((n + kLpThreads - 1) / kLpThreads + kLpUnits - 1) / kLpUnits;  // pieces of a thread and unit
  if (tid == 0) sh.n_units = 0;

  float m = -FLT_MAX, z = 0.f, s = 0.f, um[kLpUnits];
#pragma unroll
  for (int b = 0; b < kLpUnits; ++b) {
    um[b] = -INFINITY;
    const int end = min(n, (b + 1) * q * kLpThreads);
    for (int v = b * q * kLpThreads + tid; v < end; v += 4 * kLpThreads) {
      float4 x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        x[k] = v + k * kLpThreads < end ? row.load(v0 + v + k * kLpThreads)
                                        : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      float mx = -INFINITY;
#pragma unroll
      for (int k = 0; k < 4; ++k) mx = fmaxf(mx, fmaxf(fmaxf(x[k].x, x[k].y), fmaxf(x[k].z, x[k].w)));
      um[b] = fmaxf(um[b], mx);
      if (mx > m) {
        lp_move(m, mx, c, z, s);
        m = mx;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float y[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float t = (y[e] - m) * c, w = lp_ex2(t);
          z += w;
          s = fmaf(fmaxf(t, -256.f), w, s);
        }
      }
    }
  }

  // ---- the slice's and the row's sums, in a fixed order
  float mw = warp_max(m);
  lp_move(m, mw, c, z, s);
  z = warp_sum(z);
  s = warp_sum(s);
  if (lane == 0) {
    sh.m[warp] = mw;
    sh.z[warp] = z;
    sh.s[warp] = s;
  }
  __syncthreads();
  if (warp == 0) {
    m = lane < kLpWarps ? sh.m[lane] : -FLT_MAX;
    z = lane < kLpWarps ? sh.z[lane] : 0.f;
    s = lane < kLpWarps ? sh.s[lane] : 0.f;
    mw = warp_max(m);
    lp_move(m, mw, c, z, s);
    z = warp_sum(z);
    s = warp_sum(s);
    if (lane == 0) {
      sh.row[0] = mw;
      sh.row[1] = z;
      sh.row[2] = s;
    }
  }

  // ---- the slice's best
  if (d.topk > 0) {
    float tm = um[0];
#pragma unroll
    for (int b = 1; b < kLpUnits; ++b) tm = fmaxf(tm, um[b]);
    lp_join(sh.best, lp_sort(lp_key(tm)));
    const uint32_t bound = sh.best[0][d.topk - 1];
#pragma unroll
    for (int b = 0; b < kLpUnits; ++b)
      if (b * q * kLpThreads + tid < min(n, (b + 1) * q * kLpThreads) && lp_key(um[b]) >= bound)
        sh.unit[atomicAdd(&sh.n_units, 1)] = (uint16_t)(tid * kLpUnits + b);
    __syncthreads();
    uint64_t mine = 0;  // lane i: the warp's i-th best so far, (order of the logit, ~index); 0: none
    for (int i = warp; i < sh.n_units; i += kLpWarps) {
      const int t = sh.unit[i] / kLpUnits, b = sh.unit[i] % kLpUnits, end = min(n, (b + 1) * q * kLpThreads);
      for (int v = b * q * kLpThreads + t; v < end; v += 32 * kLpThreads) {
        const int at = v + lane * kLpThreads;
        const float4 x = at < end ? row.load(v0 + at) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int id = 4 * (v0 + at) - row.lead + e;
          const uint32_t k32 = lp_key(y[e]);
          uint64_t key = at < end && id >= 0 && id < d.V && k32 >= bound ? (uint64_t)k32 << 32 | (0xFFFFFFFFu - (uint32_t)id) : 0;
          for (;;) {
            const uint64_t last = __shfl_sync(0xffffffffu, mine, d.topk - 1);
            const unsigned hit = __ballot_sync(0xffffffffu, key > last);
            if (!hit) break;
            const int w = __ffs(hit) - 1;
            const uint64_t add = __shfl_sync(0xffffffffu, key, w);
            const int pos = __popc(__ballot_sync(0xffffffffu, mine > add));
            const uint64_t up = __shfl_up_sync(0xffffffffu, mine, 1);
            mine = lane < pos ? mine : lane == pos ? add : up;
            if (lane == w) key = 0;
          }
        }
      }
    }
    lp_join(sh.list, mine);
  }

  // ---- the row's results, by the cluster's first CTA
  if (nc > 1) cl.sync();
  else __syncthreads();
  if (rank == 0 && warp == 0) {
    float* other = sh.row;
    m = -FLT_MAX;
    z = s = 0.f;
    if (lane < nc) {
      other = cl.map_shared_rank(&sh.row[0], lane);
      m = other[0];
      z = other[1];
      s = other[2];
    }
    mw = warp_max(m);
    lp_move(m, mw, c, z, s);
    z = warp_sum(z);
    s = warp_sum(s);
    const bool bad = !(z > 0.5f && z < INFINITY);
    const float lnz = bad ? NAN : logf(z);
    if (lane == 0) {
      if (bad) raise_status(d.status, ST_NUMERIC);
      if (d.entropy) d.entropy[m_row] = bad ? NAN : lnz - 0.6931471805599453f * (s / z);
      if (d.tokens) {
        const int tok = d.tokens[m_row];
        if (tok >= 0 && tok < d.V) d.logprob[m_row] = (__ldg(row.p + row.lead + tok) - mw) * d.invT - lnz;
        else if (tok != DFLASH_NO_TOKEN) raise_status(d.status, ST_RANGE);
      }
    }
    if (d.topk > 0) {
      uint64_t mine = sh.list[0][lane];
      for (int r = 1; r < nc; ++r) mine = lp_merge(mine, cl.map_shared_rank(&sh.list[0][0], r)[31 - lane]);
      if (lane < d.topk) {
        const size_t o = (size_t)m_row * d.topk + lane;
        d.top_ids[o] = bad ? -1 : (int)(0xFFFFFFFFu - (uint32_t)mine);
        d.top_logprobs[o] = bad ? NAN : (lp_value((uint32_t)(mine >> 32)) - mw) * d.invT - lnz;
      }
    }
  }
  if (nc > 1) cl.sync();  // (the other CTAs' shared memory is read until here)
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobDesc& d, int num_sms, cudaStream_t st) {
  int nc = 1;
  while (nc < kLpMaxCluster && (long long)d.M * nc * 2 <= 2ll * num_sms && d.V >= nc * 2 * 4 * kLpThreads) nc *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)d.M * nc);
  cfg.blockDim = dim3(kLpThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = nc;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  trace_kernel();
  return cudaLaunchKernelEx(&cfg, logprob_kernel, d);
}

}  // namespace dfl
