// k_logprobs.cu -- log probabilities of given tokens, entropies and the best
// alternatives of rows of logits (see dflash_token_logprobs).
//
// A row is cut into contiguous slices, one per CTA of a cluster; a slice is
// read once.  Each thread keeps a running maximum m, z = sum 2^d and s = sum d
// 2^d over d = c (x - m), c = log2(e) / T, from which
//   log p(t) = (x_t - m) / T - ln z,   H = ln z - ln 2 * s / z.
// ln z is log1p of z without the maximum's own 1, which stays out of the sums
// (lp_join_sums): a token of probability 1 - p has a log probability of about -p.
// The alternatives: the topk-th largest of 32 groups' maxima bounds the topk-th
// largest element from below, and few elements reach it (of 32 groups 31 for
// topk = 20, by the chances of hitting 20 of 32 groups).  They are gathered in
// shared memory, where each counts the larger ones: its rank.  A slice of at
// most kLpHold pieces a thread stays in registers; of a longer one a thread
// keeps the maxima of four quarters (units), and warps read those again that
// reach the bound (L2).  Ties, sorted rows and rows of few finite logits may
// bring more candidates than the list holds: then warps insert them into
// sorted lists of 32, one entry per lane, at worst over a second pass.
//
// Long calls are bound by HBM (512 rows x 151936: 61 us, 76% of the copy rate;
// a CTA's next 32 KB are in flight while it exponentiates, two CTAs an SM),
// short ones by latency (one row: 6 us).  Bounds by sorting every thread's
// maximum and insertion of every candidate took 68 and 10 us.
#include <cooperative_groups.h>
#include <float.h>
#include <math.h>

#include <atomic>

#include "attn_tc.cuh"
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"

namespace cg = cooperative_groups;

namespace dfl {

namespace {

constexpr int kLpThreads = 512;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpUnits = 4;        // quarters of a thread's elements
constexpr int kLpHold = 10;        // 16-byte pieces a thread keeps in registers
constexpr int kLpList = 512;       // candidates
constexpr int kLpMaxCluster = 8;
constexpr int kLpGroup = kLpThreads / 32;  // threads of a group

struct LpShared {
  float m[kLpWarps], z[kLpWarps], s[kLpWarps];
  float own[kLpWarps];             // z of the lane that holds the maximum (z: the others')
  int who[kLpWarps];               // that lane
  float row[4];                    // the slice's m, z, s, z - 1 (read by the cluster's first CTA)
  float out[2];                    // the row's m, ln z (NaN: no distribution)
  uint32_t group[32];              // groups' maxima
  uint64_t best[32];               // the slice's best (read by the cluster's first CTA)
  int n_units, n_list;
  union {
    uint64_t list[kLpList];        // candidates, (order of the logit, ~index)
    uint64_t lists[kLpWarps][32];  // sorted lists, where the candidates are more
  };
  uint16_t unit[kLpThreads * kLpUnits];
  float unit_max[kLpUnits][kLpThreads];
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

// The larger of two numbers, NaN if one is.
__device__ __forceinline__ float lp_max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

// (z, s) moved from reference m to n >= m.
__device__ __forceinline__ void lp_move(float m, float n, float c, float& z, float& s) {
  const float d = fmaxf((m - n) * c, -256.f), f = lp_ex2(d);  // (2^-256 is 0; d * z must not become inf * 0)
  s = f * fmaf(d, z, s);
  z *= f;
}

// (x - m) / T: by halves, whose difference stays in range.
__device__ __forceinline__ float lp_over_t(float x, float m, float invT) {
  return (0.5f * x - 0.5f * m) * (2.f * invT);
}

// A row's logits in 16-byte pieces from its first aligned address on; what lies
// outside the row is -inf.
struct LpRow {
  const float* p;  // 16-byte aligned, `lead` elements before the row
  int lead, V, pieces;
  uint32_t* status;
  __device__ __forceinline__ float4 load(int v) const {
    if (!DFL_CHECK((uint32_t)v < (uint32_t)pieces, status)) return make_float4(NAN, NAN, NAN, NAN);
    if ((uint32_t)(v - 1) < (uint32_t)(pieces - 2)) return __ldg(reinterpret_cast<const float4*>(p) + v);
    const int e = 4 * v - lead;
    float x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = e + k >= 0 && e + k < V ? __ldg(p + 4 * v + k) : -INFINITY;
    return make_float4(x[0], x[1], x[2], x[3]);
  }
};

// (z, s, m) with N more pieces' elements, whose maximum is mx; two elements an
// instruction where the pipes allow.
template <int N>
__device__ __forceinline__ void lp_add(const float4 (&x)[N], float mx, float c, float& m, unsigned long long& z,
                                       unsigned long long& s) {
  if (mx > m) {
    float z0, z1, s0, s1;
    tt_unpair(z, z0, z1);
    tt_unpair(s, s0, s1);
    lp_move(m, mx, c, z0, s0);
    lp_move(m, mx, c, z1, s1);
    z = tt_pair(z0, z1);
    s = tt_pair(s0, s1);
    m = mx;
  }
  const unsigned long long m2 = tt_pair(-m, -m), c2 = tt_pair(c, c);
#pragma unroll
  for (int k = 0; k < N; ++k) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float a, b;
      tt_unpair(tt_mul2(tt_add2(e ? tt_pair(x[k].z, x[k].w) : tt_pair(x[k].x, x[k].y), m2), c2), a, b);
      a = lp_max_nan(a, -256.f);  // (2^-256 is 0; -inf * 0 would be NaN)
      b = lp_max_nan(b, -256.f);
      const unsigned long long w = tt_pair(lp_ex2(a), lp_ex2(b));
      z = tt_add2(z, w);
      s = tt_fma2(tt_pair(a, b), w, s);
    }
  }
}

// A warp's sums joined, in a fixed order, the same in every lane.  The part
// `own` of the lane that holds the maximum, which has the maximum's own 1 in it,
// stays apart from the sum of everything else: beside 1 the small terms of a
// nearly certain token would be lost, and they are its ln z.  Returns that lane.
__device__ __forceinline__ int lp_join_sums(float c, float& m, float& z, float& s, float& own) {
  const float mw = warp_max(m);
  const int owner = __ffs(__ballot_sync(0xffffffffu, m == mw)) - 1;
  const bool mine = (int)(threadIdx.x & 31) == owner;
  float t = mine ? z : z + own;
  lp_move(m, mw, c, t, s);
  if (mine) s = fmaf(0.f, own, s);  // (NaN where own is; the maximum's own term is 0)
  m = mw;
  own = __shfl_sync(0xffffffffu, own, owner);
  z = warp_sum(t);
  s = warp_sum(s);
  return owner;
}

// HOLD: the slice stays in registers.
template <bool HOLD>
__global__ void __launch_bounds__(kLpThreads, HOLD ? 1 : 2) logprob_kernel(const __grid_constant__ LogprobDesc d) {
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
    row.status = d.status;
    row.pieces = (row.lead + d.V + 3) >> 2;
  }
  const float c = d.invT * 1.4426950408889634f;
  const int per = (row.pieces + nc - 1) / nc;
  const int v0 = min(rank * per, row.pieces), n = min(per, row.pieces - v0);
  constexpr int kStep = 4 * kLpThreads;  // pieces of a block: four a thread
  const int blocks = (n + kStep - 1) / kStep, q = (blocks + kLpUnits - 1) / kLpUnits;  // of the slice, of a unit
  const float4 none = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
  auto max_of = [](const float4& x) { return fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)); };
  if (tid == 0) sh.n_units = sh.n_list = 0;
  if (tid < 32) sh.best[tid] = 0;

  float m = -FLT_MAX, tm = -INFINITY;
  unsigned long long z2 = 0, s2 = 0;
  float4 held[HOLD ? kLpHold : 1];
  if constexpr (HOLD) {
#pragma unroll
    for (int k = 0; k < kLpHold; ++k)
      held[k] = tid + k * kLpThreads < n ? row.load(v0 + tid + k * kLpThreads) : none;
#pragma unroll
    for (int k = 0; k < kLpHold; ++k) tm = fmaxf(tm, max_of(held[k]));
    lp_add(held, tm, c, m, z2, s2);
  } else {
    auto fetch = [&](float4 (&x)[4], int b) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int v = b * kStep + k * kLpThreads + tid;
        x[k] = v < n ? row.load(v0 + v) : none;
      }
    };
    float um = -INFINITY;
    int left = q, u = 0;
    auto use = [&](const float4 (&x)[4], int b) {
      const float mx = fmaxf(fmaxf(max_of(x[0]), max_of(x[1])), fmaxf(max_of(x[2]), max_of(x[3])));
      um = fmaxf(um, mx);
      lp_add(x, mx, c, m, z2, s2);
      if (--left == 0 || b + 1 == blocks) {
        if (DFL_CHECK(u < kLpUnits, d.status)) sh.unit_max[u][tid] = um;
        ++u;
        tm = fmaxf(tm, um);
        um = -INFINITY;
        left = q;
      }
    };
    float4 x[4], y[4];  // the next block's loads are in flight
    if (blocks > 0) fetch(x, 0);
#pragma unroll 1
    for (int b = 0; b < blocks; b += 2) {
      if (b + 1 < blocks) fetch(y, b + 1);
      use(x, b);
      if (b + 1 == blocks) break;
      if (b + 2 < blocks) fetch(x, b + 2);
      use(y, b + 1);
    }
  }
  float z, s;
  {
    float z1, s1;
    tt_unpair(z2, z, z1);
    tt_unpair(s2, s, s1);
    z += z1;
    s += s1;
  }

  // ---- the slice's sums
  float gm = tm;
#pragma unroll
  for (int o = kLpGroup / 2; o > 0; o >>= 1) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, o));
  if (tid % kLpGroup == 0) sh.group[tid / kLpGroup] = lp_key(gm);
  float own = z;
  z = 0.f;
  const int who = lp_join_sums(c, m, z, s, own);
  if (lane == 0) {
    sh.m[warp] = m;
    sh.z[warp] = z;
    sh.s[warp] = s;
    sh.own[warp] = own;
    sh.who[warp] = who;
  }
  __syncthreads();
  if (warp == 0) {
    m = lane < kLpWarps ? sh.m[lane] : -FLT_MAX;
    z = lane < kLpWarps ? sh.z[lane] : 0.f;
    s = lane < kLpWarps ? sh.s[lane] : 0.f;
    own = lane < kLpWarps ? sh.own[lane] : 0.f;
    const int w = lp_join_sums(c, m, z, s, own);
    float rest = own - 1.f;  // own without the maximum's 1
    if (own > 0.5f && z + own < 1.5f) {
      // a token holds most of the row: what that thread summed beside its 1, summed again without it
      rest = 0.f;
      for (int v = w * 32 + sh.who[w] + lane * kLpThreads; v < n; v += 32 * kLpThreads) {
        const float4 x = row.load(v0 + v);
        const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) rest += y[e] == m ? 0.f : lp_ex2(fmaxf((y[e] - m) * c, -256.f));
      }
      rest = warp_sum(rest);
    }
    if (lane == 0) {
      sh.row[0] = m;
      sh.row[1] = z + own;
      sh.row[2] = s;
      sh.row[3] = z + rest;
    }
  }

  // ---- the slice's best
  if (d.topk > 0) {
    const uint32_t bound = __shfl_sync(0xffffffffu, lp_sort(sh.group[lane]), d.topk - 1);
    auto key_of = [&](float y, int v, int e) {  // element e of piece v; 0: below the bound, or none of the row's
      const int id = 4 * (v0 + v) - row.lead + e;
      const uint32_t k = lp_key(y);
      return v < n && id >= 0 && id < d.V && k >= bound ? (uint64_t)k << 32 | (0xFFFFFFFFu - (uint32_t)id) : 0ull;
    };
    auto list = [&](const float4& x, int v) {
      const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint64_t key = key_of(y[e], v, e);
        if (!key) continue;
        const int at = atomicAdd(&sh.n_list, 1);
        if (at < kLpList) sh.list[at] = key;
      }
    };
    // each piece of the units that reach the bound, a unit per warp at a time
    auto units = [&](auto use) {
      for (int i = warp; i < sh.n_units && DFL_CHECK(i < kLpThreads * kLpUnits, d.status); i += kLpWarps) {
        const int t = sh.unit[i] / kLpUnits, b = sh.unit[i] % kLpUnits, end = min(n, (b + 1) * q * kStep);
        for (int v = b * q * kStep + t; v < end; v += 32 * kLpThreads) {
          const int at = v + lane * kLpThreads;
          use(at < end ? row.load(v0 + at) : none, at < end ? at : n);
        }
      }
    };
    if constexpr (HOLD) {
      if (lp_key(tm) >= bound)
#pragma unroll
        for (int k = 0; k < kLpHold; ++k)
          if (lp_key(max_of(held[k])) >= bound) list(held[k], tid + k * kLpThreads);
    } else {
#pragma unroll
      for (int b = 0; b < kLpUnits; ++b)
        if (b * q * kStep + tid < min(n, (b + 1) * q * kStep) && lp_key(sh.unit_max[b][tid]) >= bound) {
          const int at = atomicAdd(&sh.n_units, 1);
          if (DFL_CHECK(at < kLpThreads * kLpUnits, d.status)) sh.unit[at] = (uint16_t)(tid * kLpUnits + b);
        }
      __syncthreads();
      units(list);
    }
    __syncthreads();
    const int cand = sh.n_list;
    if (cand <= kLpList) {
      for (int i = tid; i < cand; i += kLpThreads) {
        const uint64_t key = sh.list[i];
        int r = 0;
#pragma unroll 8
        for (int j = 0; j < cand; ++j) r += sh.list[j] > key;
        if (r < d.topk && DFL_CHECK(r < 32, d.status)) sh.best[r] = key;
      }
    } else {
      uint64_t mine = 0;  // lane i: the warp's i-th best so far; 0: none
      auto insert = [&](const float4& x, int v) {
        const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint64_t key = key_of(y[e], v, e);
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
      };
      if constexpr (HOLD) {
#pragma unroll
        for (int k = 0; k < kLpHold; ++k) insert(held[k], tid + k * kLpThreads);
      } else {
        units(insert);
      }
      __syncthreads();  // (the candidates' list gives way to the warps' lists)
      lp_join(sh.lists, mine);
      if (warp == 0) sh.best[lane] = sh.lists[0][lane];
    }
  }

  // ---- the row's results, by the cluster's first CTA
  if (nc > 1) cl.sync();
  else __syncthreads();
  if (rank == 0) {
    if (warp == 0) {
      m = -FLT_MAX;
      z = s = own = 0.f;
      if (lane < nc) {
        const float* other = cl.map_shared_rank(&sh.row[0], lane);
        m = other[0];
        own = other[1];
        s = other[2];
        z = other[3];
      }
      const float mr = warp_max(m);
      const bool first = lane == __ffs(__ballot_sync(0xffffffffu, m == mr)) - 1;  // its maximum's 1 is left out
      lp_move(m, mr, c, own, s);
      const float rest = warp_sum(first ? z : own);
      s = warp_sum(s);
      m = mr;
      z = 1.f + rest;
      const bool bad = !(z > 0.5f && z < INFINITY);
      const float lnz = bad ? NAN : log1pf(rest);
      if (lane == 0) {
        sh.out[0] = m;
        sh.out[1] = lnz;
        if (bad) raise_status(d.status, ST_NUMERIC);
        if (d.entropy) d.entropy[m_row] = bad ? NAN : lnz - 0.6931471805599453f * (s / z);
        if (d.tokens) {
          const int tok = d.tokens[m_row];
          if (tok >= 0 && tok < d.V) d.logprob[m_row] = lp_over_t(__ldg(row.p + row.lead + tok), m, d.invT) - lnz;
          else if (tok != DFLASH_NO_TOKEN) raise_status(d.status, ST_RANGE);
        }
      }
    }
    if (d.topk > 0) {
      const int cand = nc * d.topk;  // (at most kLpMaxCluster * 32 <= kLpThreads)
      uint64_t key = 0;
      if (tid < cand) key = cl.map_shared_rank(&sh.best[0], tid / d.topk)[tid % d.topk];
      if (nc > 1 && tid < cand) sh.list[tid] = key;
      __syncthreads();
      const float mr = sh.out[0], lnz = sh.out[1];
      const size_t o = (size_t)m_row * d.topk;
      if (lnz != lnz) {  // no distribution
        if (tid < d.topk) {
          d.top_ids[o + tid] = -1;
          d.top_logprobs[o + tid] = NAN;
        }
      } else if (key) {
        int r = tid;
        if (nc > 1) {
          r = 0;
#pragma unroll 8
          for (int j = 0; j < cand; ++j) r += sh.list[j] > key;
        }
        if (r < d.topk && DFL_CHECK(m_row < d.M && 0xFFFFFFFFu - (uint32_t)key < (uint32_t)d.V, d.status)) {
          d.top_ids[o + r] = (int)(0xFFFFFFFFu - (uint32_t)key);
          d.top_logprobs[o + r] = lp_over_t(lp_value((uint32_t)(key >> 32)), mr, d.invT) - lnz;
        }
      }
    }
  }
  if (nc > 1) cl.sync();  // (the other CTAs' shared memory is read until here)
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobDesc& d, int num_sms, cudaStream_t st) {
  // A CTA per row where there are rows for every SM; fewer rows share out, as far
  // as all clusters run at once (wider ones find room on about two thirds of
  // the SMs).  V = 151936, 1 / 2 / 4 / 8 CTAs a row: 1 row 17.2 / 12.5 / 9.7 /
  // 7.8 us, 24 rows 17.5 / 12.9 / 10.3 / 15.6, 76 rows 18.6 / 13.8 / 21.1 / 44,
  // 152 rows 23.2 / 22.4 / 37 / 84.  (A slice of less than 2048 elements a CTA
  // is not worth the exchange.)
  int nc = 1;
  while (nc < kLpMaxCluster && d.V >= nc * 2 * 4 * kLpThreads &&
         (nc == 1 ? (long long)d.M * 2 <= num_sms : (long long)d.M * nc * 2 * 3 <= 2ll * num_sms))
    nc *= 2;
  const bool hold = ((d.V + 6) / 4 + nc - 1) / nc <= kLpHold * kLpThreads;  // (a row's pieces, wherever it begins)
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
  return cudaLaunchKernelEx(&cfg, hold ? logprob_kernel<true> : logprob_kernel<false>, d);
}

}  // namespace dfl
