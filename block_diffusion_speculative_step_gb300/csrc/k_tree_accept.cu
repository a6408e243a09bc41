// k_tree_accept.cu -- acceptance over a drafted tree from given random
// numbers (speculative sampling with several candidates a level), and the
// tree of a cycle from per-position candidates.
//
// Walk: at a node with target row l and, for drawn candidates, the level's
// draft row g, p_0 = softmax(l / T), q_0 = softmax(g / T); child t (token
// x_t) is accepted iff u_t q_t(x_t) < p_t(x_t), else
//   p_{t+1} = max(0, p_t - q_t) / Z_t,  Z_t = sum_v max(0, p_t - q_t),
//   q_{t+1} = q_t without x_t, normalised again.
// Given p_t and q_t this emits x_t with probability min(p_t, q_t)(x_t) and
// leaves the rest of p_t's mass, so the token of the level is distributed as
// p_0 whatever the number of children.  Only rows on the path are read: one
// pass over l (and g) per level for the softmax sums, one more per rejected
// drawn candidate (Z_t), one for the last draw.
//
// One thread-block cluster per sequence, each CTA a contiguous slice of the
// vocabulary.  Partial sums are pushed to every CTA of the cluster through
// distributed shared memory, and every CTA joins them in the same tree order,
// so all CTAs take the same decisions and a call is deterministic.  Remaining
// masses are sums over what remains (children's weights are kept out of the
// row sums and added one by one): 1 - p(x) would lose all its digits when
// p(x) is close to 1.
//
// A walk is a chain of row passes and exchanges, each waiting for the one
// before: latency bounds it for few sequences, the row's bytes for many (a
// CTA's slice at its SM's share of the bandwidth).  So a thread has a batch of
// loads in flight at once (and the next one's during its sums), and the
// weights of a slice's first batch (10240 entries) stay in registers from the
// row sums to the tests and the draw; a slice's rest is read again, from L2.
// Measured, per level: about 1.2 us over 1021 entries (a third each: the loads
// and the children, the row sums, the remaining masses; a warp scan in fp32,
// as chains of fp64 additions took twice all that), 8 us over 37984 entries a
// CTA, the draw 10 us there.  151936 entries: one sequence 23 us, 32 sequences
// 54 us (the longest walk of five levels), with the row passes unbatched and
// partial sums pulled by every CTA 104 and 253 us.
#include <cooperative_groups.h>
#include <limits.h>

#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "launch.cuh"

namespace dfl {

namespace cg = cooperative_groups;

constexpr int kTaThreads = 512;
constexpr int kTaWarps = kTaThreads / 32;
// Entries per thread and batch: 20 (two rows of them and the next batch fill
// 128 registers), 4 for slices of at most 2048, whose threads would mostly
// work on entries that are not there.
constexpr int kTaE = 20, kTaShortE = 4;
constexpr int kTaMaxCluster = 16;

__device__ __forceinline__ float ta_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Weight exp((l - m) / T) = 2^(c (l - m)) of logit l against the row's maximum
// m, c = log2(e) / T (l == m also when both are infinite: the weight is then 1
// and the caller reports the row).  Beside the argument's rounding, which
// exp((l - m) * (1 / T)) has too, the hardware's 2^x adds 2^-22.
__device__ __forceinline__ float ta_weight(float l, float m, float c) {
  return l == m ? 1.f : ta_ex2((l - m) * c);
}

struct TaSum {  // maximum and sum of weights against it
  float m, s;
};
// The warp's maximum (no NaN), by an integer reduction: floats order as their
// bits, negative ones with all but the sign flipped.
__device__ __forceinline__ float ta_max(float x) {
  const int i = __float_as_int(x), r = __reduce_max_sync(0xffffffffu, i ^ ((i >> 31) & 0x7FFFFFFF));
  return __int_as_float(r ^ ((r >> 31) & 0x7FFFFFFF));
}
// Joined over the warp, bitwise the same in every lane.
__device__ __forceinline__ TaSum ta_join(TaSum a, float c) {
  const float m = ta_max(a.m);
  float s = a.s == 0.f ? 0.f : a.s * ta_weight(a.m, m, c);  // (a NaN stays)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return {m, s};
}
__device__ __forceinline__ void ta_best_join(float& b, int& v) {  // lowest index on equal values
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float ob = __shfl_xor_sync(0xffffffffu, b, o);
    const int ov = __shfl_xor_sync(0xffffffffu, v, o);
    if (ob > b || (ob == b && ov < v)) {
      b = ob;
      v = ov;
    }
  }
}

struct TaShared {
  int parent[DFLASH_MAX_TREE];
  int tok[DFLASH_MAX_TREE];
  float u[DFLASH_MAX_TREE];
  int n_child;
  int child[DFLASH_MAX_TREE];   // children of the current node, in row order
  int ctok[DFLASH_MAX_TREE];    // -1: out of range
  float cu[DFLASH_MAX_TREE];
  float cl[DFLASH_MAX_TREE];    // the children's target / draft logits (NaN: -inf)
  float cg[DFLASH_MAX_TREE];
  int cdup[DFLASH_MAX_TREE];    // an earlier sibling has the same token, or the token is out of range
  float cp[DFLASH_MAX_TREE];    // p_t of the child's token (drawn) or its weight; its weight in the draft row, 0 once removed
  float cq[DFLASH_MAX_TREE];
  float mp, mq;                 // the rows' maxima, children included
  int bad_child, bad;           // a child's logit, a row of the level is no number or +inf, or a whole row -inf
  float sufP[DFLASH_MAX_TREE + 1];  // mass of the target row without the tokens of children [0, t)
  float invZ[DFLASH_MAX_TREE];  // 1 / Z_t, 0: nothing left, p stays
  float invY[DFLASH_MAX_TREE];  // 1 / (remaining mass of q before step t), in q's weights
  TaSum wp[kTaWarps], wq[kTaWarps];
  float wb[kTaWarps];
  int wi[kTaWarps];
  float4 xs[2][kTaMaxCluster];  // pushed by the cluster's CTAs, by exchange parity: row sums; Z; (best, token)
};

template <bool Drawn, int E>
__global__ void __launch_bounds__(kTaThreads, 1) tree_accept_kernel(const __grid_constant__ TreeAcceptDesc d) {
  constexpr int BATCH = kTaThreads * E;
  __shared__ TaShared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int NC = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int s = blockIdx.x / NC;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int V = d.V, N = d.rows;
  const int per = ((V + NC - 1) / NC + 31) & ~31;
  const int v0 = min(V, rank * per), v1 = min(V, v0 + per);
  const float c2 = d.invT * 1.44269504f;  // log2(e) / T
  const float* target = d.target + (size_t)s * N * V;
  const float* draft = Drawn ? d.draft + (size_t)s * d.levels * V : nullptr;
  const float* noise = d.noise + (size_t)s * V;
  int par = 0;  // exchange parity
  if (NC > 1) cl.sync();  // (every CTA runs before the first push into it)
  pdl_wait();
  pdl_launch_dependents();

  // a CTA's contribution to all CTAs of the cluster, from warp 0; afterwards
  // lane r of every warp holds CTA r's
  auto exchange = [&](float4 x) __attribute__((always_inline)) {
    if (NC > 1) {
      if (warp == 0 && lane < NC) cl.map_shared_rank(&sh, lane)->xs[par][rank] = x;
      cl.sync();
    } else {
      if (tid == 0) sh.xs[par][0] = x;
      __syncthreads();
    }
    const float4 r = lane < NC ? sh.xs[par][lane] : make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
    par ^= 1;
    return r;
  };
  // entries b * BATCH + j * kTaThreads + tid of the slice: scalar loads,
  // coalesced whatever the row's alignment (rows of an odd V)
  auto load = [&](const float* row, int b, float (&x)[E]) __attribute__((always_inline)) {
    const int v = v0 + b * BATCH + tid;
    if (v0 + (b + 1) * BATCH <= v1) {
#pragma unroll
      for (int j = 0; j < E; ++j) x[j] = __ldg(row + v + j * kTaThreads);
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) x[j] = v + j * kTaThreads < v1 ? __ldg(row + v + j * kTaThreads) : -INFINITY;
    }
  };

  for (int i = tid; i < N; i += kTaThreads) {
    sh.parent[i] = d.parent ? d.parent[(size_t)s * N + i] : i - 1;
    sh.tok[i] = d.tokens[(size_t)s * N + i];
    sh.u[i] = d.u[(size_t)s * N + i];
  }
  // every sequence ends with one draw: its noise comes to L2 meanwhile
  for (int v = v0 + 32 * tid; v < v1; v += 32 * kTaThreads)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(noise + v));
  __syncthreads();

  int cur = 0, k = 0;
  if (rank == 0 && tid == 0) d.path[(size_t)s * N] = 0;
  for (;;) {
    const float* l = target + (size_t)cur * V;
    const bool deep = Drawn && k >= d.levels;  // no draft row for the node's children
    float lw[E], gw[E];                  // the first batch: logits, then weights, then p_t and q's weights
    load(l, 0, lw);
    if (Drawn && !deep) load(draft + (size_t)k * V, 0, gw);
    // ---- children of cur, in row order
    if (warp == 0) {
      int n = 0;
      for (int b = 0; b < N; b += 32) {
        const int i = b + lane;
        const bool c = i < N && i > 0 && i > cur && sh.parent[i] == cur;
        const unsigned bal = __ballot_sync(0xffffffffu, c);
        if (c) sh.child[n + __popc(bal & ((1u << lane) - 1u))] = i;
        n += __popc(bal);
      }
      if (deep) {
        if (n > 0 && rank == 0 && lane == 0) raise_status(d.status, ST_RANGE);
        n = 0;
      }
      if (lane == 0) sh.n_child = n;
      __syncwarp();
      bool odd = false;
      for (int c = lane; c < n; c += 32) {
        const int i = sh.child[c];
        int x = sh.tok[i];
        if (x < 0 || x >= V) {
          if (rank == 0) raise_status(d.status, ST_RANGE);
          x = -1;  // never accepted, nothing to remove
        }
        sh.ctok[c] = x;
        sh.cu[c] = sh.u[i];
        const float a = x >= 0 ? l[x] : -INFINITY, b = Drawn && x >= 0 ? draft[(size_t)k * V + x] : -INFINITY;
        odd |= !(a < INFINITY) || !(b < INFINITY);
        sh.cl[c] = a == a ? a : -INFINITY;
        if (Drawn) sh.cg[c] = b == b ? b : -INFINITY;
        int dup = x < 0;
        for (int e = 0; e < c; ++e) dup |= sh.tok[sh.child[e]] == x;
        sh.cdup[c] = dup;
      }
      odd = __any_sync(0xffffffffu, odd);
      if (lane == 0) sh.bad_child = odd;
    }
    __syncthreads();
    const int n_child = sh.n_child;
    const float* g = Drawn && n_child > 0 ? draft + (size_t)k * V : nullptr;
    if (Drawn && !g) {
#pragma unroll
      for (int j = 0; j < E; ++j) gw[j] = -INFINITY;
    }

    // ---- maxima and sums over the slice, the children's tokens left out
    // (a NaN or +inf logit makes the sum NaN, or the maximum infinite)
    auto find = [&](int b) __attribute__((always_inline)) {  // bit j: entry j of the batch is a child's token
      uint32_t mine = 0u;
      for (int c = 0; c < n_child; ++c) {
        const int x0 = sh.ctok[c];
        const unsigned rel = (unsigned)(x0 - v0 - b * BATCH);
        if (x0 >= 0 && rel < (unsigned)BATCH && (int)(rel % kTaThreads) == tid) mine |= 1u << (rel / kTaThreads);
      }
      return mine;
    };
    auto clean = [&](uint32_t mine, float (&x)[E]) __attribute__((always_inline)) {  // those: weight 0
      if (!__any_sync(0xffffffffu, mine != 0u)) return;
#pragma unroll
      for (int j = 0; j < E; ++j) x[j] = (mine >> j) & 1u ? -INFINITY : x[j];
    };
    const uint32_t mine0 = find(0);
    auto add = [&](TaSum& a, float (&x)[E]) __attribute__((always_inline)) {  // logits -> weights against the maximum so far
      float m = a.m;
#pragma unroll
      for (int j = 0; j < E; ++j) m = fmaxf(m, x[j]);
      if (a.s != 0.f) a.s *= ta_weight(a.m, m, c2);
      a.m = m;
      const float ref = m > -INFINITY ? m : 0.f;  // (all -inf: weights 0)
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int j = 0; j < E; ++j) {
        x[j] = ta_ex2((x[j] - ref) * c2);
        if (j & 1) s1 += x[j];
        else s0 += x[j];
      }
      a.s += s0 + s1;
    };
    auto row_sum = [&](const float* row, float (&w)[E], float* m0) __attribute__((always_inline)) {
      TaSum a = {-INFINITY, 0.f};
      float x[E];
      const bool more = v1 - v0 > BATCH;
      if (more) load(row, 1, x);
      clean(mine0, w);
      add(a, w);
      *m0 = a.m;
      for (int b = 1; v0 + b * BATCH < v1; ++b) {
        float y[E];
        load(row, b + 1, y);
        clean(find(b), x);
        add(a, x);
#pragma unroll
        for (int j = 0; j < E; ++j) x[j] = y[j];
      }
      return ta_join(a, c2);
    };
    float ml, mg = -INFINITY;  // what the first batch's weights refer to
    const TaSum ap = row_sum(l, lw, &ml);
    TaSum aq = {-INFINITY, 0.f};
    if (Drawn && g) aq = row_sum(g, gw, &mg);
    if (lane == 0) {
      sh.wp[warp] = ap;
      sh.wq[warp] = aq;
    }
    __syncthreads();
    TaSum P = {-INFINITY, 0.f}, Q = {-INFINITY, 0.f};
    if (NC == 1 || warp == 0) {  // (a CTA alone: every warp for itself)
      P = ta_join(lane < kTaWarps ? sh.wp[lane] : P, c2);
      if (Drawn) Q = ta_join(lane < kTaWarps ? sh.wq[lane] : Q, c2);
    }
    if (NC > 1) {
      const float4 xs = exchange(make_float4(P.m, P.s, Q.m, Q.s));
      P = ta_join({xs.x, xs.y}, c2);
      if (Drawn) Q = ta_join({xs.z, xs.w}, c2);
    }
    // one warp forms the rows' maxima and totals with the children
    // a token is gone once its first child was rejected, so what is left
    // after t rejections is a suffix sum over the first children from t on
    if (warp == 0) {
      float cm = P.m, cn = Q.m;
      for (int c = lane; c < n_child; c += 32) {
        cm = fmaxf(cm, sh.cl[c]);
        if (Drawn) cn = fmaxf(cn, sh.cg[c]);
      }
      const float mp = ta_max(cm), mq = Drawn ? ta_max(cn) : -INFINITY;
      // no logit above -inf, +inf, or a NaN: the row is no distribution, and the
      // walk ends here.  (The last token is then some token: of the weights that
      // are numbers the largest over its noise, token 0 where there is none.)
      const bool bad = sh.bad_child || !(mp > -INFINITY && mp < INFINITY) || P.s != P.s ||
                       (Drawn && g && (!(mq > -INFINITY && mq < INFINITY) || Q.s != Q.s));
      if (bad && rank == 0 && lane == 0) raise_status(d.status, ST_NUMERIC);
      if (lane == 0) {
        sh.bad = bad;
        sh.mp = mp;
        sh.mq = mq;
      }
      for (int c = lane; c < n_child; c += 32) {
        sh.cp[c] = sh.ctok[c] < 0 ? 0.f : ta_weight(sh.cl[c], mp, c2);
        if (Drawn) sh.cq[c] = sh.ctok[c] < 0 ? 0.f : ta_weight(sh.cg[c], mq, c2);
      }
      // (a suffix scan of the warp per 32 children, the last ones first)
      float zp = P.s > 0.f ? P.s * ta_weight(P.m, mp, c2) : 0.f, zq = Drawn && Q.s > 0.f ? Q.s * ta_weight(Q.m, mq, c2) : 0.f;
      if (lane == 0) sh.sufP[n_child] = zp;
      for (int c0 = (n_child - 1) & ~31; c0 >= 0; c0 -= 32) {
        const int c = c0 + lane;
        const bool on = c < n_child && !sh.cdup[c];
        float a = on ? sh.cp[c] : 0.f, b = Drawn && on ? sh.cq[c] : 0.f;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float a2 = __shfl_down_sync(0xffffffffu, a, o), b2 = Drawn ? __shfl_down_sync(0xffffffffu, b, o) : 0.f;
          if (lane + o < 32) {
            a += a2;
            b += b2;
          }
        }
        a += zp;
        b += zq;
        if (c < n_child) {
          sh.sufP[c] = a;
          if (Drawn) sh.invY[c] = b > 0.f ? 1.f / b : 0.f;
        }
        zp = __shfl_sync(0xffffffffu, a, 0);
        zq = __shfl_sync(0xffffffffu, b, 0);
      }
      if constexpr (Drawn) {
        const float f = zp > 0.f ? 1.f / zp : 0.f;
        for (int c = lane; c < n_child; c += 32) sh.cp[c] *= f;
      }
    }
    __syncthreads();
    const float mp = sh.mp, mq = sh.mq, Zp = sh.sufP[0];
    const float invP = Zp > 0.f ? 1.f / Zp : 0.f;
    float fp = 0.f, fq = 0.f;  // a row's weights -> p, q's weights
    if constexpr (Drawn) {
      // lw := p_0, gw := the draft row's weights
      fp = ml > -INFINITY ? ta_weight(ml, mp, c2) * invP : 0.f;
      fq = mg > -INFINITY ? ta_weight(mg, mq, c2) : 0.f;
#pragma unroll
      for (int j = 0; j < E; ++j) {
        lw[j] *= fp;
        gw[j] = g ? gw[j] * fq : 0.f;
      }
    }
    // p_t (and q's weights) of a later batch, from the logits (the target row's given in p)
    auto reload = [&](int b, int t, float (&p)[E], float (&q)[E]) __attribute__((always_inline)) {
      const uint32_t mine = find(b);
      clean(mine, p);
      if (Drawn && g) {
        load(g, b, q);
        clean(mine, q);
      }
#pragma unroll
      for (int j = 0; j < E; ++j) {
        p[j] = p[j] > -INFINITY ? ta_weight(p[j], mp, c2) : 0.f;
        if constexpr (Drawn) {
          p[j] *= invP;
          q[j] = g && q[j] > -INFINITY ? ta_weight(q[j], mq, c2) : 0.f;
        }
      }
      if constexpr (Drawn) {
        for (int e = 0; e < t; ++e) {
          const float z = sh.invZ[e], y = sh.invY[e];
          if (z > 0.f) {
#pragma unroll
            for (int j = 0; j < E; ++j) {
              p[j] = fmaxf(p[j] - q[j] * y, 0.f) * z;
            }
          }
        }
      }
    };

    // ---- the tests, in order
    int went = -1, t = 0;
    const int n_test = sh.bad ? 0 : n_child;
    for (; t < n_test; ++t) {
      bool ok;
      if constexpr (Drawn) {
        const float y = sh.invY[t];
        const float qx = sh.cdup[t] ? 0.f : sh.cq[t] * y;
        ok = sh.ctok[t] >= 0 && sh.cu[t] * qx < sh.cp[t];
        if (!ok) {
          // Z_t, with the step's own q: the slice, and the children once
          float z = 0.f, pc = 0.f;
#pragma unroll
          for (int j = 0; j < E; ++j) {
            z += fmaxf(lw[j] - gw[j] * y, 0.f);
          }
          for (int b = 1; v0 + b * BATCH < v1; ++b) {
            float p[E], q[E];
            load(l, b, p);
            reload(b, t, p, q);
#pragma unroll
            for (int j = 0; j < E; ++j) {
              z += fmaxf(p[j] - q[j] * y, 0.f);
            }
          }
          if (tid < n_child) {
            pc = fmaxf(sh.cp[tid] - sh.cq[tid] * y, 0.f);
            if (rank == 0 && !sh.cdup[tid]) z += pc;
          }
          z = warp_sum(z);
          if (lane == 0) sh.wb[warp] = z;
          __syncthreads();
          float zz = NC == 1 || warp == 0 ? warp_sum(lane < kTaWarps ? sh.wb[lane] : 0.f) : 0.f;
          if (NC > 1) {
            const float4 xz = exchange(make_float4(0.f, zz, 0.f, 0.f));
            zz = warp_sum(lane < NC ? xz.y : 0.f);
          }
          // nothing left: p stays (the caller's q covers all of p, up to rounding)
          const float iz = zz > 0.f ? 1.f / zz : 0.f;
          if (iz > 0.f) {
#pragma unroll
            for (int j = 0; j < E; ++j) {
              lw[j] = fmaxf(lw[j] - gw[j] * y, 0.f) * iz;
            }
          }
          if (tid < n_child) {
            if (iz > 0.f) sh.cp[tid] = pc * iz;
            if (sh.ctok[tid] == sh.ctok[t]) sh.cq[tid] = 0.f;
          }
          if (tid == 0) sh.invZ[t] = iz;
          __syncthreads();
        }
      } else {
        ok = !sh.cdup[t] && sh.cu[t] * sh.sufP[t] < sh.cp[t];
      }
      if (ok) {
        went = sh.child[t];
        break;
      }
    }
    if (went >= 0) {
      if (rank == 0 && tid == 0) {
        d.out_tokens[(size_t)s * N + k] = sh.tok[went];
        d.path[(size_t)s * N + k + 1] = went;
      }
      ++k;
      cur = went;
      __syncthreads();
      continue;
    }

    // ---- the last token: argmax p(v) / noise(v), lowest v on equal values
    // (best-of candidates: the children's tokens are all gone; drawn ones:
    // they keep what the subtractions left)
    float best = -INFINITY;
    int bi = INT_MAX;
    auto offer = [&](float p, float n, int v) __attribute__((always_inline)) {
      const float r = __fdividef(p, n);  // (2 units in the last place; 0 for n beyond 2^126)
      if (r > best || (r == best && v < bi)) {
        best = r;
        bi = v;
      }
    };
    auto draw = [&](int b, const float (&p)[E], const float (&n)[E]) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const int v = v0 + b * BATCH + j * kTaThreads + tid;
        if (v < v1) offer(p[j], n[j], v);
      }
    };
    if constexpr (!Drawn) {  // (weights against one maximum)
      const float f = ml > -INFINITY ? ta_weight(ml, mp, c2) : 0.f;
#pragma unroll
      for (int j = 0; j < E; ++j) {
        lw[j] *= f;
      }
    }
    {
      float n[E];
      load(noise, 0, n);
      draw(0, lw, n);
    }
    for (int b = 1; v0 + b * BATCH < v1; ++b) {
      float p[E], q[E], n[E];
      load(noise, b, n);
      load(l, b, p);
      reload(b, t, p, q);
      draw(b, p, n);
    }
    if (Drawn && rank == 0 && tid < n_child && sh.ctok[tid] >= 0)
      offer(sh.cp[tid], noise[sh.ctok[tid]], sh.ctok[tid]);
    ta_best_join(best, bi);
    if (lane == 0) {
      sh.wb[warp] = best;
      sh.wi[warp] = bi;
    }
    __syncthreads();
    if (warp == 0) {
      best = lane < kTaWarps ? sh.wb[lane] : -INFINITY;
      bi = lane < kTaWarps ? sh.wi[lane] : INT_MAX;
      ta_best_join(best, bi);
    }
    const float4 xb = exchange(make_float4(best, __int_as_float(bi), 0.f, 0.f));
    if (rank == 0 && warp == 0) {
      best = lane < NC ? xb.x : -INFINITY;
      bi = lane < NC ? __float_as_int(xb.y) : INT_MAX;
      ta_best_join(best, bi);
      if (lane == 0) {
        const int x = bi == INT_MAX ? 0 : bi;
        const int P0 = d.base_pos ? d.base_pos[s] : 0;
        d.out_tokens[(size_t)s * N + k] = x;
        d.accept_len[s] = k;
        if (d.next_anchor) d.next_anchor[s] = x;
        if (d.commit_base) d.commit_base[s] = P0;
        if (d.commit_count) d.commit_count[s] = k + 1;
        if (d.update_base) d.base_pos[s] = P0 + k + 1;
      }
    }
    for (int j = tid; rank == 0 && j < N; j += kTaThreads) {
      if (j > k) {
        d.out_tokens[(size_t)s * N + j] = -1;
        d.path[(size_t)s * N + j] = -1;
      }
    }
    break;
  }
  // (nothing of a peer's shared memory is touched after the last exchange's barrier)
}

// Temperature 0: the walk over the target's argmaxes, one warp per sequence.
__global__ void __launch_bounds__(32) tree_greedy_kernel(const __grid_constant__ TreeAcceptDesc d) {
  pdl_wait();
  pdl_launch_dependents();
  const int s = blockIdx.x, N = d.rows, lane = threadIdx.x;
  const size_t o = (size_t)s * N;
  int cur = 0, k = 0;
  int want = d.argmax[o];
  if (lane == 0) d.path[o] = 0;
  // rows in order: a child of the walk's node lies behind it, and once it is
  // taken its siblings' parent is no longer the walk's node
  for (int b = 0; b < N; b += 32) {
    const int i = b + lane;
    const int p = i < N && i > 0 ? (d.parent ? d.parent[o + i] : i - 1) : DFLASH_TREE_PAD;
    const int x = i < N ? d.tokens[o + i] : -1;
    const int am = i < N ? d.argmax[o + i] : -1;
    if (i > 0 && i < N && p >= 0 && (x < 0 || x >= d.V)) raise_status(d.status, ST_RANGE);
    int from = 0;
    for (;;) {
      const unsigned hit =
          __ballot_sync(0xffffffffu, lane >= from && i > cur && p == cur && x == want && x >= 0 && x < d.V);
      if (!hit) break;
      const int w = __ffs(hit) - 1;
      if (lane == 0) {
        d.out_tokens[o + k] = want;
        d.path[o + k + 1] = b + w;
      }
      ++k;
      cur = b + w;
      want = __shfl_sync(0xffffffffu, am, w);
      from = w + 1;
    }
  }
  for (int j = k + 1 + lane; j < N; j += 32) {
    d.out_tokens[o + j] = -1;
    d.path[o + j] = -1;
  }
  if (lane == 0) {
    const int P0 = d.base_pos ? d.base_pos[s] : 0;
    d.out_tokens[o + k] = want;
    d.accept_len[s] = k;
    if (d.next_anchor) d.next_anchor[s] = want;
    if (d.commit_base) d.commit_base[s] = P0;
    if (d.commit_count) d.commit_count[s] = k + 1;
    if (d.update_base) d.base_pos[s] = P0 + k + 1;
  }
}

static cudaLaunchConfig_t ta_config(int n_seqs, int nc, cudaStream_t st, cudaLaunchAttribute (&at)[2]) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(n_seqs * nc);
  cfg.blockDim = dim3(kTaThreads);
  cfg.stream = st;
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = nc;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cfg;
}

// Does the device run clusters of 16 of this kernel?  (Asked once per device.)
static bool ta_wide(void (*kernel)(TreeAcceptDesc)) {
  static std::atomic<int> known[64];  // 0: not asked, 1: no, 2: yes (the kernels' sizes are alike)
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return false;
  int k = known[dev].load(std::memory_order_relaxed);
  if (!k) {
    cudaLaunchAttribute at[2];
    const cudaLaunchConfig_t cfg = ta_config(1, kTaMaxCluster, nullptr, at);
    int n = 0;
    k = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0 ? 2 : 1;
    if (k == 1) cudaGetLastError();
    known[dev].store(k, std::memory_order_relaxed);
  }
  return k == 2;
}

cudaError_t launch_tree_accept(const TreeAcceptDesc& d, int num_sms, cudaStream_t st) {
  if (d.invT == 0.f) return launch_pdl(tree_greedy_kernel, dim3(d.n_seqs), dim3(32), 0, st, d);
  // As many CTAs per sequence as run at once, a CTA per SM, each with at least
  // 1024 vocabulary entries.  Clusters of 16 are beyond the portable size and
  // need one GPC's SMs, so only few of them run at once.
  int nc = 1;
  while (nc < 8 && d.n_seqs * nc * 2 <= num_sms && d.V >= nc * 2 * 1024) nc *= 2;
  auto pick = [&]() {
    const bool brief = d.V <= nc * (kTaThreads * kTaShortE - 32);  // (slices are rounded up to 32)
    return d.draft ? (brief ? tree_accept_kernel<true, kTaShortE> : tree_accept_kernel<true, kTaE>)
                   : (brief ? tree_accept_kernel<false, kTaShortE> : tree_accept_kernel<false, kTaE>);
  };
  auto* kernel = pick();
  if (nc == 8 && d.n_seqs * 32 <= num_sms && d.V >= 16 * 1024) {
    nc = kTaMaxCluster;
    kernel = pick();
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess || !ta_wide(kernel)) {
      nc = 8;
      kernel = pick();
    }
  }
  cudaLaunchAttribute at[2];
  const cudaLaunchConfig_t cfg = ta_config(d.n_seqs, nc, st, at);
  trace_kernel();
  return cudaLaunchKernelEx(&cfg, kernel, d);
}

// One CTA per sequence, one thread per row.
__global__ void __launch_bounds__(DFLASH_MAX_TREE) tree_build_kernel(const __grid_constant__ TreeBuildDesc d) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ int par[DFLASH_MAX_TREE];
  const int s = blockIdx.x, i = threadIdx.x;
  if (i < d.rows) par[i] = d.parent[i];
  __syncthreads();
  if (i >= d.rows) return;
  const int anchor = d.anchor[s], P = d.base_pos[s];
  int depth = 0, j = i;
  bool ok = true;
  for (;;) {
    const int p = par[j];
    if (p == -1) break;
    if (p < 0 || p >= j) {
      if (p != DFLASH_TREE_PAD) raise_status(d.status, ST_RANGE);
      ok = false;
      break;
    }
    j = p;
    ++depth;
  }
  int tok = anchor;
  if (ok && depth > 0) {
    const int r = d.rank[i];
    if (depth > d.levels || r < 0 || r >= d.topk) {
      raise_status(d.status, ST_RANGE);
      ok = false;
    } else {
      tok = d.cand[((size_t)s * d.levels + depth - 1) * d.topk + r];
    }
  }
  const size_t o = (size_t)s * d.rows + i;
  d.parent_out[o] = ok ? par[i] : DFLASH_TREE_PAD;
  d.tokens_out[o] = tok;
  d.pos_out[o] = P + (ok ? depth : 0);
}

cudaError_t launch_tree_build(const TreeBuildDesc& d, cudaStream_t st) {
  return launch_pdl(tree_build_kernel, dim3(d.n_seqs), dim3(DFLASH_MAX_TREE), 0, st, d);
}

}  // namespace dfl
