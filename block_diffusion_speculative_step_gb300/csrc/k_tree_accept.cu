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
// vocabulary; sums cross the cluster through distributed shared memory and
// every CTA forms them in rank order, so all CTAs take the same decisions
// and a call is deterministic.  Remaining masses are sums over what remains
// (children's weights are kept out of the row sums and added one by one):
// 1 - p(x) would lose all its digits when p(x) is close to 1.
#include <cooperative_groups.h>
#include <limits.h>

#include "common.cuh"
#include "internal.h"
#include "launch.cuh"

namespace dfl {

namespace cg = cooperative_groups;

constexpr int kTaThreads = 512;
constexpr int kTaWarps = kTaThreads / 32;
constexpr int kTaMaxNC = 16;

// Weight of logit l against the row's maximum m (l == m also when both are
// infinite: the weight is then 1 and the caller reports the row).
__device__ __forceinline__ float ta_weight(float l, float m, float invT) {
  return l == m ? 1.f : expf((l - m) * invT);
}

struct TaSum {  // running maximum and sum of weights against it
  float m, s;
};
__device__ __forceinline__ TaSum ta_merge(TaSum a, TaSum b, float invT) {
  TaSum r;
  r.m = fmaxf(a.m, b.m);
  r.s = (a.s > 0.f ? a.s * ta_weight(a.m, r.m, invT) : 0.f) + (b.s > 0.f ? b.s * ta_weight(b.m, r.m, invT) : 0.f);
  return r;
}

// Calls f(v, x) for the elements of row[v0, v1), vectorised over the 16-byte
// aligned middle; the assignment of elements to threads is fixed.
template <typename F>
__device__ __forceinline__ void ta_for(const float* __restrict__ row, int v0, int v1, F f) {
  const int mis = (int)((reinterpret_cast<uintptr_t>(row + v0) >> 2) & 3);
  const int a = min(v1, v0 + ((4 - mis) & 3));
  const int b = a + ((v1 - a) & ~3);
  if (v0 + (int)threadIdx.x < a) f(v0 + (int)threadIdx.x, row[v0 + threadIdx.x]);
  for (int v = a + 4 * (int)threadIdx.x; v < b; v += 4 * kTaThreads) {
    const float4 x = *reinterpret_cast<const float4*>(row + v);
    f(v, x.x);
    f(v + 1, x.y);
    f(v + 2, x.z);
    f(v + 3, x.w);
  }
  if (b + (int)threadIdx.x < v1) f(b + (int)threadIdx.x, row[b + threadIdx.x]);
}

struct TaShared {
  int parent[DFLASH_MAX_TREE];
  int tok[DFLASH_MAX_TREE];
  float u[DFLASH_MAX_TREE];
  int n_child;
  int child[DFLASH_MAX_TREE];   // children of the current node, in row order
  int ctok[DFLASH_MAX_TREE];
  float cu[DFLASH_MAX_TREE];
  float cl[DFLASH_MAX_TREE];    // the children's target / draft logits
  float cg[DFLASH_MAX_TREE];
  int cdup[DFLASH_MAX_TREE];    // an earlier sibling has the same token, or the token is out of range
  double sufP[DFLASH_MAX_TREE + 1];  // mass of the target / draft row without the tokens of children [0, t)
  double sufQ[DFLASH_MAX_TREE + 1];
  unsigned long long bloom;     // bit (token / 4) % 64 of every child's token
  float invZ[DFLASH_MAX_TREE];  // 1 / Z_t, 0: nothing left, p stays
  float invY[DFLASH_MAX_TREE];  // 1 / (remaining mass of q before step t), in q's weights
  TaSum wp[kTaWarps], wq[kTaWarps];
  float wb[kTaWarps];
  int wi[kTaWarps];
  TaSum xp[2], xq[2];           // this CTA's partials, by parity (read by the cluster)
  float xb[2];
  int xi[2];
};

template <bool Drawn>
__global__ void __launch_bounds__(kTaThreads) tree_accept_kernel(const __grid_constant__ TreeAcceptDesc d) {
  pdl_wait();
  pdl_launch_dependents();
  __shared__ TaShared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int NC = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int s = blockIdx.x / NC;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int V = d.V, N = d.rows;
  const int per = (V + NC - 1) / NC;
  const int v0 = min(V, rank * per), v1 = min(V, v0 + per);
  const float invT = d.invT;
  const float* target = d.target + (size_t)s * N * V;
  const float* draft = Drawn ? d.draft + (size_t)s * d.levels * V : nullptr;
  int par = 0;  // exchange parity

  for (int i = tid; i < N; i += kTaThreads) {
    sh.parent[i] = d.parent ? d.parent[(size_t)s * N + i] : i - 1;
    sh.tok[i] = d.tokens[(size_t)s * N + i];
    sh.u[i] = d.u[(size_t)s * N + i];
  }
  __syncthreads();

  int cur = 0, k = 0;
  if (rank == 0 && tid == 0) d.path[(size_t)s * N] = 0;
  for (;;) {
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
      if (lane == 0) {
        sh.n_child = n;
        sh.bloom = 0ull;
      }
    }
    __syncthreads();
    int n_child = sh.n_child;
    const bool deep = Drawn && k >= d.levels;  // no draft row for these children
    if (deep) {
      if (n_child > 0 && rank == 0 && tid == 0) raise_status(d.status, ST_RANGE);
      n_child = 0;
    }
    const float* l = target + (size_t)cur * V;
    const float* g = Drawn && n_child > 0 ? draft + (size_t)k * V : nullptr;
    for (int c = tid; c < n_child; c += kTaThreads) {
      const int i = sh.child[c];
      int x = sh.tok[i];
      if (x < 0 || x >= V) {
        if (rank == 0) raise_status(d.status, ST_RANGE);
        x = -1;  // never accepted, nothing to remove
      }
      sh.ctok[c] = x;
      sh.cu[c] = sh.u[i];
      sh.cl[c] = x >= 0 ? l[x] : -INFINITY;
      if (Drawn) sh.cg[c] = x >= 0 ? g[x] : -INFINITY;
      int dup = 0;
      for (int e = 0; e < c; ++e) dup |= sh.tok[sh.child[e]] == x;
      sh.cdup[c] = dup || x < 0;
      if (x >= 0) atomicOr(&sh.bloom, 1ull << ((x >> 2) & 63));
    }
    __syncthreads();

    // ---- maxima and sums over the slice, the children's tokens left out of the sums
    const unsigned long long bloom = n_child > 0 ? sh.bloom : 0ull;
    auto is_child = [&](int v) {
      if (!((bloom >> ((v >> 2) & 63)) & 1ull)) return false;
      for (int c = 0; c < n_child; ++c)
        if (sh.ctok[c] == v) return true;
      return false;
    };
    bool nan = false;
    auto row_sum = [&](const float* row) {
      TaSum a = {-INFINITY, 0.f};
      ta_for(row, v0, v1, [&](int v, float x) {
        if (!(x < INFINITY)) nan = true;  // NaN or +inf
        if (is_child(v) || x != x) return;
        if (x > a.m) {
          a.s = a.s > 0.f ? a.s * ta_weight(a.m, x, invT) + 1.f : 1.f;
          a.m = x;
        } else if (x > -INFINITY) {
          a.s += expf((x - a.m) * invT);
        }
      });
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        TaSum b;
        b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
        b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
        a = ta_merge(a, b, invT);
      }
      return a;
    };
    TaSum ap = row_sum(l), aq = {-INFINITY, 0.f};
    if (Drawn && g) aq = row_sum(g);
    if (nan) raise_status(d.status, ST_NUMERIC);
    if (lane == 0) {
      sh.wp[warp] = ap;
      sh.wq[warp] = aq;
    }
    __syncthreads();
    if (tid == 0) {
      TaSum a = sh.wp[0], b = sh.wq[0];
      for (int w = 1; w < kTaWarps; ++w) {
        a = ta_merge(a, sh.wp[w], invT);
        b = ta_merge(b, sh.wq[w], invT);
      }
      sh.xp[par] = a;
      sh.xq[par] = b;
    }
    cl.sync();
    TaSum P = {-INFINITY, 0.f}, Q = {-INFINITY, 0.f};
    for (int r = 0; r < NC; ++r) {
      const TaShared* o = cl.map_shared_rank(&sh, r);
      P = ta_merge(P, o->xp[par], invT);
      if (Drawn) Q = ta_merge(Q, o->xq[par], invT);
    }
    par ^= 1;
    // every thread forms the rows' maxima and totals with the children, in order
    float mp = P.m, mq = Q.m;
    for (int c = 0; c < n_child; ++c) {
      const float a = sh.cl[c];
      if (a == a) mp = fmaxf(mp, a);
      if (Drawn && sh.cg[c] == sh.cg[c]) mq = fmaxf(mq, sh.cg[c]);
    }
    if (mp == -INFINITY && rank == 0 && tid == 0) raise_status(d.status, ST_NUMERIC);
    const double base_p = P.s > 0.f ? (double)P.s * ta_weight(P.m, mp, invT) : 0.0;
    const double base_q = Drawn && Q.s > 0.f ? (double)Q.s * ta_weight(Q.m, mq, invT) : 0.0;
    auto wl = [&](int c) { return sh.cl[c] == sh.cl[c] ? ta_weight(sh.cl[c], mp, invT) : 0.f; };
    auto wg = [&](int c) { return sh.cg[c] == sh.cg[c] ? ta_weight(sh.cg[c], mq, invT) : 0.f; };
    // a token is gone once its first child was rejected, so what is left
    // after t rejections is a suffix sum over the first children from t on
    if (tid == 0) {
      double z = base_p;
      sh.sufP[n_child] = z;
      for (int c = n_child - 1; c >= 0; --c) sh.sufP[c] = z += sh.cdup[c] ? 0.0 : (double)wl(c);
    }
    if (Drawn && tid == 32) {
      double z = base_q;
      sh.sufQ[n_child] = z;
      for (int c = n_child - 1; c >= 0; --c) {
        z += sh.cdup[c] ? 0.0 : (double)wg(c);
        sh.sufQ[c] = z;
        sh.invY[c] = z > 0.0 ? (float)(1.0 / z) : 0.f;
      }
    }
    __syncthreads();
    const double Zp = sh.sufP[0];
    const float invP = Zp > 0.0 ? (float)(1.0 / Zp) : 0.f;

    // p_t(v) of a token after t rejections (drawn candidates), from its logits
    auto p_after = [&](float lx, float gx, int v, int t) {
      float p = lx == lx ? ta_weight(lx, mp, invT) * invP : 0.f;
      float q = gx == gx ? ta_weight(gx, mq, invT) : 0.f;
      for (int e = 0; e < t; ++e) {
        if (sh.invZ[e] > 0.f) p = fmaxf(p - q * sh.invY[e], 0.f) * sh.invZ[e];
        if (sh.ctok[e] == v) q = 0.f;
      }
      return p;
    };

    // ---- the tests, in order
    int went = -1, t = 0;
    for (; t < n_child; ++t) {
      const int x = sh.ctok[t];
      bool ok;
      if constexpr (Drawn) {
        const float px = p_after(sh.cl[t], sh.cg[t], x, t);
        const float qx = sh.cdup[t] ? 0.f : wg(t) * sh.invY[t];
        ok = x >= 0 && sh.cu[t] * qx < px;
        if (!ok) {
          // Z_t over the slice, with the step's own q
          float z = 0.f;
          ta_for(l, v0, v1, [&](int v, float lx) {
            const float gx = g[v];
            const float p = p_after(lx, gx, v, t);
            float q = gx == gx ? ta_weight(gx, mq, invT) * sh.invY[t] : 0.f;
            for (int e = 0; e < t; ++e)
              if (sh.ctok[e] == v) q = 0.f;
            z += fmaxf(p - q, 0.f);
          });
          z = warp_sum(z);
          if (lane == 0) sh.wb[warp] = z;
          __syncthreads();
          if (tid == 0) {
            float a = 0.f;
            for (int w = 0; w < kTaWarps; ++w) a += sh.wb[w];
            sh.xb[par] = a;
          }
          cl.sync();
          double zz = 0.0;
          for (int r = 0; r < NC; ++r) zz += (double)cl.map_shared_rank(&sh, r)->xb[par];
          par ^= 1;
          __syncthreads();
          if (tid == 0) sh.invZ[t] = zz > 0.0 ? (float)(1.0 / zz) : 0.f;
          __syncthreads();
        }
      } else {
        ok = !sh.cdup[t] && (double)sh.cu[t] * sh.sufP[t] < (double)wl(t);
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
    float best = -INFINITY;
    int bi = INT_MAX;
    const float* noise = d.noise + (size_t)s * V;
    ta_for(l, v0, v1, [&](int v, float lx) {
      float p;
      if (Drawn) {
        p = p_after(lx, g ? g[v] : -INFINITY, v, t);
      } else {
        p = lx == lx ? ta_weight(lx, mp, invT) : 0.f;
        for (int e = 0; e < t; ++e)
          if (sh.ctok[e] == v) p = 0.f;
      }
      const float r = p / noise[v];
      if (r > best || (r == best && v < bi)) {
        best = r;
        bi = v;
      }
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float ob = __shfl_xor_sync(0xffffffffu, best, o);
      const int oi = __shfl_xor_sync(0xffffffffu, bi, o);
      if (ob > best || (ob == best && oi < bi)) {
        best = ob;
        bi = oi;
      }
    }
    if (lane == 0) {
      sh.wb[warp] = best;
      sh.wi[warp] = bi;
    }
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kTaWarps; ++w)
        if (sh.wb[w] > sh.wb[0] || (sh.wb[w] == sh.wb[0] && sh.wi[w] < sh.wi[0])) {
          sh.wb[0] = sh.wb[w];
          sh.wi[0] = sh.wi[w];
        }
      sh.xb[par] = sh.wb[0];
      sh.xi[par] = sh.wi[0];
    }
    cl.sync();
    if (rank == 0 && tid == 0) {
      float b = -INFINITY;
      int x = INT_MAX;
      for (int r = 0; r < NC; ++r) {
        const TaShared* o = cl.map_shared_rank(&sh, r);
        if (o->xb[par] > b || (o->xb[par] == b && o->xi[par] < x)) {
          b = o->xb[par];
          x = o->xi[par];
        }
      }
      if (x == INT_MAX) x = 0;
      const int P0 = d.base_pos ? d.base_pos[s] : 0;
      d.out_tokens[(size_t)s * N + k] = x;
      d.accept_len[s] = k;
      if (d.next_anchor) d.next_anchor[s] = x;
      if (d.commit_base) d.commit_base[s] = P0;
      if (d.commit_count) d.commit_count[s] = k + 1;
      if (d.update_base) d.base_pos[s] = P0 + k + 1;
    }
    for (int j = tid; rank == 0 && j < N; j += kTaThreads) {
      if (j > k) {
        d.out_tokens[(size_t)s * N + j] = -1;
        d.path[(size_t)s * N + j] = -1;
      }
    }
    break;
  }
  cl.sync();  // peers read this CTA's shared memory until here
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

cudaError_t launch_tree_accept(const TreeAcceptDesc& d, int num_sms, cudaStream_t st) {
  if (d.invT == 0.f) return launch_pdl(tree_greedy_kernel, dim3(d.n_seqs), dim3(32), 0, st, d);
  // As many CTAs per sequence as fit at once, at most 8 (the portable cluster
  // size), each with at least 1024 vocabulary entries.
  int nc = 1;
  while (nc < 8 && d.n_seqs * nc * 2 <= num_sms && d.V >= nc * 2 * 1024) nc *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(d.n_seqs * nc);
  cfg.blockDim = dim3(kTaThreads);
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
  return d.draft ? cudaLaunchKernelEx(&cfg, tree_accept_kernel<true>, d)
                 : cudaLaunchKernelEx(&cfg, tree_accept_kernel<false>, d);
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
