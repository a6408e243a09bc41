// k_tree_attn.cu -- attention of a drafted tree's rows over the cached context
// and over their own ancestors (dflash_tree_attention, DFLASH_ATTN_TREE).
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "tree_attn.cuh"

namespace dfl {

// ------------------------------------------------------ CUDA-core path
//
// One CTA per (split, KV head x query tile, sequence): 32 query vectors
// against 64 to 256 key slots (the last split: the tree's rows), 64 keys at a time.
// S = Q K^T and O += P V are register-blocked 4 x 4 and 4 x (d / 16) tiles
// per thread, the online softmax's maximum and sum are shared by the 16
// threads of a row.  Splits sit at fixed slot offsets, so a row's bits depend
// on its own context only.  Bound by fp32 FMAs: 4 d flops per query vector
// and key at 128 FMA lanes per SM.
constexpr int kTsThreads = 128;
constexpr int kTsQT = 32;     // query vectors per CTA
constexpr int kTsKT = 64;     // keys per step

struct TsGeom {
  int grp, nqv, n_qt, split, n_split;  // key slots per split; context splits + the tree's
};
__host__ __device__ inline TsGeom ts_geom(const TreeAttnDesc& a) {
  TsGeom g;
  g.grp = a.nq / a.nkv;
  g.nqv = a.rows * g.grp;
  g.n_qt = (g.nqv + kTsQT - 1) / kTsQT;
  // Short contexts want many CTAs, long ones few partials.  By the bound of the
  // contexts, not by the batch: a row's bits do not depend on what runs beside
  // it.  64 / 256 slots measured: 3 sequences up to 131 slots 11.1 / 13.4 us, 2 of
  // 1000 17.3 / 28.0 us, 4 of 8190 110 / 65 us (128: 13.4, 19.2, 79.5 us).
  g.split = a.max_pos <= 1024 ? 64 : a.max_pos <= 4096 ? 128 : 256;
  g.n_split = (a.max_pos + g.split - 1) / g.split + 1;
  return g;
}

template <typename T, bool Q8, int D>
__global__ void __launch_bounds__(kTsThreads) tree_simt_kernel(const __grid_constant__ TreeAttnDesc a) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int LD = D + 4;
  extern __shared__ float ts_sm[];
  float* Qs = ts_sm;              // [32][LD]
  float* Ks = Qs + kTsQT * LD;    // [64][LD]
  float* Vs = Ks + kTsKT * LD;    // [64][LD]
  float* Ps = Vs + kTsKT * LD;    // [32][64 + 4]
  constexpr int PLD = kTsKT + 4;
  __shared__ int par[DFLASH_MAX_TREE];
  __shared__ uint32_t mask[kTsQT][4];
  __shared__ int node_ok[kTsQT];

  const TsGeom gm = ts_geom(a);
  const int sp = blockIdx.x, g = blockIdx.y / gm.n_qt, qt = blockIdx.y % gm.n_qt, s = blockIdx.z;
  const bool tree = sp == gm.n_split - 1;
  const int base = __ldg(a.base_pos + s), n_ctx = min(max(base, 0), a.max_pos);
  const int j0 = sp * gm.split;
  if (!tree && j0 >= n_ctx) return;  // the merge knows which splits hold keys
  const int n_keys = tree ? a.rows : min(gm.split, n_ctx - j0);
  const int tid = threadIdx.x;
  const int qv0 = qt * kTsQT, nq_tile = min(kTsQT, gm.nqv - qv0);
  const int QD = a.nq * D;

  if (tree) {
    if (base != n_ctx && tid == 0) raise_status(a.status, ST_RANGE);
    if (a.parent)
      for (int i = tid; i < a.rows; i += kTsThreads) par[i] = a.parent[(size_t)s * a.rows + i];
    __syncthreads();
    if (tid < kTsQT) {
      uint32_t w[4] = {0u, 0u, 0u, 0u};
      bool ok = false, bad = false;
      if (tid < nq_tile) {
        const int row = (qv0 + tid) / gm.grp;
        ok = tree_row_mask(a.parent ? par : nullptr, row, w, &bad);
        if (ok && a.pos) bad = (uint32_t)__ldg(a.pos + (size_t)s * a.rows + row) >= (uint32_t)a.pos_end;
      }
      if (bad) raise_status(a.status, ST_RANGE);
      node_ok[tid] = ok;
      for (int i = 0; i < 4; ++i) mask[tid][i] = w[i];
    }
  }
  for (int t = tid; t < kTsQT * (D / 8); t += kTsThreads) {
    const int qi = t / (D / 8), e = (t % (D / 8)) * 8;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (qi < nq_tile) {
      const int qv = qv0 + qi, row = qv / gm.grp, head = g * gm.grp + qv % gm.grp;
      load8(reinterpret_cast<const T*>(a.q) + ((size_t)s * a.rows + row) * QD + (size_t)head * D + e, v);
    }
    for (int i = 0; i < 8; ++i) Qs[qi * LD + e + i] = v[i] * a.scale;
  }

  const int ty = tid >> 4, tx = tid & 15;  // 4 query vectors ty*4.., keys tx + 16 j, columns tx*4 + 64 c
  constexpr int NC = D / 64;               // float4 columns per thread
  float O[4][4 * NC];
  float m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < 4 * NC; ++c) O[i][c] = 0.f;
  }
  const KvMap km{a.pages, a.cap, a.ps, a.max_pages, a.pool, a.nkv};
  for (int k0 = 0; k0 < n_keys; k0 += kTsKT) {
    const int nk = min(kTsKT, n_keys - k0);
    __syncthreads();
    // ---- this step's keys and values (rows past the last key zero)
    size_t row0 = 0;
    if (!tree) {  // 64-slot steps never span two pages
      bool bad = false;
      row0 = (size_t)km.row0(s, j0 + k0, &bad) + (size_t)g * km.head_rows();
      if (bad && tid == 0) raise_status(a.status, ST_RANGE);  // reads page 0 instead
    }
    for (int t = tid; t < kTsKT * (D / 8); t += kTsThreads) {
      const int j = t / (D / 8), e = (t % (D / 8)) * 8;
      float kv[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, vv[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (j < nk) {
        if (tree) {
          const size_t o = (((size_t)s * a.rows + k0 + j) * a.nkv + g) * D + e;
          load8(reinterpret_cast<const T*>(a.kb) + o, kv);
          load8(reinterpret_cast<const T*>(a.vb) + o, vv);
        } else if constexpr (Q8) {
          load8_e4m3(a.kc, a.k_exp, row0 + j, D, e, kv);
          load8_e4m3(a.vc, a.v_exp, row0 + j, D, e, vv);
        } else {
          load8(reinterpret_cast<const T*>(a.kc) + (row0 + j) * D + e, kv);
          load8(reinterpret_cast<const T*>(a.vc) + (row0 + j) * D + e, vv);
        }
      }
      *reinterpret_cast<float4*>(Ks + j * LD + e) = make_float4(kv[0], kv[1], kv[2], kv[3]);
      *reinterpret_cast<float4*>(Ks + j * LD + e + 4) = make_float4(kv[4], kv[5], kv[6], kv[7]);
      *reinterpret_cast<float4*>(Vs + j * LD + e) = make_float4(vv[0], vv[1], vv[2], vv[3]);
      *reinterpret_cast<float4*>(Vs + j * LD + e + 4) = make_float4(vv[4], vv[5], vv[6], vv[7]);
    }
    __syncthreads();
    // ---- scores of 4 query vectors x 4 keys
    float S[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) S[i][j] = 0.f;
#pragma unroll 4
    for (int e = 0; e < D; e += 4) {
      float4 q[4], k[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = *reinterpret_cast<const float4*>(Qs + (ty * 4 + i) * LD + e);
#pragma unroll
      for (int j = 0; j < 4; ++j) k[j] = *reinterpret_cast<const float4*>(Ks + (tx + 16 * j) * LD + e);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          S[i][j] = fmaf(q[i].x, k[j].x, S[i][j]);
          S[i][j] = fmaf(q[i].y, k[j].y, S[i][j]);
          S[i][j] = fmaf(q[i].z, k[j].z, S[i][j]);
          S[i][j] = fmaf(q[i].w, k[j].w, S[i][j]);
        }
    }
    // ---- online softmax; hidden keys carry P = -1 (skipped below, so that a
    // NaN or infinity in a row that is not visible cannot reach the output)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mx = m[i];
      bool vis[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = k0 + tx + 16 * j;
        vis[j] = tx + 16 * j < nk && (!tree || ((mask[ty * 4 + i][key >> 5] >> (key & 31)) & 1u));
        if (vis[j]) mx = fmaxf(mx, S[i][j]);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float alpha = m[i] == mx ? 1.f : exp2f(m[i] - mx);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float p = -1.f;
        if (vis[j]) {
          p = S[i][j] == mx ? 1.f : exp2f(S[i][j] - mx);
          sum += p;
        }
        Ps[(ty * 4 + i) * PLD + tx + 16 * j] = p;
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      l[i] = fmaf(l[i], alpha, sum);
      m[i] = mx;
#pragma unroll
      for (int c = 0; c < 4 * NC; ++c) O[i][c] *= alpha;
    }
    __syncwarp();  // a row's P is written and read by the same half-warp
    // ---- O += P V
    for (int j = 0; j < nk; ++j) {
      float p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = Ps[(ty * 4 + i) * PLD + j];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float4 v = *reinterpret_cast<const float4*>(Vs + j * LD + 64 * c + tx * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!(p[i] < 0.f)) {
            O[i][4 * c] = fmaf(p[i], v.x, O[i][4 * c]);
            O[i][4 * c + 1] = fmaf(p[i], v.y, O[i][4 * c + 1]);
            O[i][4 * c + 2] = fmaf(p[i], v.z, O[i][4 * c + 2]);
            O[i][4 * c + 3] = fmaf(p[i], v.w, O[i][4 * c + 3]);
          }
      }
    }
  }
  // ---- the split's partial: [row][D] outputs, then maxima and sums (l < 0: a padding row)
  const size_t slot = (((size_t)s * a.nkv + g) * gm.n_qt + qt) * gm.n_split + sp;
  float* po = static_cast<float*>(a.work) + slot * (size_t)(kTsQT * (D + 2));
  float* pm = po + kTsQT * D;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int qi = ty * 4 + i;
    if (qi >= nq_tile) continue;
#pragma unroll
    for (int c = 0; c < NC; ++c)
      *reinterpret_cast<float4*>(po + qi * D + 64 * c + tx * 4) =
          make_float4(O[i][4 * c], O[i][4 * c + 1], O[i][4 * c + 2], O[i][4 * c + 3]);
    if (tx == 0) {
      pm[qi] = m[i];
      pm[kTsQT + qi] = tree && !node_ok[qi] ? -1.f : l[i];
    }
  }
}

// One warp per query vector: the partials of its splits in order.
template <typename T, int D>
__global__ void __launch_bounds__(256) tree_simt_merge_kernel(const __grid_constant__ TreeAttnDesc a) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int E = D / 32;
  const TsGeom gm = ts_geom(a);
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (w >= (long long)a.n_seqs * a.nkv * gm.nqv) return;
  const int qv = (int)(w % gm.nqv), g = (int)(w / gm.nqv % a.nkv), s = (int)(w / gm.nqv / a.nkv);
  const int qt = qv / kTsQT, qi = qv % kTsQT;
  const int n_ctx = min(max(__ldg(a.base_pos + s), 0), a.max_pos);
  const int n_sp = (n_ctx + gm.split - 1) / gm.split;  // context splits that hold keys
  const size_t slot0 = (((size_t)s * a.nkv + g) * gm.n_qt + qt) * gm.n_split;
  const float* base = static_cast<const float*>(a.work);
  constexpr size_t PS = kTsQT * (D + 2);
  auto part = [&](int i) { return base + (slot0 + (i < n_sp ? i : gm.n_split - 1)) * PS; };
  const bool pad = part(n_sp)[kTsQT * D + kTsQT + qi] < 0.f;
  if (pad && !a.zero_pad) return;  // left as it was
  float M = -INFINITY;
  for (int i = 0; i <= n_sp; ++i) M = fmaxf(M, part(i)[kTsQT * D + qi]);
  float L = 0.f, O[E];
#pragma unroll
  for (int e = 0; e < E; ++e) O[e] = 0.f;
  for (int i = 0; i <= n_sp; ++i) {
    const float* p = part(i);
    const float mi = p[kTsQT * D + qi];
    const float wi = mi == M ? 1.f : exp2f(mi - M);
    L = fmaf(p[kTsQT * D + kTsQT + qi], wi, L);
#pragma unroll
    for (int e = 0; e < E; ++e) O[e] = fmaf(p[qi * D + lane * E + e], wi, O[e]);
  }
  const int row = qv / gm.grp, head = g * gm.grp + qv % gm.grp;
  T* o = reinterpret_cast<T*>(a.out) + ((size_t)s * a.rows + row) * a.nq * D + (size_t)head * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = from_f<T>(pad ? 0.f : O[e] / L);
}

static size_t ts_workspace(const TreeAttnDesc& a) {
  const TsGeom g = ts_geom(a);
  return (size_t)a.n_seqs * a.nkv * g.n_qt * g.n_split * (kTsQT * (a.d + 2)) * sizeof(float);
}

template <typename T, bool Q8, int D>
static cudaError_t ts_launch(const TreeAttnDesc& a, cudaStream_t st) {
  constexpr int LD = D + 4;
  constexpr size_t smem = (size_t)((kTsQT + 2 * kTsKT) * LD + kTsQT * (kTsKT + 4)) * sizeof(float);
  cudaError_t e = cudaFuncSetAttribute(tree_simt_kernel<T, Q8, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const TsGeom g = ts_geom(a);
  e = launch_pdl(tree_simt_kernel<T, Q8, D>, dim3(g.n_split, a.nkv * g.n_qt, a.n_seqs), dim3(kTsThreads), smem, st, a);
  if (e != cudaSuccess) return e;
  const long long warps = (long long)a.n_seqs * a.nkv * g.nqv;
  return launch_pdl(tree_simt_merge_kernel<T, D>, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0, st, a);
}

static cudaError_t ts_dispatch(const TreeAttnDesc& a, cudaStream_t st) {
  const bool q8 = a.k_exp != nullptr;
  if (a.d == 128) return q8 ? ts_launch<float, true, 128>(a, st) : ts_launch<float, false, 128>(a, st);
  return q8 ? ts_launch<float, true, 64>(a, st) : ts_launch<float, false, 64>(a, st);
}

size_t tree_attn_workspace(const TreeAttnDesc& a, int num_sms) {
  return a.dtype == DFLASH_BF16 ? tree_tc_workspace(a, num_sms) : ts_workspace(a);
}

cudaError_t launch_tree_attention(const TreeAttnDesc& a, int num_sms, cudaStream_t st) {
  return a.dtype == DFLASH_BF16 ? launch_tree_tc(a, num_sms, st) : ts_dispatch(a, st);
}

}  // namespace dfl
