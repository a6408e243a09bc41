// k_prompt_attn.cu -- causal attention of packed prompts in fp32, and the choice
// between it and the tensor-core kernel (k_prompt_attn_tc.cu, bf16).
//
// A CTA has a tile of 64 query vectors of one (sequence, KV head), the group's
// query heads side by side (vector = token * group + head), and walks the keys
// that the tile sees in chunks of 64: cached slots, then the sequence's own
// rows up to the tile's last token.  Scores and outputs are register tiles
// (4 x 4 and 4 x d/16 per thread), the softmax runs along with a running
// maximum and sum.  Full precision has no tensor-core form, so the fp32 units
// bound it.  Where few tiles would leave SMs idle, the chunks of a tile are cut
// into `split` parts of equal number that a second kernel joins.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "prompt_attn.cuh"

namespace dfl {

namespace {

constexpr int kPsQ = 64;        // query vectors of a tile
constexpr int kPsK = 64;        // keys of a chunk
constexpr int kPsThreads = 256;

template <int D>
struct PsCfg {
  static constexpr int QP = kPsQ + 4;  // pitches, in floats (transposed tiles: rows of 64 vectors)
  static constexpr int VP = D + 4;
  static constexpr int Q_OFF = 0;                // [D][QP]
  static constexpr int K_OFF = Q_OFF + D * QP;   // [D][QP]
  static constexpr int V_OFF = K_OFF + D * QP;   // [64][VP]
  static constexpr int P_OFF = V_OFF + kPsK * VP;  // [64 keys][QP]
  static constexpr int FLOATS = P_OFF + kPsK * QP;
  static constexpr size_t SMEM = FLOATS * sizeof(float);
};

// Query tiles of a sequence of n rows, and the launch's bound on their number.
__host__ __device__ __forceinline__ int ps_tiles(int n, int grp) {
  return (int)(((long long)n * grp + kPsQ - 1) / kPsQ);
}
long long ps_max_tiles(const PromptAttnDesc& a) {
  return (long long)a.M * (a.nq / a.nkv) / kPsQ + std::min(a.n_seqs, a.M);
}

// Parts of a tile's chunks: enough tiles x parts for two CTAs an SM, each part
// at least 4 chunks of the longest tile.
int ps_split(const PromptAttnDesc& a, int num_sms) {
  const long long ctas = ps_max_tiles(a) * a.nkv, chunks = a.max_pos / kPsK + a.M / kPsK + 2;
  return (int)std::max(1ll, std::min(std::min(2ll * num_sms / std::max(ctas, 1ll), chunks / 4), 64ll));
}

struct PsSeq {
  int row0, n, ctx;  // first row, rows, cached positions
};
__device__ __forceinline__ PsSeq ps_seq(const PromptAttnDesc& a, int s, bool* bad, bool* far) {
  const int c = a.base_pos ? __ldg(a.base_pos + s) : 0;
  PsSeq q;
  q.row0 = __ldg(a.row_start + s);
  q.n = __ldg(a.row_start + s + 1) - q.row0;
  q.ctx = min(max(c, 0), a.max_pos);
  *bad |= q.row0 < 0 || q.row0 > a.M || q.n < 0 || q.n > a.M - q.row0;
  *far |= q.ctx != c;
  return q;
}

template <int D>
__global__ void __launch_bounds__(kPsThreads) prompt_simt_kernel(const __grid_constant__ PromptAttnDesc a, int split) {
  using C = PsCfg<D>;
  constexpr int QP = C::QP, VP = C::VP, OC = D / 16;
  extern __shared__ __align__(16) float ps_smem[];
  float *Qs = ps_smem + C::Q_OFF, *Ks = ps_smem + C::K_OFF, *Vs = ps_smem + C::V_OFF, *Ps = ps_smem + C::P_OFF;
  __shared__ int sh_s, sh_tile, sh_good;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, grp = a.nq / a.nkv, g = blockIdx.y;
  // ---- which sequence's tile this is (the last tiles, which see most, first)
  if (tid < 32) {
    const int want = gridDim.x - 1 - blockIdx.x;
    int before = 0, s = -1, t = 0;
    bool bad = false, far = false;
    for (int b = 0; b < a.n_seqs; b += 32) {
      int k = 0;
      if (b + tid < a.n_seqs) {
        const PsSeq q = ps_seq(a, b + tid, &bad, &far);
        k = bad ? 0 : ps_tiles(q.n, grp);
      }
      int inc = k;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (tid >= o) inc += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, before + inc > want);
      if (hit && s < 0) {
        const int w = __ffs(hit) - 1;
        s = b + w;
        t = want - (before + __shfl_sync(0xffffffffu, inc - k, w));
      }
      before += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (bad || far) raise_status(a.status, ST_RANGE);
    const bool good = !__any_sync(0xffffffffu, bad);
    if (!good) s = -1;  // row_start leaves [0, M] or decreases: nothing is computed
    if (tid == 0) {
      sh_good = good;
      sh_s = s;
      sh_tile = t;
    }
  }
  __syncthreads();
  if ((a.pos || a.zero_pad) && blockIdx.y == 0 && blockIdx.z == 0)
    prompt_layer_rows<float>(a, sh_good, (long long)blockIdx.x * kPsThreads + tid, (long long)gridDim.x * kPsThreads);
  const int s = sh_s;
  if (s < 0) return;
  bool bad = false, far = false;
  const PsSeq sq = ps_seq(a, s, &bad, &far);
  const int qv0 = sh_tile * kPsQ, nqv = min(kPsQ, sq.n * grp - qv0);
  const int last = (qv0 + nqv - 1) / grp;                        // the tile's last token
  const int cctx = (sq.ctx + kPsK - 1) / kPsK, nch = cctx + last / kPsK + 1;
  const int z = blockIdx.z, c_lo = (int)((long long)nch * z / split), c_hi = (int)((long long)nch * (z + 1) / split);
  const float* q = static_cast<const float*>(a.q);
  const size_t QD = (size_t)a.nq * D, KD = (size_t)a.nkv * D;

  for (int i = tid; i < kPsQ * (D / 4); i += kPsThreads) {
    const int r = i / (D / 4), e = i % (D / 4) * 4, qv = qv0 + r;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < nqv)
      x = __ldg(reinterpret_cast<const float4*>(q + (sq.row0 + qv / grp) * QD + (size_t)(g * grp + qv % grp) * D + e));
    Qs[e * QP + r] = x.x;
    Qs[(e + 1) * QP + r] = x.y;
    Qs[(e + 2) * QP + r] = x.z;
    Qs[(e + 3) * QP + r] = x.w;
  }
  const int ty = tid >> 4, tx = tid & 15;  // rows 4 ty .., score columns 4 tx .., output columns tx OC ..
  int tok[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) tok[i] = (qv0 + 4 * ty + i) / grp;
  float m[4], l[4], o[4][OC];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int k = 0; k < OC; ++k) o[i][k] = 0.f;
  }
  const KvMap km{a.pages, a.cap, a.ps, a.max_pages, a.pool, a.nkv};

  for (int c = c_lo; c < c_hi; ++c) {
    const bool ctx = c < cctx;
    const int j0 = (ctx ? c : c - cctx) * kPsK;                   // first slot, or first own row
    const int nk = min(kPsK, ctx ? sq.ctx - j0 : last + 1 - j0);  // keys that some row of the tile sees
    const float *kp, *vp;
    size_t pitch;
    if (ctx) {
      bool badp = false;
      const size_t r0 = (size_t)km.row0(s, j0, &badp) + (size_t)g * km.head_rows();
      if (badp && tid == 0) raise_status(a.status, ST_RANGE);  // reads page 0 instead
      kp = static_cast<const float*>(a.kc) + r0 * D;
      vp = static_cast<const float*>(a.vc) + r0 * D;
      pitch = D;
    } else {
      const size_t r0 = (size_t)(sq.row0 + j0) * KD + (size_t)g * D;
      kp = static_cast<const float*>(a.kb) + r0;
      vp = static_cast<const float*>(a.vb) + r0;
      pitch = KD;
    }
    __syncthreads();  // the chunk before has been used
    for (int i = tid; i < kPsK * (D / 4); i += kPsThreads) {
      const int r = i / (D / 4), e = i % (D / 4) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      if (r < nk) {
        x = __ldg(reinterpret_cast<const float4*>(kp + r * pitch + e));
        y = __ldg(reinterpret_cast<const float4*>(vp + r * pitch + e));
      }
      Ks[e * QP + r] = x.x;
      Ks[(e + 1) * QP + r] = x.y;
      Ks[(e + 2) * QP + r] = x.z;
      Ks[(e + 3) * QP + r] = x.w;
      *reinterpret_cast<float4*>(Vs + r * VP + e) = y;
    }
    __syncthreads();
    float sc[4][4] = {};
#pragma unroll 8
    for (int e = 0; e < D; ++e) {
      const float4 x = *reinterpret_cast<const float4*>(Qs + e * QP + 4 * ty);
      const float4 y = *reinterpret_cast<const float4*>(Ks + e * QP + 4 * tx);
      const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) sc[i][k] = fmaf(xs[i], ys[k], sc[i][k]);
    }
    // keys of the chunk that row i sees
    int see[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) see[i] = ctx ? nk : min(nk, tok[i] + 1 - j0);
    float p[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        sc[i][k] = 4 * tx + k < see[i] ? sc[i][k] * a.scale : -INFINITY;
        mx = fmaxf(mx, sc[i][k]);
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float mn = fmaxf(m[i], mx), ref = mn == -INFINITY ? 0.f : mn;
      const float alpha = exp2f(m[i] - ref);  // (0 for the first keys)
      m[i] = mn;
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        p[i][k] = exp2f(sc[i][k] - ref);
        sum += p[i][k];
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      l[i] = l[i] * alpha + sum;
#pragma unroll
      for (int k = 0; k < OC; ++k) o[i][k] *= alpha;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      *reinterpret_cast<float4*>(Ps + (4 * tx + k) * QP + 4 * ty) = make_float4(p[0][k], p[1][k], p[2][k], p[3][k]);
    __syncthreads();
    // keys that every row of this thread sees, then the rest one row at a time:
    // a hidden value may be NaN or infinite, and 0 times it is NaN
    const int all = max(0, min(min(see[0], see[1]), min(see[2], see[3])));
    auto product = [&](int j, bool some) {
      const float4 w = *reinterpret_cast<const float4*>(Ps + j * QP + 4 * ty);
      const float ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < OC; k += 4) {
        const float4 v = *reinterpret_cast<const float4*>(Vs + j * VP + tx * OC + k);
        const float vs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!some || j < see[i])
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][k + e] = fmaf(ws[i], vs[e], o[i][k + e]);
      }
    };
#pragma unroll 4
    for (int j = 0; j < all; ++j) product(j, false);
#pragma unroll 1
    for (int j = all; j < nk; ++j) product(j, true);
  }

#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ty + i;
    if (r >= nqv) continue;
    const int qv = qv0 + r, head = g * grp + qv % grp;
    const size_t row = (size_t)(sq.row0 + qv / grp);
    if (split == 1) {
      const float inv = 1.f / l[i];  // (every row sees itself: l > 0, or NaN)
      float* out = static_cast<float*>(a.out) + row * QD + (size_t)head * D + tx * OC;
#pragma unroll
      for (int k = 0; k < OC; k += 4)
        *reinterpret_cast<float4*>(out + k) =
            make_float4(o[i][k] * inv, o[i][k + 1] * inv, o[i][k + 2] * inv, o[i][k + 3] * inv);
    } else {
      float* part = static_cast<float*>(a.work) + ((size_t)z * a.M * a.nq + row * a.nq + head) * (D + 4);
#pragma unroll
      for (int k = 0; k < OC; k += 4)
        *reinterpret_cast<float4*>(part + tx * OC + k) = make_float4(o[i][k], o[i][k + 1], o[i][k + 2], o[i][k + 3]);
      if (tx == 0) {
        part[D] = m[i];
        part[D + 1] = l[i];
      }
    }
  }
}

// Joins the parts of each query vector, one warp each.
template <int D>
__global__ void __launch_bounds__(128) prompt_simt_merge_kernel(const __grid_constant__ PromptAttnDesc a, int split) {
  pdl_wait();
  pdl_launch_dependents();
  const int w = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (w >= a.M * a.nq) return;
  // rows of no sequence are left as they were
  const int row = w / a.nq;
  bool in = false, bad = false, far = false;
  for (int b = lane; b < a.n_seqs; b += 32) {
    const PsSeq q = ps_seq(a, b, &bad, &far);
    in |= row >= q.row0 && row - q.row0 < q.n;
  }
  if (!__any_sync(0xffffffffu, in) || __any_sync(0xffffffffu, bad)) return;
  const float* part = static_cast<const float*>(a.work) + (size_t)w * (D + 4);
  const size_t step = (size_t)a.M * a.nq * (D + 4);
  float M = -INFINITY, L = 0.f, o[D / 32] = {};
  for (int z = 0; z < split; ++z) M = fmaxf(M, part[z * step + D]);
  for (int z = 0; z < split; ++z) {
    const float f = exp2f(part[z * step + D] - (M == -INFINITY ? 0.f : M));
    L = fmaf(part[z * step + D + 1], f, L);
#pragma unroll
    for (int k = 0; k < D / 32; ++k) o[k] = fmaf(part[z * step + lane + 32 * k], f, o[k]);
  }
  float* out = static_cast<float*>(a.out) + (size_t)w * D;
#pragma unroll
  for (int k = 0; k < D / 32; ++k) out[lane + 32 * k] = o[k] / L;
}

template <int D>
cudaError_t ps_launch(const PromptAttnDesc& a, int num_sms, cudaStream_t st) {
  const int split = ps_split(a, num_sms);
  cudaError_t e =
      cudaFuncSetAttribute(prompt_simt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)PsCfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_pdl(prompt_simt_kernel<D>, dim3((unsigned)ps_max_tiles(a), a.nkv, split), dim3(kPsThreads),
                 PsCfg<D>::SMEM, st, a, split);
  if (e != cudaSuccess || split == 1) return e;
  return launch_pdl(prompt_simt_merge_kernel<D>, dim3((unsigned)(((long long)a.M * a.nq + 3) / 4)), dim3(128), 0, st, a,
                    split);
}

}  // namespace

size_t prompt_attn_workspace(const PromptAttnDesc& a, int num_sms) {
  if (a.dtype == DFLASH_BF16) return prompt_tc_workspace(a, num_sms);
  const int split = ps_split(a, num_sms);
  return split == 1 ? 0 : (size_t)split * a.M * a.nq * (a.d + 4) * sizeof(float);
}

cudaError_t launch_prompt_attention(const PromptAttnDesc& a, int num_sms, cudaStream_t st) {
  if (a.dtype == DFLASH_BF16) return launch_prompt_tc(a, num_sms, st);
  return a.d == 128 ? ps_launch<128>(a, num_sms, st) : ps_launch<64>(a, num_sms, st);
}

}  // namespace dfl
