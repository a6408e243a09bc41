// k_prompt_attn.cu -- causal attention of packed prompts in fp32, and the choice
// between it and the tensor-core kernel (k_prompt_attn_tc.cu, bf16).
//
// A CTA has a tile of 64 (or 16) query vectors of one (sequence, KV head), the group's
// query heads side by side (vector = token * group + head), and walks the keys
// that the tile sees in chunks of 64: cached slots, then the sequence's own
// rows up to the tile's last token.  Scores and outputs are register tiles
// (4 x 4 and 4 x d/16 per thread, 64 multiply-adds for eight 16-byte reads of
// shared memory), the softmax runs along with a running maximum and sum.  Full
// precision has no tensor-core form, so the fp32 units bound it.  Where few tiles would leave SMs idle, the chunks of a tile are cut
// into `split` parts of equal number that a second kernel joins.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "prompt_attn.cuh"

namespace dfl {

namespace {

constexpr int kPsK = 64;        // keys of a chunk
constexpr int kPsThreads = 256;

// R: query vectors per thread; a tile holds 16 R.
template <int D, int R>
struct PsCfg {
  static constexpr int Q = 16 * R;
  static constexpr int RP = D + 4;  // pitches, in floats: 16-byte reads of eight rows meet all banks
  static constexpr int PP = kPsK + 4;
  static constexpr int Q_OFF = 0;                  // [Q][RP]
  static constexpr int K_OFF = Q_OFF + Q * RP;      // [64][RP]
  static constexpr int V_OFF = K_OFF + kPsK * RP;  // [64][RP]
  static constexpr int P_OFF = V_OFF + kPsK * RP;  // [Q][PP]
  static constexpr int FLOATS = P_OFF + Q * PP;
  static constexpr size_t SMEM = FLOATS * sizeof(float);
};

// Query tiles (of `size` vectors) of a sequence of n rows, and the launch's
// bound on their number.
__host__ __device__ __forceinline__ int ps_tiles(int n, int grp, int size) {
  return (int)(((long long)n * grp + size - 1) / size);
}
long long ps_max_tiles(const PromptAttnDesc& a, int size) {
  return (long long)a.M * (a.nq / a.nkv) / size + std::min(a.n_seqs, a.M);
}

// Tiles of 64 vectors, or of 16 where those leave SMs idle (three prompts of 64
// rows, 4 heads: 6.4 us, 10.4 with 64).
int ps_rows(const PromptAttnDesc& a, int num_sms) { return ps_max_tiles(a, 64) * a.nkv < num_sms ? 1 : 4; }

// Parts of a tile's chunks: enough tiles x parts for two CTAs an SM, each part
// at least 4 chunks of the longest tile.
int ps_split(const PromptAttnDesc& a, int num_sms) {
  const long long ctas = ps_max_tiles(a, 16 * ps_rows(a, num_sms)) * a.nkv, chunks = a.max_pos / kPsK + a.M / kPsK + 2;
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

template <int D, int R>
__global__ void __launch_bounds__(kPsThreads) prompt_simt_kernel(const __grid_constant__ PromptAttnDesc a, int split) {
  using C = PsCfg<D, R>;
  constexpr int RP = C::RP, PP = C::PP, OV = D / 64;  // OV: float4s of an output row per thread
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
        k = bad ? 0 : ps_tiles(q.n, grp, C::Q);
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
  const int qv0 = sh_tile * C::Q, nqv = min(C::Q, sq.n * grp - qv0);
  const int last = (qv0 + nqv - 1) / grp;                        // the tile's last token
  const int cctx = (sq.ctx + kPsK - 1) / kPsK, nch = cctx + last / kPsK + 1;
  const int z = blockIdx.z, c_lo = (int)((long long)nch * z / split), c_hi = (int)((long long)nch * (z + 1) / split);
  const float* q = static_cast<const float*>(a.q);
  const size_t QD = (size_t)a.nq * D, KD = (size_t)a.nkv * D;

  for (int i = tid; i < C::Q * (D / 4); i += kPsThreads) {
    const int r = i / (D / 4), e = i % (D / 4) * 4, qv = qv0 + r;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < nqv && DFL_CHECK(sq.row0 + qv / grp < a.M, a.status))
      x = __ldg(reinterpret_cast<const float4*>(q + (sq.row0 + qv / grp) * QD + (size_t)(g * grp + qv % grp) * D + e));
    *reinterpret_cast<float4*>(Qs + r * RP + e) = x;
  }
  // a thread's rows are ty + 16 i, its score columns tx + 16 k, its output columns 64 v + 4 tx ..
  const int ty = tid >> 4, tx = tid & 15;
  int tok[R];
#pragma unroll
  for (int i = 0; i < R; ++i) tok[i] = (qv0 + ty + 16 * i) / grp;
  float m[R], l[R];
  float4 o[R][OV];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int v = 0; v < OV; ++v) o[i][v] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const KvMap km{a.pages, a.cap, a.ps, a.max_pages, a.pool, a.nkv};

  for (int c = c_lo; c < c_hi; ++c) {
    const bool ctx = c < cctx;
    const int j0 = (ctx ? c : c - cctx) * kPsK;                   // first slot, or first own row
    const int nk = min(kPsK, ctx ? sq.ctx - j0 : last + 1 - j0);  // keys that some row of the tile sees
    const float *kp, *vp;
    size_t pitch;
    long long first, rows;  // the chunk's first row, those of its buffer
    if (ctx) {
      bool badp = false;
      const size_t r0 = (size_t)km.row0(s, j0, &badp) + (size_t)g * km.head_rows();
      if (badp && tid == 0) raise_status(a.status, ST_RANGE);  // reads page 0 instead
      kp = static_cast<const float*>(a.kc) + r0 * D;
      vp = static_cast<const float*>(a.vc) + r0 * D;
      pitch = D;
      first = (long long)r0;
      rows = (long long)(a.pages ? a.pool : a.n_seqs) * a.nkv * km.head_rows();
    } else {
      const size_t r0 = (size_t)(sq.row0 + j0) * KD + (size_t)g * D;
      kp = static_cast<const float*>(a.kb) + r0;
      vp = static_cast<const float*>(a.vb) + r0;
      pitch = KD;
      first = sq.row0 + j0;
      rows = a.M;
    }
    __syncthreads();  // the chunk before has been used
    bool odd = false;  // a value is NaN or infinite
    for (int i = tid; i < kPsK * (D / 4); i += kPsThreads) {
      const int r = i / (D / 4), e = i % (D / 4) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      if (r < nk && DFL_CHECK(first + r < rows, a.status)) {
        x = __ldg(reinterpret_cast<const float4*>(kp + r * pitch + e));
        y = __ldg(reinterpret_cast<const float4*>(vp + r * pitch + e));
      }
      *reinterpret_cast<float4*>(Ks + r * RP + e) = x;
      *reinterpret_cast<float4*>(Vs + r * RP + e) = y;
      odd |= !(fabsf(y.x) < INFINITY && fabsf(y.y) < INFINITY && fabsf(y.z) < INFINITY && fabsf(y.w) < INFINITY);
    }
    odd = __syncthreads_or(odd) != 0;
    float sc[R][4] = {};
#pragma unroll 4
    for (int e = 0; e < D; e += 4) {
      float4 x[R], y[4];
#pragma unroll
      for (int i = 0; i < R; ++i) x[i] = *reinterpret_cast<const float4*>(Qs + (ty + 16 * i) * RP + e);
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = *reinterpret_cast<const float4*>(Ks + (tx + 16 * k) * RP + e);
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          sc[i][k] = fmaf(x[i].x, y[k].x, sc[i][k]);
          sc[i][k] = fmaf(x[i].y, y[k].y, sc[i][k]);
          sc[i][k] = fmaf(x[i].z, y[k].z, sc[i][k]);
          sc[i][k] = fmaf(x[i].w, y[k].w, sc[i][k]);
        }
    }
    // keys of the chunk that row i sees
    int see[R];
#pragma unroll
    for (int i = 0; i < R; ++i) see[i] = ctx ? nk : min(nk, tok[i] + 1 - j0);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        sc[i][k] = tx + 16 * k < see[i] ? sc[i][k] * a.scale : -INFINITY;
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
        const float p = exp2f(sc[i][k] - ref);
        Ps[(ty + 16 * i) * PP + tx + 16 * k] = p;
        sum += p;
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      l[i] = l[i] * alpha + sum;
#pragma unroll
      for (int v = 0; v < OV; ++v)
        o[i][v] = make_float4(o[i][v].x * alpha, o[i][v].y * alpha, o[i][v].z * alpha, o[i][v].w * alpha);
    }
    __syncwarp();  // (a row's weights come from the half warp that uses them)
    // All keys, four at a time: what is hidden has weight 0 (behind the last key
    // values are 0 too).  But 0 times a NaN or infinite value is NaN: where
    // there are such, keys that every row of this thread sees, then the rest
    // one row at a time.
    int all = (nk + 3) & ~3;
    if (odd) {
      all = nk;
#pragma unroll
      for (int i = 0; i < R; ++i) all = min(all, see[i]);
      all = max(all, 0) & ~3;
    }
    auto axpy = [](float w, const float4& v, float4& y) {
      y.x = fmaf(w, v.x, y.x);
      y.y = fmaf(w, v.y, y.y);
      y.z = fmaf(w, v.z, y.z);
      y.w = fmaf(w, v.w, y.w);
    };
#pragma unroll 2
    for (int j = 0; j < all; j += 4) {
      float4 w[R];
#pragma unroll
      for (int i = 0; i < R; ++i) w[i] = *reinterpret_cast<const float4*>(Ps + (ty + 16 * i) * PP + j);
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int v = 0; v < OV; ++v) {
          const float4 x = *reinterpret_cast<const float4*>(Vs + (j + e) * RP + 64 * v + 4 * tx);
#pragma unroll
          for (int i = 0; i < R; ++i) axpy(e == 0 ? w[i].x : e == 1 ? w[i].y : e == 2 ? w[i].z : w[i].w, x, o[i][v]);
        }
    }
#pragma unroll 1
    for (int j = all; j < nk; ++j)
#pragma unroll
      for (int v = 0; v < OV; ++v) {
        const float4 x = *reinterpret_cast<const float4*>(Vs + j * RP + 64 * v + 4 * tx);
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (j < see[i]) axpy(Ps[(ty + 16 * i) * PP + j], x, o[i][v]);
      }
  }

#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = ty + 16 * i;
    if (r >= nqv) continue;
    const int qv = qv0 + r, head = g * grp + qv % grp;
    const size_t row = (size_t)(sq.row0 + qv / grp);
    if (!DFL_CHECK(row < (size_t)a.M && head < a.nq && z < split, a.status)) continue;
    const float f = split == 1 ? 1.f / l[i] : 1.f;  // (every row sees itself: l > 0, or NaN)
    float* part = static_cast<float*>(a.work) + ((size_t)z * a.M * a.nq + row * a.nq + head) * (D + 4);
    float* out = split == 1 ? static_cast<float*>(a.out) + row * QD + (size_t)head * D : part;
#pragma unroll
    for (int v = 0; v < OV; ++v)
      *reinterpret_cast<float4*>(out + 64 * v + 4 * tx) =
          make_float4(o[i][v].x * f, o[i][v].y * f, o[i][v].z * f, o[i][v].w * f);
    if (split > 1 && tx == 0) {
      part[D] = m[i];
      part[D + 1] = l[i];
    }
  }
}

// Joins the parts (at most 64) of each query vector, one warp each.
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
  float m[2], l[2];  // of parts lane, lane + 32
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int z = lane + 32 * k;
    m[k] = z < split ? part[z * step + D] : -INFINITY;
    l[k] = z < split ? part[z * step + D + 1] : 0.f;
  }
  const float M = warp_max(fmaxf(m[0], m[1])), ref = M == -INFINITY ? 0.f : M;
  float L = 0.f, o[D / 32] = {};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    m[k] = exp2f(m[k] - ref);
    L = fmaf(l[k], m[k], L);
  }
  L = warp_sum(L);
#pragma unroll 1
  for (int b = 0; b < split; b += 8) {  // eight parts' loads in flight
    float x[8][D / 32];
#pragma unroll
    for (int u = 0; u < 8; ++u)
#pragma unroll
      for (int k = 0; k < D / 32; ++k) x[u][k] = b + u < split ? part[(b + u) * step + lane + 32 * k] : 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float f = __shfl_sync(0xffffffffu, b < 32 ? m[0] : m[1], (b + u) & 31);
#pragma unroll
      for (int k = 0; k < D / 32; ++k) o[k] = fmaf(x[u][k], f, o[k]);
    }
  }
  float* out = static_cast<float*>(a.out) + (size_t)w * D;
#pragma unroll
  for (int k = 0; k < D / 32; ++k) out[lane + 32 * k] = o[k] / L;
}

template <int D, int R>
cudaError_t ps_launch(const PromptAttnDesc& a, int num_sms, cudaStream_t st) {
  using C = PsCfg<D, R>;
  const int split = ps_split(a, num_sms);
  cudaError_t e =
      cudaFuncSetAttribute(prompt_simt_kernel<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_pdl(prompt_simt_kernel<D, R>, dim3((unsigned)ps_max_tiles(a, C::Q), a.nkv, split), dim3(kPsThreads),
                 C::SMEM, st, a, split);
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
  if (ps_rows(a, num_sms) == 1) return a.d == 128 ? ps_launch<128, 1>(a, num_sms, st) : ps_launch<64, 1>(a, num_sms, st);
  return a.d == 128 ? ps_launch<128, 4>(a, num_sms, st) : ps_launch<64, 4>(a, num_sms, st);
}

}  // namespace dfl
