// k_qk_norm.cu -- RMS norms of query and key heads with the position rotation,
// in one pass over the QKV projection's output (see dflash_qk_norm_rope).
//
// A group of d / 8 lanes has a head: lane i holds elements 4i .. 4i+3 and their
// rotation partners d/2 further on, so the head's sum of squares is a few
// shuffles and the rotation needs no exchange.  Every element is read once and
// written once, which bounds the kernel: 8192 rows of 32 + 16 heads of 128, fp32
// to bf16, 302 MB in 48 us, 94% of the copy rate.  A group takes two heads of a
// row, so that four 16-byte loads a thread are in flight and the position's
// cosines are fetched once for both; 1 / 2 / 3 / 4 / 8 heads 58 / 49 / 49 / 50 /
// 58 us, 256 threads a CTA instead of 128 51.
#include "common.cuh"
#include "epilogue.cuh"
#include "internal.h"
#include "launch.cuh"

namespace dfl {

namespace {

constexpr int kQnThreads = 128;
constexpr int kQnHeads = 2;  // heads of a group

// Four consecutive elements as floats.
template <typename T>
__device__ __forceinline__ float4 qn_load(const T* p);
template <>
__device__ __forceinline__ float4 qn_load<float>(const float* p) {
  return __ldg(reinterpret_cast<const float4*>(p));
}
template <>
__device__ __forceinline__ float4 qn_load<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xFFFF0000u));
}
__device__ __forceinline__ void qn_store(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void qn_store(__nv_bfloat16* p, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// HPG consecutive heads of a row per group.
template <typename TI, typename TO, int D, int HPG>
__global__ void __launch_bounds__(kQnThreads) qk_norm_kernel(const __grid_constant__ QkNormDesc a, uint32_t per_row,
                                                             uint32_t groups) {
  constexpr int L = D / 8;  // lanes of a group
  pdl_launch_dependents();
  const uint32_t u = blockIdx.x * (kQnThreads / L) + threadIdx.x / L;
  const int i = threadIdx.x % L;
  pdl_wait();
  const int heads = a.nq + 2 * a.nkv;
  const int m = (int)(min(u, groups - 1) / per_row), h0 = (int)(min(u, groups - 1) % per_row) * HPG;
  const TI* src = static_cast<const TI*>(a.qkv) + (size_t)m * a.stride + (size_t)h0 * D + 4 * i;
  float4 x[HPG], y[HPG];
#pragma unroll
  for (int j = 0; j < HPG; ++j) {
    x[j] = y[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (h0 + j < heads) {
      x[j] = qn_load<TI>(src + j * D);
      y[j] = qn_load<TI>(src + j * D + D / 2);
    }
  }
  const int s = m / a.rows;
  const int pos = __ldg(a.base_pos + s) + m % a.rows;
  bool live = u < groups;
  if (live && (pos < 0 || pos >= a.rope_max_pos)) {
    if (h0 == 0 && i == 0) raise_status(a.status, ST_RANGE);
    live = false;
  }
  const float4* cs = reinterpret_cast<const float4*>(a.rope_cs + ((size_t)(live ? pos : 0) * (D / 2) + 4 * i) * 2);
  const float4 c0 = __ldg(cs), c1 = __ldg(cs + 1);  // (cos, sin) of elements 4i, 4i+1; 4i+2, 4i+3
  // where the row's keys and values go
  size_t row = (size_t)m * a.nkv, step = 1, rows = (size_t)a.M * a.nkv;  // (rows: of the destination)
  bool kv_live = live;
  if (a.cache && h0 + HPG > a.nq) {
    const KvMap km{a.pages, a.cap, a.ps, a.max_pages, a.pool, a.nkv};
    bool bad = live && pos >= a.cap;
    if (live && !bad) {
      row = km.row0(s, pos, &bad);
      step = km.head_rows();
      rows = (size_t)(a.pages ? a.pool : a.M / a.rows) * a.nkv * step;
    }
    if (bad) {
      if (i == 0) raise_status(a.status, ST_RANGE);
      kv_live = false;
    }
  }
#pragma unroll
  for (int j = 0; j < HPG; ++j) {
    const int h = h0 + j;
    const bool is_q = h < a.nq, is_v = h >= a.nq + a.nkv;
    const TO* gain = static_cast<const TO*>(is_q ? a.q_norm : is_v ? nullptr : a.k_norm);
    float4 p = x[j], q = y[j];
    float ss = p.x * p.x + p.y * p.y + p.z * p.z + p.w * p.w + (q.x * q.x + q.y * q.y + q.z * q.z + q.w * q.w);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (gain) {
      const float r = rsqrtf(ss * (1.f / D) + a.eps);
      const float4 g0 = qn_load<TO>(gain + 4 * i), g1 = qn_load<TO>(gain + D / 2 + 4 * i);
      p = make_float4(p.x * r * g0.x, p.y * r * g0.y, p.z * r * g0.z, p.w * r * g0.w);
      q = make_float4(q.x * r * g1.x, q.y * r * g1.y, q.z * r * g1.z, q.w * r * g1.w);
    }
    if (!is_v) {
      rope_rot(p.x, q.x, c0.x, c0.y, p.x, q.x);
      rope_rot(p.y, q.y, c0.z, c0.w, p.y, q.y);
      rope_rot(p.z, q.z, c1.x, c1.y, p.z, q.z);
      rope_rot(p.w, q.w, c1.z, c1.w, p.w, q.w);
    }
    if (h >= heads || !(is_q ? live : kv_live)) continue;
    if (!DFL_CHECK(is_q ? m < a.M : row + (size_t)((h - a.nq) % a.nkv) * step < rows, a.status)) continue;
    TO* out = is_q ? static_cast<TO*>(a.q) + ((size_t)m * a.nq + h) * D
                   : static_cast<TO*>(is_v ? a.v : a.k) + (row + (size_t)((h - a.nq) % a.nkv) * step) * D;
    qn_store(out + 4 * i, p);
    qn_store(out + D / 2 + 4 * i, q);
  }
}

template <typename TI, typename TO, int D, int HPG>
cudaError_t qn_launch(const QkNormDesc& a, cudaStream_t st) {
  const int per_row = (a.nq + 2 * a.nkv + HPG - 1) / HPG;
  const long long groups = (long long)a.M * per_row;
  constexpr int PER = kQnThreads / (D / 8);
  return launch_pdl(qk_norm_kernel<TI, TO, D, HPG>, dim3((unsigned)((groups + PER - 1) / PER)), dim3(kQnThreads), 0, st,
                    a,
                    (uint32_t)per_row, (uint32_t)groups);
}

template <typename TI, typename TO>
cudaError_t qn_by_dim(const QkNormDesc& a, cudaStream_t st) {
  return a.d == 128 ? qn_launch<TI, TO, 128, kQnHeads>(a, st) : qn_launch<TI, TO, 64, kQnHeads>(a, st);
}

}  // namespace

cudaError_t launch_qk_norm(const QkNormDesc& a, cudaStream_t st) {
  if (a.dtype == DFLASH_BF16)
    return a.src_dtype == DFLASH_BF16 ? qn_by_dim<__nv_bfloat16, __nv_bfloat16>(a, st)
                                      : qn_by_dim<float, __nv_bfloat16>(a, st);
  return a.src_dtype == DFLASH_BF16 ? qn_by_dim<__nv_bfloat16, float>(a, st) : qn_by_dim<float, float>(a, st);
}

}  // namespace dfl
