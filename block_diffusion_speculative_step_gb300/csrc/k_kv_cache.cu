// k_kv_cache.cu -- cache rows written (quantised to 8 bits, or copied) and
// read back, for many layers in one launch.
//
// An 8-bit row is x_i = c_i 2^e with c_i in e4m3 and one exponent e per
// (slot, KV head): e is the smallest exponent with max |x| <= 448 * 2^e, the
// largest e4m3 value.  With max |x| = f 2^k, f in [1/2, 1) (frexp) and 448 =
// 7/8 * 2^9 this is e = k - 9, plus one when f > 7/8.  A power of two scales
// without rounding (the largest codes land in (224, 448]), so the only error
// is e4m3's own half step, 2^-4 relative, and elements below 2^-17 of the
// row's maximum reach e4m3's subnormals.  e is held to [-60, 60]: magnitudes
// outside 448 * 2^+-60 do not occur in a trained model's cache, and within it
// no product of scales that attention forms leaves the fp32 range.
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"
#include "launch.cuh"

namespace dfl {

constexpr int kKvThreads = 256;
constexpr int kKvExpLim = 60;
constexpr int kKvExpBias = 127;

__device__ __forceinline__ float pow2_f(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// Slot of row i (position base_pos[s] + i) of sequence s, as the cache row of
// KV head 0; false when the row is skipped.
__device__ __forceinline__ bool kv_row(const KvRowsDesc& k, const int32_t* pages, int s, int i, int n, size_t* row,
                                       uint32_t* head_rows) {
  const long long pos = (long long)__ldg(k.base_pos + s) + i;
  if (k.window > 0 && i + k.window < n) return false;  // a later row of this call takes the same slot
  const long long slot = k.window > 0 ? pos % k.window : pos;
  if (pos < 0 || slot >= k.cap) {
    raise_status(k.status, ST_RANGE);
    return false;
  }
  const KvMap km{pages, k.cap, k.ps, k.max_pages, k.pool, k.nkv};
  bool bad = false;
  *row = km.row0(s, (int)slot, &bad);
  *head_rows = (uint32_t)km.head_rows();
  if (bad) raise_status(k.status, ST_RANGE);
  return !bad;
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint4 u;
  __nv_bfloat162* b = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = u;
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

// Grid: x over row vectors (s, i, head), y = 2 * layer + (0: K, 1: V).
// Every d / 8 neighbouring threads hold one vector, 8 elements each.
template <typename T, bool Q8>
__global__ void __launch_bounds__(kKvThreads) kv_write_kernel(const __grid_constant__ KvRowsDesc k,
                                                              const __grid_constant__ KvRowsLayers l) {
  pdl_wait();
  pdl_launch_dependents();
  const int tpv = k.d / 8;  // threads per vector: 8 or 16
  const long long t = (long long)blockIdx.x * kKvThreads + threadIdx.x;
  const long long vec = t / tpv;
  const int e0 = (int)(t % tpv) * 8;
  const int layer = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  bool on = vec < (long long)k.S * k.rows * k.nkv;
  const int m = on ? (int)(vec / k.nkv) : 0, head = (int)(vec % k.nkv);
  const int s = m / k.rows, i = m % k.rows;
  const int n = k.valid ? min(__ldg(k.valid + s), k.rows) : k.rows;
  on = on && i < n;
  int src = i;
  if (on && k.row_index) {
    src = __ldg(k.row_index + m);
    if (src < 0 || src >= k.rows) {
      raise_status(k.status, ST_RANGE);
      on = false;
    }
  }
  size_t row = 0;
  uint32_t hr = 0;
  on = on && kv_row(k, l.pages[layer], s, i, n, &row, &hr);
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.f;
  if (on) {
    const T* p = reinterpret_cast<const T*>(is_v ? l.src_v[layer] : l.src_k[layer]);
    load8(p + (((size_t)s * k.rows + src) * k.nkv + head) * k.d + e0, v);
  }
  row += (size_t)head * hr;
  void* dst = is_v ? l.dst_v[layer] : l.dst_k[layer];
  if constexpr (!Q8) {
    if (on) store8(reinterpret_cast<T*>(dst) + row * k.d + e0, v);
  } else {
    float mx = 0.f;
    uint32_t odd = 0;  // bit j: element j is NaN or infinite
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = fabsf(v[j]);
      if (a < INFINITY) mx = fmaxf(mx, a);
      else odd |= 1u << j;
    }
    for (int o = tpv >> 1; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (!on) return;
    if (odd) raise_status(k.status, ST_NUMERIC);
    int e = -kKvExpLim;
    if (mx > 0.f) {
      int kk;
      const float f = frexpf(mx, &kk);
      e = min(max(kk - 9 + (f > 0.875f ? 1 : 0), -kKvExpLim), kKvExpLim);
    }
    const float inv = pow2_f(-e);
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const __nv_fp8x2_storage_t a = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * h] * inv, v[4 * h + 1] * inv),
                                                              __NV_SATFINITE, __NV_E4M3);
      const __nv_fp8x2_storage_t b = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * h + 2] * inv, v[4 * h + 3] * inv),
                                                              __NV_SATFINITE, __NV_E4M3);
      w[h] = (uint32_t)a | ((uint32_t)b << 16);
    }
    if (odd) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if ((odd >> j) & 1u) w[j >> 2] = (w[j >> 2] & ~(0xFFu << (8 * (j & 3)))) | (0x7Fu << (8 * (j & 3)));
    }
    *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(dst) + row * k.d + e0) = make_uint2(w[0], w[1]);
    if (e0 == 0) (is_v ? l.v_exp[layer] : l.k_exp[layer])[row] = (uint8_t)(e + kKvExpBias);
  }
}

template <typename T, bool Q8>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const __grid_constant__ KvRowsDesc k,
                                                             const __grid_constant__ KvRowsLayers l) {
  pdl_wait();
  pdl_launch_dependents();
  const int tpv = k.d / 8;
  const long long t = (long long)blockIdx.x * kKvThreads + threadIdx.x;
  const long long vec = t / tpv;
  const int e0 = (int)(t % tpv) * 8;
  const int layer = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  if (vec >= (long long)k.S * k.rows * k.nkv) return;
  const int m = (int)(vec / k.nkv), head = (int)(vec % k.nkv);
  const int s = m / k.rows, i = m % k.rows;
  const int n = k.valid ? min(__ldg(k.valid + s), k.rows) : k.rows;
  if (i >= n) return;
  size_t row;
  uint32_t hr;
  if (!kv_row(k, l.pages[layer], s, i, 0, &row, &hr)) return;
  row += (size_t)head * hr;
  const void* src = is_v ? l.src_v[layer] : l.src_k[layer];
  float v[8];
  if constexpr (!Q8) {
    load8(reinterpret_cast<const T*>(src) + row * k.d + e0, v);
  } else {
    const uint2 c = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(src) + row * k.d + e0);
    const float sc = pow2_f((int)__ldg((is_v ? l.v_exp[layer] : l.k_exp[layer]) + row) - kKvExpBias);
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
  void* dst = is_v ? l.dst_v[layer] : l.dst_k[layer];
  store8(reinterpret_cast<T*>(dst) + ((size_t)m * k.nkv + head) * k.d + e0, v);
}

template <typename F>
static cudaError_t kv_launch(F kernel, const KvRowsDesc& k, const KvRowsLayers& l, cudaStream_t st) {
  const long long thr = (long long)k.S * k.rows * k.nkv * (k.d / 8);
  if (thr == 0) return cudaSuccess;
  const dim3 grid((unsigned)((thr + kKvThreads - 1) / kKvThreads), 2 * k.n_layers);
  return launch_pdl(kernel, grid, dim3(kKvThreads), 0, st, k, l);
}

cudaError_t launch_kv_write(const KvRowsDesc& k, const KvRowsLayers& l, cudaStream_t st) {
  const bool q8 = l.k_exp[0] != nullptr;
  if (k.dtype == DFLASH_BF16)
    return q8 ? kv_launch(kv_write_kernel<__nv_bfloat16, true>, k, l, st)
              : kv_launch(kv_write_kernel<__nv_bfloat16, false>, k, l, st);
  return q8 ? kv_launch(kv_write_kernel<float, true>, k, l, st) : kv_launch(kv_write_kernel<float, false>, k, l, st);
}

cudaError_t launch_kv_read(const KvRowsDesc& k, const KvRowsLayers& l, cudaStream_t st) {
  const bool q8 = l.k_exp[0] != nullptr;
  if (k.dtype == DFLASH_BF16)
    return q8 ? kv_launch(kv_read_kernel<__nv_bfloat16, true>, k, l, st)
              : kv_launch(kv_read_kernel<__nv_bfloat16, false>, k, l, st);
  return q8 ? kv_launch(kv_read_kernel<float, true>, k, l, st) : kv_launch(kv_read_kernel<float, false>, k, l, st);
}

}  // namespace dfl
