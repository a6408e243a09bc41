// k_kv_cache.cu -- cache rows written (quantised to 8 bits, or copied) and
// read back, for many layers in one launch.
//
// An 8-bit row is x_i = c_i 2^e with c_i in e4m3 and one exponent e per
// (slot, KV head): e is the smallest exponent with max |x| <= 448 * 2^e, the
// largest e4m3 value.  With max |x| = f 2^k, f in [1/2, 1) (frexp) and 448 =
// 7/8 * 2^9 this is e = k - 9, plus one when f > 7/8.  A power of two scales
// without rounding (the largest codes land in (224, 448]), so the only error
// is e4m3's own half step: 2^-4 relative, and for elements below about 2^-14 of
// the row's maximum, e4m3's subnormals, 2^-10 * 2^e, at most 2^-10 / 224 of the
// maximum.  e is held to [-60, 60]: magnitudes
// outside 448 * 2^+-60 do not occur in a trained model's cache, and within it
// no product of scales that attention forms leaves the fp32 range.
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"
#include "launch.cuh"

namespace dfl {

constexpr int kKvThreads = 128;
constexpr int kKvHeads = 4;
constexpr int kKvExpLim = 60;
constexpr int kKvExpBias = 127;

__device__ __forceinline__ float pow2_f(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// Slot of row i (position base + i) of sequence s, as the cache row of
// KV head 0; false when the row is skipped.
__device__ __forceinline__ bool kv_row(const KvRowsDesc& k, const int32_t* pages, int s, int base, int i, int n, size_t* row,
                                       uint32_t* head_rows) {
  if (k.window > 0 && i + k.window < n) return false;  // a later row of this call takes the same slot
  const uint32_t pos = (uint32_t)base + (uint32_t)i;   // (i < 2^27: from base >= 0 no wrap)
  const uint32_t slot = k.window > 0 ? pos % (uint32_t)k.window : pos;
  if ((base < 0 && (int)pos < 0) || slot >= (uint32_t)k.cap) {
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

// A thread's share: 8 elements of up to kKvHeads neighbouring heads of one row
// of K or V.  A row's cost should be its bytes (read once, written once), but
// with a head per thread the issue slots went to addresses -- position, page,
// divisions -- and to frexp and shuffles; so an address serves four heads,
// whose loads are in flight together.  32 sequences x 16 rows x 8 heads of 128
// x 36 layers, written in 8 bits and read back: 77 -> 43 us, 33 us with the
// maxima taken on bit patterns, 31 us in blocks of 128 (the rows' bytes alone
// would take 18).  Two and eight heads a thread: 41 and 33 us against 32.
struct KvUnit {
  int s, i, m, head, heads, e0, layer;
  bool is_v, on;
  __device__ __forceinline__ KvUnit(const KvRowsDesc& k) {
    const uint32_t tpv = (uint32_t)k.d >> 3;  // threads per vector: 8 or 16
    const uint32_t n_hg = ((uint32_t)k.nkv + kKvHeads - 1) / kKvHeads;
    const uint32_t u = blockIdx.x * (kKvThreads / tpv) + threadIdx.x / tpv;  // < 2^27 + 32
    m = (int)(u / n_hg);
    head = (int)(u % n_hg) * kKvHeads;
    heads = min(kKvHeads, k.nkv - head);
    e0 = (int)(threadIdx.x % tpv) * 8;
    s = (int)((uint32_t)m / (uint32_t)k.rows);
    i = m - s * k.rows;
    layer = blockIdx.y >> 1;
    is_v = blockIdx.y & 1;
    on = s < k.S;
  }
};

// Eight elements as loaded, their magnitudes' largest bit pattern (patterns of
// non-negative floats order as integers), and their codes.
template <typename T>
struct KvRow8;
template <>
struct KvRow8<__nv_bfloat16> {
  uint32_t w[4];
  static constexpr uint32_t kInf = 0x7F80u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  }
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0u; }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ float at(int j) const {
    return __uint_as_float(j & 1 ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
  }
  __device__ __forceinline__ uint32_t top() const {
    constexpr uint32_t M = 0x7FFF7FFFu;
    const uint32_t m = __vimax3_u16x2(w[0] & M, w[1] & M, __vmaxu2(w[2] & M, w[3] & M));
    return max(m >> 16, m & 0xFFFFu);
  }
  static __device__ __forceinline__ float value(uint32_t top) { return __uint_as_float(top << 16); }
};
template <>
struct KvRow8<float> {
  float v[8];
  static constexpr uint32_t kInf = 0x7F800000u;
  __device__ __forceinline__ void load(const float* p) { load8(p, v); }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
  }
  __device__ __forceinline__ void store(float* p) const { store8(p, v); }
  __device__ __forceinline__ float at(int j) const { return v[j]; }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    return m;
  }
  static __device__ __forceinline__ float value(uint32_t top) { return __uint_as_float(top); }
};

// The smallest e with mx <= 448 * 2^e, held to the limits.  mx = g 2^x with g
// in [1, 2): e = x - 8, plus one when g > 1.75.  (0 and subnormals: the lower limit.)
__device__ __forceinline__ int kv_exponent(float mx) {
  const int b = __float_as_int(mx);
  const int e = (b >> 23) - 127 - 8 + ((b & 0x7FFFFF) > 0x600000 ? 1 : 0);
  return min(max(e, -kKvExpLim), kKvExpLim);
}

// Grid: x over units, y = 2 * layer + (0: K, 1: V).
template <typename T, bool Q8>
__global__ void __launch_bounds__(kKvThreads) kv_write_kernel(const __grid_constant__ KvRowsDesc k,
                                                              const __grid_constant__ KvRowsLayers l) {
  pdl_wait();
  pdl_launch_dependents();
  KvUnit u(k);
  // (the count, the row's index and the position in one round trip)
  const int n = u.on ? (k.valid ? min(__ldg(k.valid + u.s), k.rows) : k.rows) : 0;
  const int src = u.on && k.row_index ? __ldg(k.row_index + u.m) : u.i;
  const int base = u.on ? __ldg(k.base_pos + u.s) : 0;
  u.on = u.on && u.i < n;
  if (u.on && (src < 0 || src >= k.rows)) {
    raise_status(k.status, ST_RANGE);
    u.on = false;
  }
  KvRow8<T> v[kKvHeads];
#pragma unroll
  for (int h = 0; h < kKvHeads; ++h) v[h].zero();
  if (u.on) {
    const T* p = reinterpret_cast<const T*>(u.is_v ? l.src_v[u.layer] : l.src_k[u.layer]) +
                 (((size_t)u.s * k.rows + src) * k.nkv + u.head) * k.d + u.e0;
#pragma unroll
    for (int h = 0; h < kKvHeads; ++h)
      if (h < u.heads) v[h].load(p + h * k.d);
  }
  size_t row = 0;
  uint32_t hr = 0;
  u.on = u.on && kv_row(k, l.pages[u.layer], u.s, base, u.i, n, &row, &hr);
  row += (size_t)u.head * hr;
  void* dst = u.is_v ? l.dst_v[u.layer] : l.dst_k[u.layer];
  if constexpr (!Q8) {
#pragma unroll
    for (int h = 0; h < kKvHeads; ++h, row += hr)
      if (u.on && h < u.heads) v[h].store(reinterpret_cast<T*>(dst) + row * k.d + u.e0);
  } else {
    uint32_t top[kKvHeads];
    uint32_t odd[kKvHeads];  // bit j: element j is NaN or infinite
#pragma unroll
    for (int h = 0; h < kKvHeads; ++h) {
      top[h] = v[h].top();
      odd[h] = 0u;
      if (top[h] >= KvRow8<T>::kInf) {
        top[h] = 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float a = fabsf(v[h].at(j));
          if (a < INFINITY) top[h] = max(top[h], __float_as_uint(a) >> (sizeof(T) == 2 ? 16 : 0));
          else odd[h] |= 1u << j;
        }
      }
    }
    // the maximum over a row's threads, a half or a quarter of a warp (two bf16 heads per shuffle)
    if constexpr (sizeof(T) == 2) {
      static_assert(kKvHeads % 2 == 0, "");
#pragma unroll
      for (int h = 0; h < kKvHeads; h += 2) {
        uint32_t m = top[h] | top[h + 1] << 16;
        for (int o = k.d >> 4; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
        top[h] = m & 0xFFFFu;
        top[h + 1] = m >> 16;
      }
    } else {
#pragma unroll
      for (int h = 0; h < kKvHeads; ++h)
        for (int o = k.d >> 4; o > 0; o >>= 1) top[h] = max(top[h], __shfl_xor_sync(0xffffffffu, top[h], o));
    }
    if (!u.on) return;
#pragma unroll
    for (int h = 0; h < kKvHeads; ++h, row += hr) {
      if (h >= u.heads) break;
      const int e = kv_exponent(KvRow8<T>::value(top[h]));
      const float inv = pow2_f(-e);
      uint32_t w[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const __nv_fp8x2_storage_t a = __nv_cvt_float2_to_fp8x2(
            make_float2(v[h].at(4 * q) * inv, v[h].at(4 * q + 1) * inv), __NV_SATFINITE, __NV_E4M3);
        const __nv_fp8x2_storage_t b = __nv_cvt_float2_to_fp8x2(
            make_float2(v[h].at(4 * q + 2) * inv, v[h].at(4 * q + 3) * inv), __NV_SATFINITE, __NV_E4M3);
        w[q] = (uint32_t)a | ((uint32_t)b << 16);
      }
      if (odd[h]) {
        raise_status(k.status, ST_NUMERIC);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if ((odd[h] >> j) & 1u) w[j >> 2] = (w[j >> 2] & ~(0xFFu << (8 * (j & 3)))) | (0x7Fu << (8 * (j & 3)));
      }
      *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(dst) + row * k.d + u.e0) = make_uint2(w[0], w[1]);
      if (u.e0 == 0) (u.is_v ? l.v_exp[u.layer] : l.k_exp[u.layer])[row] = (uint8_t)(e + kKvExpBias);
    }
  }
}

template <typename T, bool Q8>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const __grid_constant__ KvRowsDesc k,
                                                             const __grid_constant__ KvRowsLayers l) {
  pdl_wait();
  pdl_launch_dependents();
  const KvUnit u(k);
  if (!u.on) return;
  const int n = k.valid ? min(__ldg(k.valid + u.s), k.rows) : k.rows, base = __ldg(k.base_pos + u.s);
  if (u.i >= n) return;
  size_t row;
  uint32_t hr;
  if (!kv_row(k, l.pages[u.layer], u.s, base, u.i, 0, &row, &hr)) return;
  row += (size_t)u.head * hr;
  const void* src = u.is_v ? l.src_v[u.layer] : l.src_k[u.layer];
  T* out = reinterpret_cast<T*>(u.is_v ? l.dst_v[u.layer] : l.dst_k[u.layer]) +
           ((size_t)u.m * k.nkv + u.head) * k.d + u.e0;
  float v[kKvHeads][8];
  if constexpr (!Q8) {
#pragma unroll
    for (int h = 0; h < kKvHeads; ++h)
      if (h < u.heads) load8(reinterpret_cast<const T*>(src) + (row + (size_t)h * hr) * k.d + u.e0, v[h]);
  } else {
    const uint8_t* ex = u.is_v ? l.v_exp[u.layer] : l.k_exp[u.layer];
    uint2 c[kKvHeads];
    int e[kKvHeads];
#pragma unroll
    for (int h = 0; h < kKvHeads; ++h) {
      if (h < u.heads) {
        const size_t r = row + (size_t)h * hr;
        c[h] = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(src) + r * k.d + u.e0);
        e[h] = ex[r];
      }
    }
#pragma unroll
    for (int h = 0; h < kKvHeads; ++h) {
      if (h >= u.heads) break;
      const float sc = pow2_f(e[h] - kKvExpBias);
      const uint32_t w[2] = {c[h].x, c[h].y};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __half2_raw x =
            __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((w[j >> 1] >> (16 * (j & 1))) & 0xFFFFu), __NV_E4M3);
        const float2 f = __half22float2(__half2(x));
        v[h][2 * j] = f.x * sc;
        v[h][2 * j + 1] = f.y * sc;
      }
    }
  }
#pragma unroll
  for (int h = 0; h < kKvHeads; ++h)
    if (h < u.heads) store8(out + h * k.d, v[h]);
}

template <typename F>
static cudaError_t kv_launch(F kernel, const KvRowsDesc& k, const KvRowsLayers& l, cudaStream_t st) {
  const int upb = kKvThreads / (k.d / 8);
  const long long units = (long long)k.S * k.rows * ((k.nkv + kKvHeads - 1) / kKvHeads);
  const dim3 grid((unsigned)((units + upb - 1) / upb), 2 * k.n_layers);
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
