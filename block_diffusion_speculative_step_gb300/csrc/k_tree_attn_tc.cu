// k_tree_attn_tc.cu -- tree attention on the tcgen05 tensor cores (bf16
// queries; bf16 or 8-bit cache).
//
// Work: an item is (sequence, KV head, group of NT x 128 query vectors); its
// chunks are the 128-slot chunks of the context and, last, the tree's own
// rows.  The chunks of all items in a row are cut into equal runs, one per
// CTA (one CTA per SM), so every SM streams the same number of K/V bytes
// whatever the lengths.  A CTA walks its run as segments (the part of one
// item inside the run): a whole item is normalised and written at once, the
// first and the last segment may leave a partial (O, m, l) in the workspace
// that the merge kernel joins in order.
//
// Two streams per CTA, each an independent online softmax with its own
// score and output accumulators in tensor memory (S 128 + O D columns each):
// with NT = 2 stream t holds query tile t and takes every chunk; with NT = 1
// both hold the same tile and take chunks alternately, and are joined when
// the segment ends.  Per chunk and stream (128 query vectors x 128 keys):
//   S = Q K^T        tcgen05.mma, both operands in shared memory
//   P = 2^(c S - m)  one thread per query vector; written over S as 16-bit
//   O += P V         tcgen05.mma, P from tensor memory, V MN-major
// While one stream's softmax runs, the other stream's products do.  The
// reference maximum m moves only when a chunk exceeds it by more than 8 (a
// factor 256 in P), so O is rarely rescaled.
//
// P is rounded to 16 bits for its product: bf16 next to a bf16 V (2^-8
// relative per weight, as the output itself is rounded), fp16 with an 8-bit
// cache (2^-11).  The sum l uses the unrounded weights.
//
// 8-bit cache: K and V arrive as e4m3 codes (half the bytes), and four warps
// rewrite each tile as fp16 operands: code * 2^(e_row - E) with E the chunk's
// largest exponent, exact but for rows 2^-15 and more below it (whose low
// bits, 2^-24 of the chunk's largest element, go).  E of a K chunk joins the
// score scale; E of a V chunk joins the exponent of P.  The tree's bf16 rows
// and the queries become fp16 the same way (power-of-two scale per chunk /
// per query vector: bf16's 8 bits fit in fp16's 11).
//
// Bound by HBM (K/V bytes) up to 256 query vectors per KV head: per 128-key
// chunk an SM's share of the bandwidth takes 2.8k cycles in bf16 (1.4k in 8
// bits), the two products 1.0k per query tile.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "tc_ptx.cuh"
#include "tmap.h"
#include "tree_attn.cuh"

namespace dfl {

namespace {

constexpr int kTtCH = 128;      // keys per chunk
constexpr int kTtRows = 128;    // query vectors per tile
constexpr int kTtRing = 8;      // chunks whose scale exponents and bad rows are kept (roles run at most 4 apart)

struct TtTma {
  CUtensorMap kc, vc;  // cache rows [..][D]: bf16 boxes of 64 dims, or e4m3 boxes of D bytes, 128 rows
  CUtensorMap kb, vb;  // tree rows [M][nkv][D] (bf16 cache)
  TreeAttnDesc a;
  int n_pt;            // query tile groups per KV head
};

template <int D, int NT, bool Q8>
struct TtCfg {
  static constexpr int TILE = kTtCH * D * 2;                   // one 16-bit K or V tile
  static constexpr int RAW = kTtCH * D;                        // one e4m3 tile
  static constexpr int NSK = Q8 ? (NT == 2 ? 1 : 2) : (D == 64 ? 4 : (NT == 2 ? 2 : 3));
  static constexpr int NSV = Q8 ? 2 : (D == 64 ? 4 : 2);
  static constexpr int NRK = Q8 ? 2 : 0;                       // raw K / V slots
  static constexpr int NRV = Q8 ? 1 : 0;
  static constexpr int WARPS = Q8 ? 16 : 12;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int Q_OFF = 0;
  static constexpr int K_OFF = NT * TILE;
  static constexpr int V_OFF = K_OFF + NSK * TILE;
  static constexpr int R_OFF = V_OFF + NSV * TILE;             // raw K slots, raw V slots
  static constexpr int X_OFF = R_OFF + (NRK + NRV) * RAW;      // exchange, masks, barriers
  static constexpr int X_BYTES = 6144;
  static constexpr size_t SMEM = X_OFF + X_BYTES + 1024;
  static_assert(SMEM <= 232448, "shared memory of one CTA");
};

struct TtShared {  // after the tiles
  float xm[2][128], xl[2][128], xu[2][128];  // a segment's stream statistics (NT = 1): maximum, sum, unit of O
  int par[DFLASH_MAX_TREE];
  int ek[kTtRing], ev[kTtRing];   // chunk scale exponents (8-bit cache), by chunk counter
  uint32_t badv[kTtRing][4];      // tree rows whose V holds a NaN or infinity, by chunk counter
  float cmax[2][2][4];            // converters: the warps' maxima of the tree rows (K, V)
  int s0, it0, c0, len;           // the CTA's run: first item and chunk, number of chunks
  uint64_t kfull[4], kempty[4], vfull[4], vempty[4];
  uint64_t rkfull[2], rkempty[2], rvfull[2], rvempty[2];
  uint64_t sfull[2], pdone[2], ofull[2], qfull, qempty;
  uint32_t tslot;
  int abort;
  int8_t qe[4][2][128];           // query vectors' scale exponents (8-bit cache), by segment
};

// D[tmem] (+)= A[tmem] * B[smem]: A packed 16-bit, two per column, K along columns.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}

// kind::f16 with both operands fp16 (type code 0) instead of bf16 (1).
template <bool F16>
__host__ __device__ constexpr uint32_t tt_idesc(int M, int N, bool b_mn) {
  const uint32_t base = b_mn ? tc::idesc_bf16_f32_bmn(M, N) : tc::idesc_bf16_f32(M, N);
  return F16 ? base & ~((7u << 7) | (7u << 10)) : base;
}

// 32 packed columns of this thread's lane; returns once stored (one statement:
// the source registers are read until the wait).
__device__ __forceinline__ void tmem_st32u(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {"
      "%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ float tt_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool F16>
__device__ __forceinline__ uint32_t tt_pack(float lo, float hi) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// Byte offset of (row, 16-byte piece) in a 16-bit tile of 128 rows kept as
// 64-element boxes with the 128-byte swizzle.
__device__ __forceinline__ uint32_t tt_off(int row, int ch) {
  return (uint32_t)((ch >> 3) * (kTtCH * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
}

// A CTA's run walked segment by segment; every role keeps its own copy.
struct Seg {
  const TreeAttnDesc* a;
  int ips, left;       // items per sequence; chunks of the run not yet walked
  int s, it;           // sequence, item of the sequence
  int n_ctx, nch;      // context slots, chunks of the item (the last one the tree)
  int c0, c1;          // the segment's chunks
  __device__ __forceinline__ void load() {
    n_ctx = min(max(__ldg(a->base_pos + s), 0), a->max_pos);
    nch = (n_ctx + kTtCH - 1) / kTtCH + 1;
  }
  __device__ __forceinline__ bool begin(const TreeAttnDesc* d, int ips_, const TtShared* sh) {
    a = d;
    ips = ips_;
    left = sh->len;
    if (left <= 0) return false;
    s = sh->s0;
    it = sh->it0;
    load();
    c0 = sh->c0;
    c1 = min(nch, c0 + left);
    return true;
  }
  __device__ __forceinline__ bool next() {
    left -= c1 - c0;
    if (left <= 0) return false;
    if (++it == ips) {
      it = 0;
      ++s;
      load();
    }
    c0 = 0;
    c1 = min(nch, left);
    return true;
  }
  __device__ __forceinline__ bool is_tree(int c) const { return c == nch - 1; }
  __device__ __forceinline__ int keys(int c) const { return is_tree(c) ? a->rows : min(kTtCH, n_ctx - c * kTtCH); }
};

// The run of CTA b among nb: chunks [b * per, (b + 1) * per) of all items'
// chunks, per = ceil(total / nb).  One warp; sequences are scanned 32 at a time.
__device__ __forceinline__ long long tt_total(const TreeAttnDesc& a, int ips) {
  const int lane = threadIdx.x & 31;
  long long t = 0;
  for (int s = lane; s < a.n_seqs; s += 32) {
    const int n = min(max(__ldg(a.base_pos + s), 0), a.max_pos);
    t += (long long)((n + kTtCH - 1) / kTtCH + 1) * ips;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  return t;
}

// First chunk of sequence s in that order.
__device__ __forceinline__ void tt_locate(const TreeAttnDesc& a, int ips, long long x, int* s_out, int* it_out,
                                          int* c_out) {
  const int lane = threadIdx.x & 31;
  long long before = 0;
  for (int b = 0; b < a.n_seqs; b += 32) {
    const int s = b + lane;
    const int n = s < a.n_seqs ? min(max(__ldg(a.base_pos + s), 0), a.max_pos) : 0;
    const int nch = s < a.n_seqs ? (n + kTtCH - 1) / kTtCH + 1 : 0;
    long long inc = (long long)nch * ips;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + inc > x);
    if (hit) {
      const int w = __ffs(hit) - 1;
      const long long start = before + __shfl_sync(0xffffffffu, inc, w) - (long long)__shfl_sync(0xffffffffu, nch, w) * ips;
      const int k = __shfl_sync(0xffffffffu, nch, w);
      *s_out = b + w;
      *it_out = (int)((x - start) / k);
      *c_out = (int)((x - start) % k);
      return;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  *s_out = a.n_seqs;
  *it_out = *c_out = 0;
}

// Scale 2^d as fp16 (d <= 0; 0 below the subnormals).
__device__ __forceinline__ __half2 tt_half_pow2(int d) {
  const uint32_t h = d >= -14 ? (uint32_t)(15 + d) << 10 : d >= -24 ? 1u << (24 + d) : 0u;
  const uint32_t w = h | (h << 16);
  return *reinterpret_cast<const __half2*>(&w);
}

// Exponent e with |x| * 2^-e <= 2^8 for |x| up to mx, at least -120.
__device__ __forceinline__ int tt_exp_of(float mx) {
  if (!(mx > 0.f)) return -120;
  int k;
  frexpf(mx, &k);
  return max(k - 8, -120);
}

// x * 2^e for |e| <= 250 (two factors: one alone may leave the fp32 range).
__device__ __forceinline__ float tt_scale(float x, int e) {
  const int h = e / 2;
  return x * __int_as_float((127 + h) << 23) * __int_as_float((127 + (e - h)) << 23);
}

__device__ __forceinline__ float tt_finite_max(const float (&v)[8]) {
  float mx = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(v[e]) < INFINITY ? fabsf(v[e]) : 0.f);
  return mx;
}

// Eight elements scaled by 2^-e to fp16.
__device__ __forceinline__ uint4 tt_to_half(const float (&v)[8], int e) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = tt_pack<true>(tt_scale(v[2 * i], -e), tt_scale(v[2 * i + 1], -e));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 e4m3 codes times f -> 16 fp16 values (two 16-byte pieces).
__device__ __forceinline__ void tt_codes_to_half(const uint4& c, __half2 f, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu), __NV_E4M3);
    const __half2 m = __hmul2(__half2(h), f);
    o[i] = *reinterpret_cast<const uint32_t*>(&m);
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// Where a segment's partial lies: slot 0 of CTA b when the item began in an
// earlier CTA, slot 1 when it ends in a later one.  A slot holds D / 4 column
// groups of [128 rows] float4 per tile, then maxima and sums: a warp's 32
// rows are 512 contiguous bytes on both sides.
template <int D, int NT>
__host__ __device__ constexpr size_t tt_slot_floats() {
  return (size_t)NT * kTtRows * (D + 2);
}

template <int D, int NT, bool Q8>
__global__ void __launch_bounds__(TtCfg<D, NT, Q8>::THREADS, 1) tree_tc_kernel(const __grid_constant__ TtTma p) {
  using Cfg = TtCfg<D, NT, Q8>;
  constexpr int TILE = Cfg::TILE, RAW = Cfg::RAW, NSK = Cfg::NSK, NSV = Cfg::NSV;
  extern __shared__ __align__(1024) uint8_t tt_smem[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(tt_smem) + 1023) & ~uintptr_t(1023));
  uint8_t* Qs = sm + Cfg::Q_OFF;
  uint8_t* Ks = sm + Cfg::K_OFF;
  uint8_t* Vs = sm + Cfg::V_OFF;
  uint8_t* Rk = sm + Cfg::R_OFF;
  uint8_t* Rv = Rk + Cfg::NRK * RAW;
  TtShared* sh = reinterpret_cast<TtShared*>(sm + Cfg::X_OFF);
  static_assert(sizeof(TtShared) <= Cfg::X_BYTES, "exchange area");
  volatile int* abort = &sh->abort;

  const TreeAttnDesc& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int grp = a.nq / a.nkv, nqv = a.rows * grp, QD = a.nq * D;
  const int ips = a.nkv * p.n_pt;
  uint32_t* status = a.status;

  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(&sh->kfull[i], Q8 ? 128 : 1);
      tc::mbar_init(&sh->kempty[i], 1);
      tc::mbar_init(&sh->vfull[i], Q8 ? 128 : 1);
      tc::mbar_init(&sh->vempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sh->rkfull[i], 1);
      tc::mbar_init(&sh->rkempty[i], 128);
      tc::mbar_init(&sh->rvfull[i], 1);
      tc::mbar_init(&sh->rvempty[i], 128);
      // the product's commit, and the issuer's own arrival: what the issuer has
      // observed (scale exponents, bad rows) is visible to who waits here
      tc::mbar_init(&sh->sfull[i], 2);
      tc::mbar_init(&sh->pdone[i], 128);
      tc::mbar_init(&sh->ofull[i], 2);
    }
    tc::mbar_init(&sh->qfull, 64);
    tc::mbar_init(&sh->qempty, 1);
    sh->abort = 0;
    tc::fence_mbar_init();
    tc::tma_prefetch_desc(&p.kc);
    tc::tma_prefetch_desc(&p.vc);
  }
  if (warp == 1) tc::tmem_alloc(&sh->tslot, 512);
  pdl_wait();
  pdl_launch_dependents();
  if (warp == 0) {
    const long long total = tt_total(a, ips);
    const long long per = (total + gridDim.x - 1) / gridDim.x;
    const long long x0 = (long long)blockIdx.x * per;
    int s0 = 0, it0 = 0, c0 = 0;
    if (x0 < total) tt_locate(a, ips, x0, &s0, &it0, &c0);
    if (lane == 0) {
      sh->s0 = s0;
      sh->it0 = it0;
      sh->c0 = c0;
      sh->len = x0 < total ? (int)min(per, total - x0) : 0;
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = sh->tslot;
  const uint64_t lim_ns = wait_limit_ns(status);
  const bool stall = stall_kv_loads(status);  // test switch: issue no K/V copy
  const KvMap km{a.pages, a.cap, a.ps, a.max_pages, a.pool, a.nkv};
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t par) {
    if (ok && !tc::mbar_wait(bar, par & 1u, abort, lim_ns)) {
      raise_status(status, ST_TIMEOUT);
      *abort = 1;
      ok = false;
    }
    return ok;
  };
  // The same for a whole warp (its lanes go on together: what follows shuffles).
  auto wait_warp = [&](uint64_t* bar, uint32_t par) {
    wait(bar, par);
    ok = __all_sync(0xffffffffu, ok);
    return ok;
  };
  Seg sg;

  if (warp == 0) {
    // ---------------------------------------------------- K/V copies
    if (lane == 0 && !stall) {
      int nk = 0, nv = 0;  // copies issued
      constexpr int SK = Q8 ? Cfg::NRK : NSK, SV = Q8 ? Cfg::NRV : NSV;
      uint64_t* kf = Q8 ? sh->rkfull : sh->kfull;
      uint64_t* ke = Q8 ? sh->rkempty : sh->kempty;
      uint64_t* vf = Q8 ? sh->rvfull : sh->vfull;
      uint64_t* ve = Q8 ? sh->rvempty : sh->vempty;
      const uint64_t pol = tc::policy_evict_first();
      for (bool on = sg.begin(&a, ips, sh); on && ok; on = sg.next()) {
        const int g = sg.it / p.n_pt;
        for (int c = sg.c0; c < sg.c1 && ok; ++c) {
          const bool tree = sg.is_tree(c);
          if (Q8 && tree) continue;  // the converters read the tree's rows themselves
          int row = 0;
          if (!tree) {
            bool bad = false;
            row = (int)(km.row0(sg.s, c * kTtCH, &bad) + (uint32_t)g * (uint32_t)km.head_rows());
            if (bad) raise_status(status, ST_RANGE);  // reads page 0 instead
          }
          if (nk >= SK && !wait(&ke[nk % SK], (uint32_t)(nk / SK - 1))) break;
          if constexpr (Q8) {
            tc::mbar_arrive_expect_tx(&kf[nk % SK], RAW);
            tc::tma_load_2d(Rk + (nk % SK) * RAW, &p.kc, 0, row, &kf[nk % SK], pol);
          } else {
            tc::mbar_arrive_expect_tx(&kf[nk % SK], TILE);
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
              uint8_t* dst = Ks + (nk % SK) * TILE + h * (kTtCH * 128);
              if (tree) tc::tma_load_3d(dst, &p.kb, 64 * h, g, sg.s * a.rows, &kf[nk % SK]);
              else tc::tma_load_2d(dst, &p.kc, 64 * h, row, &kf[nk % SK], pol);
            }
          }
          ++nk;
          if (nv >= SV && !wait(&ve[nv % SV], (uint32_t)(nv / SV - 1))) break;
          if constexpr (Q8) {
            tc::mbar_arrive_expect_tx(&vf[nv % SV], RAW);
            tc::tma_load_2d(Rv + (nv % SV) * RAW, &p.vc, 0, row, &vf[nv % SV], pol);
          } else {
            tc::mbar_arrive_expect_tx(&vf[nv % SV], TILE);
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
              uint8_t* dst = Vs + (nv % SV) * TILE + h * (kTtCH * 128);
              if (tree) tc::tma_load_3d(dst, &p.vb, 64 * h, g, sg.s * a.rows, &vf[nv % SV]);
              else tc::tma_load_2d(dst, &p.vc, 64 * h, row, &vf[nv % SV], pol);
            }
          }
          ++nv;
        }
      }
      // every copy has landed before the CTA's shared memory goes away
      for (int i = max(0, nk - SK); i < nk; ++i) tc::mbar_wait(&kf[i % SK], (uint32_t)(i / SK) & 1u, nullptr, lim_ns);
      for (int i = max(0, nv - SV); i < nv; ++i) tc::mbar_wait(&vf[i % SV], (uint32_t)(i / SV) & 1u, nullptr, lim_ns);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------- MMA issue
    if (lane == 0) {
      constexpr uint32_t idS = tt_idesc<Q8>(kTtRows, kTtCH, false);
      constexpr uint32_t idV = tt_idesc<Q8>(kTtRows, D, true);
      const uint32_t qb = tc::smem_u32(Qs), kb = tc::smem_u32(Ks), vb = tc::smem_u32(Vs);
      // Jobs in order: (chunk, stream); stream = job & 1.  S of job j + 2 is
      // issued after P V of job j, whose P lies in the same columns.
      Seg ss;               // the S side's segment
      int sj = 0, sc = 0;   // next S job, its chunk counter
      int c = 0, seg_no = 0;
      bool s_on = ss.begin(&a, ips, sh);
      if (s_on) c = ss.c0;
      auto issue_s = [&]() {  // S of job sj
        const int t = sj & 1, slot = sc % NSK;
        if (c == ss.c0 && (NT == 1 || t == 0) && !wait(&sh->qfull, (uint32_t)seg_no)) return;
        if ((NT == 1 || t == 0) && !wait(&sh->kfull[slot], (uint32_t)(sc / NSK))) return;
        tc::tc_fence_after();
        const uint32_t q = qb + (NT == 2 ? t * TILE : 0), k = kb + slot * TILE;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          const uint32_t off = (uint32_t)((j >> 2) * (kTtCH * 128) + (j & 3) * 32);
          tc::mma_bf16(tmem + t * 128, tc::sdesc_sw128(q + off), tc::sdesc_sw128(k + off), idS, j > 0 ? 1u : 0u);
        }
        tc::mma_commit(&sh->sfull[t]);
        tc::mbar_arrive(&sh->sfull[t]);
        ++sj;
        if (NT == 2 && t == 0) return;
        tc::mma_commit(&sh->kempty[slot]);
        ++sc;
        if (++c == ss.c1) {
          tc::mma_commit(&sh->qempty);
          ++seg_no;
          s_on = ss.next();
          c = ss.c0;
        }
      };
      for (int i = 0; i < 2 && s_on && ok; ++i) issue_s();
      int vc = 0, vj = 0;
      for (bool on = sg.begin(&a, ips, sh); on && ok; on = sg.next()) {
        bool fresh[2] = {true, true};  // the stream's next P V starts its accumulator
        for (int x = sg.c0; x < sg.c1 && ok; ++x, ++vc) {
          const int slot = vc % NSV;
#pragma unroll
          for (int u = 0; u < NT; ++u, ++vj) {
            const int t = vj & 1;
            if (!wait(&sh->pdone[t], (uint32_t)(vj >> 1))) break;
            if (u == 0 && !wait(&sh->vfull[slot], (uint32_t)(vc / NSV))) break;
            tc::tc_fence_after();
#pragma unroll
            for (int j = 0; j < kTtCH / 16; ++j)
              mma_ts(tmem + 256 + t * 128, tmem + t * 128 + 8 * j,
                     tc::sdesc_sw128_mn(vb + slot * TILE + (uint32_t)j * 2048u, kTtCH * 128, 1024), idV,
                     (!fresh[t] || j > 0) ? 1u : 0u);
            fresh[t] = false;
            if (u == NT - 1) tc::mma_commit(&sh->vempty[slot]);
            // the stream's last job of the segment: its output is complete
            if (NT == 2 ? x == sg.c1 - 1 : x >= sg.c1 - 2) {
              tc::mma_commit(&sh->ofull[t]);
              tc::mbar_arrive(&sh->ofull[t]);
            }
            if (s_on) issue_s();
          }
        }
      }
    }
  } else if (warp < 4) {
    // ---------------------------------------------------- queries
    const int qt = tid - 64;
    int seg_no = 0;
    for (bool on = sg.begin(&a, ips, sh); on && ok; on = sg.next(), ++seg_no) {
      const int g = sg.it / p.n_pt, qv0 = (sg.it % p.n_pt) * (NT * kTtRows);
      if (seg_no > 0 && !wait_warp(&sh->qempty, (uint32_t)(seg_no - 1))) break;
      constexpr int CPR = D / 8;
      for (int i = qt; i < NT * kTtRows * CPR; i += 64) {
        const int r = i / CPR, ch = i % CPR, qv = qv0 + r;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (qv < nqv) {
          const int row = qv / grp, head = g * grp + qv % grp;
          w = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.q) +
                                                   ((size_t)sg.s * a.rows + row) * QD + (size_t)head * D) + ch);
        }
        if constexpr (Q8) {
          float v[8];
          const __nv_bfloat162* b2 = reinterpret_cast<const __nv_bfloat162*>(&w);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = __bfloat1622float2(b2[e]);
            v[2 * e] = f.x;
            v[2 * e + 1] = f.y;
          }
          float mx = tt_finite_max(v);
#pragma unroll
          for (int o = CPR / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          const int e = tt_exp_of(mx);
          w = tt_to_half(v, e);
          if (ch == 0) sh->qe[seg_no & 3][r >> 7][r & 127] = (int8_t)e;
        }
        *reinterpret_cast<uint4*>(Qs + (r >> 7) * TILE + tt_off(r & 127, ch)) = w;
      }
      tc::fence_proxy_async_smem();
      tc::mbar_arrive(&sh->qfull);
    }
  } else if (warp < 12) {
    // ---------------------------------------------------- softmax: stream t, one query vector per thread
    const int t = (warp - 4) >> 2;
    const int r = (warp & 3) * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t ts = lane_base + t * 128, to = lane_base + 256 + t * 128;
    int nj = 0;         // jobs this stream has done
    int cc = 0;         // chunk counter
    int no[2] = {0, 0}; // segments in which each stream had a job
    int seg_no = 0;
    for (bool on = sg.begin(&a, ips, sh); on; on = sg.next(), ++seg_no) {
      const int g = sg.it / p.n_pt, qv0 = (sg.it % p.n_pt) * (NT * kTtRows);
      const int qv = qv0 + (NT == 2 ? t * kTtRows : 0) + r;
      const bool has_row = qv < nqv;
      const bool warp_on = __any_sync(0xffffffffu, has_row);
      const int node = has_row ? qv / grp : 0;
      const bool has_tree = sg.c1 == sg.nch;  // the segment ends with the tree's rows
      const int tree_ring = (cc + sg.c1 - 1 - sg.c0) % kTtRing;
      float m_run = -INFINITY, l_run = 0.f;
      int e_run = 0;      // O is kept in units of 2^e_run (8-bit cache)
      const int nj0 = nj;
      bool row_ok = true;
      uint32_t tm[4] = {0u, 0u, 0u, 0u};
      if (has_tree) {
        tc::named_bar(4, 256);  // the parents of the item before have been read
        if (t == 0 && a.parent && r < a.rows) sh->par[r] = __ldg(a.parent + (size_t)sg.s * a.rows + r);
        if (!Q8 && t == 0 && r < 4) sh->badv[tree_ring][r] = 0u;
        tc::named_bar(4, 256);
        bool bad = false;
        row_ok = has_row && tree_row_mask(a.parent ? sh->par : nullptr, node, tm, &bad);
        if (bad) raise_status(status, ST_RANGE);
      }
      for (int c = sg.c0; c < sg.c1; ++c, ++cc) {
        if (NT == 1 && (cc & 1) != t) continue;
        const bool tree = sg.is_tree(c);
        const int nk = sg.keys(c);
        const bool masked = tree || nk < kTtCH;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = nk - 32 * i;
          w[i] = n >= 32 ? 0xffffffffu : n > 0 ? (1u << n) - 1u : 0u;
          if (tree) w[i] &= row_ok ? tm[i] : 0u;
        }
        if constexpr (!Q8) {
          // Values of slots past the last key may be anything (unwritten
          // cache rows); a hidden tree row's may too.  0 * NaN is NaN, so
          // such rows are cleared before the product (NT = 2: by stream 0,
          // whose product comes first); of the tree's rows only NaN and
          // infinite elements, which the segment's end adds to who sees them.
          if (masked && (NT == 1 || t == 0)) {
            const int slot = cc % NSV;
            uint8_t* vt = Vs + slot * TILE;
            if (wait(&sh->vfull[slot], (uint32_t)(cc / NSV))) {
              for (int i = r; i < kTtCH * (D / 8); i += 128) {
                const int j = i / (D / 8), ch = i % (D / 8);
                uint4* q = reinterpret_cast<uint4*>(vt + tt_off(j, ch));
                if (j >= nk) {
                  *q = make_uint4(0, 0, 0, 0);
                } else if (tree) {
                  uint4 v = *q;
                  uint32_t e[4] = {v.x, v.y, v.z, v.w};
                  bool odd = false;
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    if ((e[k] & 0x7F80u) == 0x7F80u) { e[k] &= 0xFFFF0000u; odd = true; }
                    if ((e[k] & 0x7F800000u) == 0x7F800000u) { e[k] &= 0xFFFFu; odd = true; }
                  }
                  if (odd) {
                    *q = make_uint4(e[0], e[1], e[2], e[3]);
                    atomicOr(&sh->badv[tree_ring][j >> 5], 1u << (j & 31));
                  }
                }
              }
            }
          }
        }
        wait(&sh->sfull[t], (uint32_t)nj);
        __syncwarp();
        tc::tc_fence_after();
        if (warp_on) {
          float cs = a.scale;  // score scale (log2 units)
          int dv = 0;          // exponent of the chunk's V against O's unit
          int up = 0;          // how far O's unit moves first
          if constexpr (Q8) {
            cs = tt_scale(a.scale, sh->ek[cc % kTtRing] + sh->qe[seg_no & 3][NT == 2 ? t : 0][r]);
            const int ev = sh->ev[cc % kTtRing];
            if (nj == nj0) e_run = ev;
            dv = ev - e_run;
            if (dv > 6) {  // P reaches 2^(8 + dv): fp16 holds 2^15
              up = dv;
              e_run = ev;
              dv = 0;
            }
          }
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float x[32];
            tc::tmem_ld32(ts + 32 * i, x);
            if (masked) {
#pragma unroll
              for (int k = 0; k < 32; ++k) x[k] = (w[i] >> k) & 1u ? x[k] : -INFINITY;
            }
#pragma unroll
            for (int k = 0; k < 32; ++k) m4[k & 3] = fmaxf(m4[k & 3], x[k]);
          }
          const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * cs;
          const float m_new = (m_run == -INFINITY || mx > m_run + 8.f) ? fmaxf(mx, m_run) : m_run;
          const float alpha = m_run == -INFINITY ? 0.f : tt_ex2(m_run - m_new);
          // O holds the stream's chunks before this one: their products
          // precede this chunk's S in the tensor pipe, so they are complete.
          const float beta = up ? tt_scale(alpha, -up) : alpha;
          if (nj > nj0 && __any_sync(0xffffffffu, beta != 1.f)) {
#pragma unroll
            for (int q = 0; q < D / 16; ++q) {
              float o[16];
              tc::tmem_ld16(to + 16 * q, o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] *= beta;
              tc::tmem_st16(to + 16 * q, o);
            }
          }
          const float sub = m_new == -INFINITY ? 0.f : (float)dv - m_new;
          float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t pk[32];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float x[32];
              tc::tmem_ld32(ts + 64 * h + 32 * i, x);
              if (masked) {
#pragma unroll
                for (int k = 0; k < 32; ++k) x[k] = (w[2 * h + i] >> k) & 1u ? x[k] : -INFINITY;
              }
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                x[k] = tt_ex2(fmaf(x[k], cs, sub));
                s4[k & 3] += x[k];
              }
#pragma unroll
              for (int k = 0; k < 16; ++k) pk[16 * i + k] = tt_pack<Q8>(x[2 * k], x[2 * k + 1]);
            }
            tmem_st32u(ts + 32 * h, pk);  // over the scores just read
          }
          float sum = (s4[0] + s4[1]) + (s4[2] + s4[3]);
          if constexpr (Q8) sum = tt_scale(sum, -dv);
          l_run = fmaf(l_run, alpha, sum);
          m_run = m_new;
        }
        tc::fence_proxy_async_smem();
        tc::tc_fence_before();
        tc::mbar_arrive(&sh->pdone[t]);
        ++nj;
      }

      // ---- the segment's end: normalise and write, or leave a partial
      bool had[2];  // streams with a job in this segment
      had[t] = nj > nj0;
      had[t ^ 1] = NT == 2 ? false : (sg.c1 - sg.c0) > (nj - nj0);
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (had[u]) wait(&sh->ofull[u], (uint32_t)no[u]++);
      __syncwarp();
      tc::tc_fence_after();
      float M = m_run, L = l_run, f_own = Q8 ? tt_scale(1.f, e_run) : 1.f, f_oth = 0.f;
      if constexpr (NT == 1) {
        sh->xm[t][r] = m_run;
        sh->xl[t][r] = l_run;
        sh->xu[t][r] = f_own;
        tc::named_bar(4, 256);
        const float mo = sh->xm[t ^ 1][r];
        M = fmaxf(m_run, mo);
        const float ao = mo == -INFINITY ? 0.f : tt_ex2(mo - M), as = m_run == -INFINITY ? 0.f : tt_ex2(m_run - M);
        // (both streams' threads form the same sum: stream 0's term first)
        const float t0 = t == 0 ? l_run * as : sh->xl[0][r] * ao, t1 = t == 0 ? sh->xl[1][r] * ao : l_run * as;
        L = t0 + t1;
        f_own *= as;
        f_oth = ao * sh->xu[t ^ 1][r];
      }
      if (warp_on) {
        const bool whole = sg.c0 == 0 && has_tree;
        const float inv = whole ? (L > 0.f ? 1.f / L : L == L ? 0.f : L) : 1.f;
        f_own *= inv;
        f_oth *= inv;
        uint32_t bad[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) bad[i] = has_tree ? tm[i] & sh->badv[tree_ring][i] : 0u;
        const bool any_bad = (bad[0] | bad[1] | bad[2] | bad[3]) != 0u;
        constexpr int NCOL = NT == 1 ? D / 2 : D;       // columns this thread writes
        const int col0 = NT == 1 ? t * NCOL : 0;
        const uint32_t o_own = to, o_oth = lane_base + 256 + (t ^ 1) * 128;
        float* part = static_cast<float*>(a.work) +
                      ((size_t)2 * blockIdx.x + (sg.c0 > 0 ? 0 : 1)) * tt_slot_floats<D, NT>();
        const int prow = (NT == 2 ? t * kTtRows : 0) + r;
        __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(a.out) + ((size_t)sg.s * a.rows + node) * QD +
                             (size_t)(g * grp + (has_row ? qv % grp : 0)) * D;
#pragma unroll
        for (int q = 0; q < NCOL / 16; ++q) {
          const int col = col0 + 16 * q;
          float o[16], x[16];
          __syncwarp();  // the loads below are warp-collective
          if (had[t]) {
            tc::tmem_ld16(o_own + col, o);
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = 0.f;
          }
          if (NT == 1 && had[t ^ 1]) {
            tc::tmem_ld16(o_oth + col, x);
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) x[k] = 0.f;
          }
          // (stream 0's term first whichever thread adds them)
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = t == 0 ? fmaf(o[k], f_own, x[k] * f_oth) : fmaf(x[k], f_oth, o[k] * f_own);
          if (any_bad) {  // visible NaN or infinite values: added as they are
            for (int i = 0; i < 4; ++i)
              for (uint32_t b = bad[i]; b; b &= b - 1) {
                const int j = 32 * i + __ffs(b) - 1;
                const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(a.vb) +
                                         (((size_t)sg.s * a.rows + j) * a.nkv + g) * D + col;
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                  const float f = __bfloat162float(v[k]);
                  if (!(fabsf(f) < INFINITY)) o[k] += f;
                }
              }
          }
          if (whole) {
            if (row_ok && has_row && DFL_CHECK(node < a.rows, status)) {
              uint4* d4 = reinterpret_cast<uint4*>(dst + col);
              d4[0] = make_uint4(tt_pack<false>(o[0], o[1]), tt_pack<false>(o[2], o[3]), tt_pack<false>(o[4], o[5]),
                                 tt_pack<false>(o[6], o[7]));
              d4[1] = make_uint4(tt_pack<false>(o[8], o[9]), tt_pack<false>(o[10], o[11]),
                                 tt_pack<false>(o[12], o[13]), tt_pack<false>(o[14], o[15]));
            }
          } else if (has_row) {
            float4* p4 = reinterpret_cast<float4*>(part) + (size_t)(prow >> 7) * (kTtRows * D / 4);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              p4[(size_t)(col / 4 + k) * kTtRows + (prow & 127)] =
                  make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
        }
        if (!whole && has_row && (NT == 2 || t == 0)) {
          float* ml = part + (size_t)NT * kTtRows * D;
          ml[prow] = M;
          ml[NT * kTtRows + prow] = row_ok ? L : -1.f;
        }
      }
      if constexpr (NT == 1) tc::named_bar(4, 256);  // both outputs read before either stream goes on
    }
  } else {
    // ---------------------------------------------------- 8-bit cache: tiles to fp16 operands
    if constexpr (Q8) {
      const int ct = tid - 384, cw = warp - 12;
      constexpr int LPR = D / 16;       // lanes per code row (16 codes each)
      constexpr int RPP = 128 / LPR;    // rows per pass
      constexpr int NP = 128 / RPP;     // passes
      int i = 0, nr = 0;                // chunks, raw chunks
      // (after a wait gave up the loops run on without work, to meet the barrier)
      for (bool on = sg.begin(&a, ips, sh); on; on = sg.next()) {
        const int g = sg.it / p.n_pt;
        int e_top = -1000;              // largest V exponent of the segment so far
        for (int c = sg.c0; c < sg.c1; ++c, ++i) {
          const bool tree = sg.is_tree(c);
          const int nk = sg.keys(c);
          const int ks = i % NSK, vs = i % NSV;
          uint8_t *kt = Ks + ks * TILE, *vt = Vs + vs * TILE;
          if (!tree) {
            bool badp = false;
            const size_t row0 = (size_t)km.row0(sg.s, c * kTtCH, &badp) + (size_t)g * km.head_rows();
            int ek4[4], ev4[4];  // rows lane + 32 j
            int ekm = -1000, evm = -1000;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int r = lane + 32 * j;
              ek4[j] = r < nk ? (int)__ldg(a.k_exp + row0 + r) - 127 : -1000;
              ev4[j] = r < nk ? (int)__ldg(a.v_exp + row0 + r) - 127 : -1000;
              ekm = max(ekm, ek4[j]);
              evm = max(evm, ev4[j]);
            }
            ekm = __reduce_max_sync(0xffffffffu, ekm);
            evm = max(__reduce_max_sync(0xffffffffu, evm), e_top - 30);
            e_top = max(e_top, evm);
            if (ct == 0) {
              sh->ek[i % kTtRing] = ekm;
              sh->ev[i % kTtRing] = evm;
            }
#pragma unroll
            for (int v = 0; v < 2; ++v) {  // K, then V
              constexpr int NRK = Cfg::NRK, NRV = Cfg::NRV;
              const int rs = v ? nr % NRV : nr % NRK, rn = v ? nr / NRV : nr / NRK;
              const uint8_t* raw = (v ? Rv : Rk) + rs * RAW;
              uint8_t* dstt = v ? vt : kt;
              if (v ? i >= NSV && !wait_warp(&sh->vempty[vs], (uint32_t)(i / NSV - 1))
                    : i >= NSK && !wait_warp(&sh->kempty[ks], (uint32_t)(i / NSK - 1)))
                continue;
              if (!wait_warp(v ? &sh->rvfull[rs] : &sh->rkfull[rs], (uint32_t)rn)) continue;
#pragma unroll
              for (int ps = 0; ps < NP; ++ps) {
                const int r = ps * RPP + ct / LPR, pc = ct % LPR;
                const int e = __shfl_sync(0xffffffffu, v ? ev4[ps * RPP / 32] : ek4[ps * RPP / 32], r & 31);
                uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
                if (r < nk) {
                  const uint4 code = *reinterpret_cast<const uint4*>(raw + r * D + pc * 16);
                  tt_codes_to_half(code, tt_half_pow2(e - (v ? evm : ekm)), lo, hi);
                }
                *reinterpret_cast<uint4*>(dstt + tt_off(r, 2 * pc)) = lo;
                *reinterpret_cast<uint4*>(dstt + tt_off(r, 2 * pc + 1)) = hi;
              }
              tc::fence_proxy_async_smem();
              tc::mbar_arrive(v ? &sh->vfull[vs] : &sh->kfull[ks]);
              tc::mbar_arrive(v ? &sh->rvempty[rs] : &sh->rkempty[rs]);
            }
            ++nr;
          } else {
            // the tree's bf16 rows: one scale per chunk from their largest finite element
            constexpr int CPR = D / 8;
            const size_t base = ((size_t)sg.s * a.rows * a.nkv + g) * D;
            const size_t rstr = (size_t)a.nkv * D;
            const __nv_bfloat16* kb = reinterpret_cast<const __nv_bfloat16*>(a.kb) + base;
            const __nv_bfloat16* vb = reinterpret_cast<const __nv_bfloat16*>(a.vb) + base;
            float mk = 0.f, mv = 0.f;
            for (int q = ct; q < nk * CPR; q += 128) {
              float x[8];
              load8(kb + (q / CPR) * rstr + (q % CPR) * 8, x);
              mk = fmaxf(mk, tt_finite_max(x));
              load8(vb + (q / CPR) * rstr + (q % CPR) * 8, x);
              mv = fmaxf(mv, tt_finite_max(x));
            }
            mk = warp_max(mk);
            mv = warp_max(mv);
            float(*cm)[4] = sh->cmax[i & 1];
            if (lane == 0) {
              cm[0][cw] = mk;
              cm[1][cw] = mv;
            }
            if (ct < 4) sh->badv[i % kTtRing][ct] = 0u;
            tc::named_bar(5, 128);
            mk = fmaxf(fmaxf(cm[0][0], cm[0][1]), fmaxf(cm[0][2], cm[0][3]));
            mv = fmaxf(fmaxf(cm[1][0], cm[1][1]), fmaxf(cm[1][2], cm[1][3]));
            const int ekm = tt_exp_of(mk);
            const int evm = max(tt_exp_of(mv), e_top - 30);
            if (ct == 0) {
              sh->ek[i % kTtRing] = ekm;
              sh->ev[i % kTtRing] = evm;
            }
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              if (v ? i >= NSV && !wait_warp(&sh->vempty[vs], (uint32_t)(i / NSV - 1))
                    : i >= NSK && !wait_warp(&sh->kempty[ks], (uint32_t)(i / NSK - 1)))
                continue;
              for (int q = ct; q < kTtCH * CPR; q += 128) {
                const int r = q / CPR, ch = q % CPR;
                uint4 o = make_uint4(0, 0, 0, 0);
                if (r < nk) {
                  float x[8];
                  load8((v ? vb : kb) + r * rstr + ch * 8, x);
                  if (v) {  // a NaN or infinity must not meet a hidden row's weight 0
                    bool odd = false;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                      if (!(fabsf(x[e]) < INFINITY)) {
                        x[e] = 0.f;
                        odd = true;
                      }
                    if (odd) atomicOr(&sh->badv[i % kTtRing][r >> 5], 1u << (r & 31));
                  }
                  o = tt_to_half(x, v ? evm : ekm);
                }
                *reinterpret_cast<uint4*>((v ? vt : kt) + tt_off(r, ch)) = o;
              }
              tc::fence_proxy_async_smem();
              tc::mbar_arrive(v ? &sh->vfull[vs] : &sh->kfull[ks]);
            }
          }
        }
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

// Joins the partials of the items that several CTAs shared.  One warp per
// (item, tile, 32 rows, 16 columns): lanes are rows, so the partials' reads are
// 512 contiguous bytes; items of one CTA return at once.
template <int D, int NT>
__global__ void __launch_bounds__(128) tree_tc_merge_kernel(const __grid_constant__ TreeAttnDesc a, int n_pt, int nb) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int ips = a.nkv * n_pt, grp = a.nq / a.nkv, nqv = a.rows * grp;
  constexpr int RG = NT * 4, CG = D / 16;  // row groups, column groups of an item
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (w >= (long long)a.n_seqs * ips * RG * CG) return;
  const int cg = (int)(w % CG), rg = (int)(w / CG % RG);
  const int it = (int)(w / CG / RG % ips), s = (int)(w / CG / RG / ips);
  const int g = it / n_pt, qv = (it % n_pt) * (NT * kTtRows) + rg * 32 + lane;
  if (qv - lane >= nqv) return;
  // the item's chunks [X, X + nch) among all chunks, and the runs that hold them
  const int n = min(max(__ldg(a.base_pos + s), 0), a.max_pos);
  const int nch = (n + kTtCH - 1) / kTtCH + 1;
  long long X = 0, total = 0;
  for (int q = lane; q < a.n_seqs; q += 32) {
    const int m = min(max(__ldg(a.base_pos + q), 0), a.max_pos);
    const long long k = (long long)((m + kTtCH - 1) / kTtCH + 1) * ips;
    total += k;
    if (q < s) X += k;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    X += __shfl_xor_sync(0xffffffffu, X, o);
    total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  X += (long long)it * nch;
  const long long per = (total + nb - 1) / nb;
  const int b0 = (int)(X / per), b1 = (int)((X + nch - 1) / per);
  if (b0 == b1) return;  // written by its CTA
  const int tile = rg >> 2, prow = (rg & 3) * 32 + lane;
  const float* base = static_cast<const float*>(a.work);
  auto slot = [&](int b) {
    return base + ((size_t)2 * b + ((long long)b * per > X ? 0 : 1)) * tt_slot_floats<D, NT>();
  };
  constexpr int ML = NT * kTtRows * D;
  const int mrow = tile * kTtRows + prow;
  const float lb1 = qv < nqv ? slot(b1)[ML + NT * kTtRows + mrow] : -1.f;
  float M = -INFINITY, L = 0.f, o[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) o[k] = 0.f;
  for (int b = b0; b <= b1; ++b) {
    const float* sl = slot(b);
    float4 v[4];
    const float4* p4 = reinterpret_cast<const float4*>(sl) + (size_t)tile * (kTtRows * D / 4) + (size_t)(cg * 4) * kTtRows + prow;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = p4[(size_t)k * kTtRows];
    const float mb = sl[ML + mrow], lb = sl[ML + NT * kTtRows + mrow];
    const float Mn = fmaxf(M, mb);
    const float x = M == -INFINITY ? 0.f : tt_ex2(M - Mn), y = mb == -INFINITY ? 0.f : tt_ex2(mb - Mn);
    M = Mn;
    L = L * x + lb * y;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      o[4 * k] = fmaf(v[k].x, y, o[4 * k] * x);
      o[4 * k + 1] = fmaf(v[k].y, y, o[4 * k + 1] * x);
      o[4 * k + 2] = fmaf(v[k].z, y, o[4 * k + 2] * x);
      o[4 * k + 3] = fmaf(v[k].w, y, o[4 * k + 3] * x);
    }
  }
  if (qv >= nqv || lb1 < 0.f) return;
  const float inv = L > 0.f ? 1.f / L : L == L ? 0.f : L;
  const int node = qv / grp, head = g * grp + qv % grp;
  uint4* d4 = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.out) +
                                       ((size_t)s * a.rows + node) * a.nq * D + (size_t)head * D + cg * 16);
  uint32_t u[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) u[k] = tt_pack<false>(o[2 * k] * inv, o[2 * k + 1] * inv);
  d4[0] = make_uint4(u[0], u[1], u[2], u[3]);
  d4[1] = make_uint4(u[4], u[5], u[6], u[7]);
}

template <int D, int NT, bool Q8>
cudaError_t tt_launch(const TreeAttnDesc& a, int num_sms, cudaStream_t st) {
  using Cfg = TtCfg<D, NT, Q8>;
  TtTma p;
  p.a = a;
  const int nqv = a.rows * (a.nq / a.nkv);
  p.n_pt = (nqv + NT * kTtRows - 1) / (NT * kTtRows);
  const uint64_t rows = a.pages ? (uint64_t)a.pool * a.nkv * a.ps : (uint64_t)a.n_seqs * a.nkv * a.cap;
  bool okm;
  if (Q8) {
    okm = make_tmap_u8(&p.kc, a.kc, D, rows, kTtCH) && make_tmap_u8(&p.vc, a.vc, D, rows, kTtCH);
    p.kb = p.kc;
    p.vb = p.vc;
  } else {
    const uint64_t M = (uint64_t)a.n_seqs * a.rows;
    okm = make_tmap_bf16(&p.kc, a.kc, D, rows, kTtCH) && make_tmap_bf16(&p.vc, a.vc, D, rows, kTtCH) &&
          make_tmap3_bf16(&p.kb, a.kb, D, a.nkv, M, 1, kTtCH) && make_tmap3_bf16(&p.vb, a.vb, D, a.nkv, M, 1, kTtCH);
  }
  if (!okm) return cudaErrorInvalidValue;
  cudaError_t e =
      cudaFuncSetAttribute(tree_tc_kernel<D, NT, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_pdl(tree_tc_kernel<D, NT, Q8>, dim3(num_sms), dim3(Cfg::THREADS), Cfg::SMEM, st, p);
  if (e != cudaSuccess) return e;
  const long long warps = (long long)a.n_seqs * a.nkv * p.n_pt * (NT * 4) * (D / 16);
  return launch_pdl(tree_tc_merge_kernel<D, NT>, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0, st, a, p.n_pt,
                    num_sms);
}

}  // namespace

size_t tree_tc_workspace(const TreeAttnDesc& a, int num_sms) {
  const int nt = a.rows * (a.nq / a.nkv) > kTtRows ? 2 : 1;
  return (size_t)2 * num_sms * nt * kTtRows * (a.d + 2) * sizeof(float);
}

cudaError_t launch_tree_tc(const TreeAttnDesc& a, int num_sms, cudaStream_t st) {
  const bool two = a.rows * (a.nq / a.nkv) > kTtRows, q8 = a.k_exp != nullptr;
  if (a.d == 128) {
    if (two) return q8 ? tt_launch<128, 2, true>(a, num_sms, st) : tt_launch<128, 2, false>(a, num_sms, st);
    return q8 ? tt_launch<128, 1, true>(a, num_sms, st) : tt_launch<128, 1, false>(a, num_sms, st);
  }
  if (two) return q8 ? tt_launch<64, 2, true>(a, num_sms, st) : tt_launch<64, 2, false>(a, num_sms, st);
  return q8 ? tt_launch<64, 1, true>(a, num_sms, st) : tt_launch<64, 1, false>(a, num_sms, st);
}

}  // namespace dfl
