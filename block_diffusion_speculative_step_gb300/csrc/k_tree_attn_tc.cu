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
//   P = 2^(c S - m)  one thread per query vector, written over S
//   O += P V         tcgen05.mma, P from tensor memory, V MN-major
// With NT = 2 the streams' softmaxes take turns, so that one stream's products
// run beside the other's softmax (left alone both fall in step and wait for
// their products together): the next one starts after this one's second part
// (bf16: its last; 8-bit, whose softmax is longer: of four).  32 sequences x 64
// rows, 8k: 247 us without turns, 183 so, 213 from the second half on in bf16;
// after one, two, three, four quarters 281, 261, 268, 282 in 8 bits.
// The reference m stays while the weights' sum suits bf16, which has fp32's
// exponents: it starts at m = 0 and takes sums of 2^-30 .. 2^30, so the usual
// chunk needs no maximum and no rescaling of O, and O stays in range up to
// values of 2^97.  Otherwise the part of the
// chunk (a half; 8-bit a quarter) is done again with its maximum: its scores
// stay until its sum is known.
//
// Roles: warp 0 K/V copies; warps 1, 2 the products of stream 0, 1 (a job's
// waits and commits take about 600 cycles of one thread, so each stream has a
// warp); warp 3 query copies, the tree's ancestor masks, rows of V to clear;
// warps 4..11 the softmax, a query vector per thread; 8-bit: warps 12..15
// convert.  Eight softmax warps with many registers measured faster than
// sixteen: two threads a row spend more instructions on exchanging maxima and
// votes than they save.  Registers are what the softmax is short of: shared
// memory leaves the first-level cache next to nothing, so a spilled value is
// an L2 access (a softmax that spilled 300 bytes took 3.5k cycles a chunk
// instead of 1.6k).  Hence scores in 16-column pieces, and an 8-bit chunk in
// quarters.
//
// The softmax is no rounding point: the weights enter their product as two
// bf16 operands, P = P_hi + P_lo (2^-16 relative), whose products share V's tile
// and the accumulator; one rounding to bf16 alone moved outputs by 0.16%
// (2-norm), as much as their own rounding.  The second product costs 183 us
// against 160 (32 sequences x 64 rows, 8k).  Starting a part's product beside
// the next part's weights: 185, and not worth its barriers.  The sum l uses the
// unrounded weights.
//
// 8-bit cache: K's codes go to the product as they are (kind::f8f6f4, the
// codes' rate is twice the 16-bit one), with the query vector as the sum of
// two e4m3 codes an element (4 + 4 significant bits hold bf16's 8; see
// tt_split8) and the tree's keys as two codes too; the keys' scales 2^e are
// multiplied to the scores.  V is rewritten to bf16 by four warps: code * 2^e,
// exact whatever the rows' exponents.  (As fp16, over a scale per chunk, small
// rows beside large ones -- hidden rows and padding among the tree's -- lost
// their digits or vanished: 243 us where this takes 265.  Rewriting K as well
// made each chunk's scores wait for a conversion: 365 against 243.)
//
// What bounds it, per 128-key chunk and SM at NT = 2: HBM 2.9k cycles in
// bf16, 1.5k in 8 bits; the tensor core 3.2k (6 x 8 products of 67
// cycles); measured 4.1k in bf16 -- a stream's scores, softmax and products are
// one chain, and the other stream's products stand in its way -- and about 6.4k
// in 8 bits, where the chain has the scales' loads and multiplications in it and
// 128 registers a thread leave little in flight.
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
constexpr int kTtKeyExp = -40;  // 8-bit cache: tree keys' smallest scale (their elements are held to 2^-50)
constexpr int kTtRing = 8;      // chunks whose scale exponents and bad rows are kept (roles run at most 4 apart)

struct TtTma {
  CUtensorMap kc, vc;  // cache rows [..][D]: bf16 boxes of 64 dims, or e4m3 boxes of D bytes, 128 rows
  CUtensorMap kb, vb;  // tree rows [M][nkv][D] (bf16 cache)
  CUtensorMap q3;      // queries [M][nq][D], box 64 dims x group x 128 / group tokens (q_tma)
  int q_tma;           // the group divides 128: a query tile is one box per 64 dims
  TreeAttnDesc a;
  int n_pt;            // query tile groups per KV head
  uint32_t grp_mul;    // ceil(2^32 / group) for groups of 2 .. 256 query heads, else 0
};

// qv / grp.  For grp <= 256 and qv < 128 grp the product's error, qv (grp - 1)
// 2^-32 at most, stays below 1 / grp.
__device__ __forceinline__ int tt_div_grp(const TtTma& p, int qv, int grp) {
  return p.grp_mul ? (int)__umulhi((uint32_t)qv, p.grp_mul) : qv / grp;
}

template <int D, int NT, bool Q8>
struct TtCfg {
  static constexpr int TILE = kTtCH * D * 2;                   // one 16-bit K or V tile
  static constexpr int RAW = kTtCH * D;                        // one e4m3 tile
  // (NT = 1: even, so that a slot always serves the same stream and its
  // issuer sees every phase of the slot's barriers)
  static constexpr int NSK = D == 64 ? 4 : 2;                  // K slots
  static constexpr int NSV = !Q8 && D == 64 ? 4 : 2;           // V slots (16 bit)
  static constexpr int NRV = !Q8 ? 0 : NT == 2 && D == 128 ? 1 : 2;  // raw V slots
  static constexpr int KT = Q8 ? RAW : TILE;                   // K slot
  static constexpr int WARPS = Q8 ? 16 : 12;                   // copies, 2 issuers, queries and clearing, 2 x 4 softmax (, 4 converters)
  static constexpr int THREADS = WARPS * 32;
  static constexpr int Q_OFF = 0;
  static constexpr int K_OFF = NT * TILE;
  static constexpr int T_OFF = K_OFF + NSK * KT;               // 8-bit: the tree's K in two e4m3 tiles
  static constexpr int V_OFF = T_OFF + (Q8 ? 2 * RAW : 0);
  static constexpr int R_OFF = V_OFF + NSV * TILE;             // raw V slots
  static constexpr int X_OFF = R_OFF + NRV * RAW;              // exchange, masks, barriers
  static constexpr int X_BYTES = 16384;
  static constexpr size_t SMEM = X_OFF + X_BYTES + 1024;
  static_assert(SMEM <= 232448, "shared memory of one CTA");
};

struct TtShared {  // after the tiles
  float xm[2][128], xl[2][128];  // a segment's stream statistics (NT = 1): maximum, sum
  int par[DFLASH_MAX_TREE];
  uint32_t mask[4][DFLASH_MAX_TREE][4];      // the tree rows' ancestors and themselves (none: padding)
  float kf[4][kTtCH];             // 8-bit: the keys' scales 2^e, by chunk counter (two V slots keep the converters at most 3 ahead)
  uint32_t badv[kTtRing][4];      // tree rows whose V holds a NaN or infinity, by chunk counter
  float fac[2][kTtCH];            // converters: the V rows' scales 2^e, by chunk & 1
  int s0, it0, c0, len, n0;       // the CTA's run: first item, position in it, number of positions; context of s0
  int setup;
  uint64_t kfull[4], kempty[4], vfull[4], vempty[4];
  uint64_t rvfull[2], rvempty[2];
  uint64_t kfr[kTtRing];          // kf written
  uint64_t tkfull[2], tkempty;    // the tree's K tiles (NT = 1: by the stream that takes them)
  uint64_t sfull[2], pdone[2], ofull[2], qraw[2];
  uint64_t qfull[2], qfree[2];    // see tt_qi
  uint64_t mready[4];             // ancestor masks written, by buffer
  uint64_t vraw[4];               // V tiles with rows to clear, copied (at most NSV <= 4 are ahead of their P V)
  uint32_t tslot;
  int abort;
  int8_t qe[4][2][128];           // query vectors' scale exponents (8-bit cache), by segment
};

__device__ __forceinline__ void named_arrive(int id, int nthreads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

// One lane of the warp (the same one each time).
__device__ __forceinline__ bool tt_elect() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* m, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global [%0, {%1, %2, %3}];" ::"l"(reinterpret_cast<uint64_t>(m)),
               "r"(x), "r"(y), "r"(z)
               : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]: A packed 16-bit, two per column, K along columns.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}

// D[tmem] (+)= A[smem] * B[smem], e4m3 operands, 32 of K.
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}

// Descriptor of a K-major tile with rows of 128 bytes, or of 64 with their swizzle.
template <int ROW>
__device__ __forceinline__ uint64_t tt_sdesc(uint32_t saddr) {
  const uint64_t d = tc::sdesc_sw128(saddr);
  if (ROW == 128) return d;
  // 64-byte swizzle (type 4 in bits 61..63), groups of 8 rows 512 bytes apart
  return (d & ~((7ull << 61) | (0x3FFFull << 32))) | (4ull << 61) | ((uint64_t)(512 >> 4) << 32);
}
// Byte offset of (row, 16-byte piece) in such a tile of codes.
template <int ROW>
__device__ __forceinline__ uint32_t tt_off8(int row, int ch) {
  return ROW == 128 ? (uint32_t)(row * 128 + ((ch ^ (row & 7)) << 4)) : (uint32_t)(row * 64 + ((ch ^ ((row >> 1) & 3)) << 4));
}

// Both operands e4m3 (type code 0 of kind::f8f6f4) instead of bf16 (1 of kind::f16).
__host__ __device__ constexpr uint32_t tt_idesc_e4m3(int M, int N) {
  return tc::idesc_bf16_f32(M, N) & ~((7u << 7) | (7u << 10));
}

// 16 columns of this thread's lane, not waited for: the registers hold them
// after tmem_wait on the same array (which makes the compiler keep the order).
__device__ __forceinline__ void tmem_ld_async(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]),
                 "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}

// 16 packed columns of this thread's lane; returns once stored (one statement:
// the source registers are read until the wait).
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// The same for the 32 columns r[0 .. 31].
__device__ __forceinline__ void tmem_st32u(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// Packed fp32 pairs (two fused multiply-adds / additions per instruction).
__device__ __forceinline__ unsigned long long tt_pair(float lo, float hi) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void tt_unpair(unsigned long long v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ unsigned long long tt_fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ unsigned long long tt_add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ unsigned long long tt_mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float tt_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t tt_pack(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The pair (lo, hi) as bf16 values h and the bf16 values l of what they left:
// h + l carries it to 2^-16 relative (half a step of half a step).
__device__ __forceinline__ void tt_split_bf16(float lo, float hi, uint32_t& h, uint32_t& l) {
  h = tt_pack(lo, hi);
  const unsigned long long r = tt_fma2(tt_pair(__uint_as_float(h << 16), __uint_as_float(h & 0xFFFF0000u)),
                                       tt_pair(-1.f, -1.f), tt_pair(lo, hi));
  tt_unpair(r, lo, hi);
  l = tt_pack(lo, hi);
}

// Index and phase of the query barriers (qfull, qfree) of stream t's tile in
// segment `seg`.  NT = 2: a barrier per stream, whose issuer reads the tile in
// every segment.  NT = 1: both issuers read one tile, but an issuer has no
// chunk in a segment of one chunk that the other takes (of two such segments in
// a row it has one).  It lets such a segment go at once, without having waited
// for its queries, and may so be a segment ahead of the other issuer.  A barrier
// per segment parity keeps its arrival apart from the other's for the segment
// before, and the phase that it does wait for next to the one before it.
template <int NT>
__device__ __forceinline__ int tt_qi(int t, int seg) { return NT == 2 ? t : seg & 1; }
template <int NT>
__device__ __forceinline__ uint32_t tt_qp(int seg) { return (uint32_t)(NT == 2 ? seg : seg >> 1); }

// Byte offset of (row, 16-byte piece) in a 16-bit tile of 128 rows kept as
// 64-element boxes with the 128-byte swizzle.
__device__ __forceinline__ uint32_t tt_off(int row, int ch) {
  return (uint32_t)((ch >> 3) * (kTtCH * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
}

// A CTA's run walked segment by segment; every role keeps its own copy.
struct Seg {
  const TreeAttnDesc* a;
  bool uniform;        // a whole warp walks: loaded values through a reduction, which the compiler
                       // knows to be the same in every lane
  int ips, left;       // items per sequence; positions of the run not yet walked
  int setup;           // positions an item has before its chunks
  int s, it;           // sequence, item of the sequence
  int n_ctx, nch;      // context slots, chunks of the item (the last one the tree)
  int n_next;          // the next sequence's length, loaded ahead
  int c0, c1;          // the segment's chunks
  __device__ __forceinline__ void ahead() { n_next = s + 1 < a->n_seqs ? __ldg(a->base_pos + s + 1) : 0; }
  __device__ __forceinline__ void load() {
    n_ctx = min(max(n_next, 0), a->max_pos);
    if (uniform) n_ctx = __reduce_max_sync(0xffffffffu, n_ctx);
    nch = (n_ctx + kTtCH - 1) / kTtCH + 1;
    ahead();
  }
  // The part of the current item from position v on, at most `left` positions.
  __device__ __forceinline__ void take(int v) {
    const int n = min(nch + setup - v, left);
    c0 = max(0, v - setup);
    c1 = max(0, v + n - setup);
    left -= n;
  }
  __device__ __forceinline__ bool begin(const TreeAttnDesc* d, int ips_, const TtShared* sh, bool uni = false) {
    a = d;
    ips = ips_;
    uniform = uni;
    auto same = [&](int x) { return uniform ? __reduce_max_sync(0xffffffffu, x) : x; };
    left = same(sh->len);
    if (left <= 0) return false;
    s = same(sh->s0);
    it = same(sh->it0);
    setup = same(sh->setup);
    n_ctx = same(sh->n0);
    nch = (n_ctx + kTtCH - 1) / kTtCH + 1;
    ahead();
    take(same(sh->c0));
    return c1 > c0 || next();
  }
  __device__ __forceinline__ bool next() {
    do {
      if (left <= 0) return false;
      if (++it == ips) {
        it = 0;
        ++s;
        load();
      }
      take(0);
    } while (c1 <= c0);
    return true;
  }
  __device__ __forceinline__ bool is_tree(int c) const { return c == nch - 1; }
  __device__ __forceinline__ int keys(int c) const { return is_tree(c) ? a->rows : min(kTtCH, n_ctx - c * kTtCH); }
};

// How the chunks of all items are cut into runs, one per CTA (the host checks
// that their number fits 31 bits):
//   flat     CTA b takes positions [b per, (b + 1) per) of all items in a row,
//            per = ceil(total / nb): every CTA the same number.  An item has
//            tt_setup positions before its chunks', for what it costs besides
//            them (queries, masks, first chunk, output: about 8k cycles, and
//            an 8-bit cache's conversion of queries and tree).  32 sequences
//            x 64 rows, 8k: 1 / 2 / 3 positions 190 / 186 / 187 us in bf16, 279
//            / 265 / 266 us in 8 bits;
//   aligned  an item's chunks are cut into runs of `per` and every run has a
//            CTA of its own, per the smallest for which nb CTAs suffice: no
//            CTA has parts of two items, which costs a second query load,
//            prologue and partial (about 6 us).
// Aligned where its runs are at most one chunk longer than the flat ones, i.e.
// for few items: 8 items of 33 chunks take 2 chunks on 136 CTAs, flat 2 on
// 132 of which 7 straddle two items (batch 1, 4k context: 12 us against 18).
__device__ __forceinline__ int tt_setup(const TreeAttnDesc& a) { return a.k_exp ? 3 : 2; }
struct Part {
  int aligned, per;  // flat: positions per CTA; aligned: chunks
  int sp;            // aligned: CTAs of every item, or 0: as many as its own chunks need
  int total;         // positions (flat)
};

__device__ __forceinline__ int tt_chunks(const TreeAttnDesc& a, int s, int* n) {
  *n = min(max(__ldg(a.base_pos + s), 0), a.max_pos);
  return (*n + kTtCH - 1) / kTtCH + 1;
}

// One warp.  status (or null): told of lengths outside their bound.
__device__ __forceinline__ Part tt_part(const TreeAttnDesc& a, int ips, int nb, uint32_t* status) {
  int t = 0, mx = 0, n;
  for (int s = threadIdx.x & 31; s < a.n_seqs; s += 32) {
    const int k = tt_chunks(a, s, &n);
    if (__ldg(a.base_pos + s) != n) raise_status(status, ST_RANGE);
    t += k;
    mx = max(mx, k);
  }
  Part p;
  t = __reduce_add_sync(0xffffffffu, t);
  mx = __reduce_max_sync(0xffffffffu, mx);
  p.total = (t + a.n_seqs * tt_setup(a)) * ips;
  p.per = (p.total + nb - 1) / nb;
  p.aligned = p.sp = 0;
  if (a.n_seqs * ips > nb) return p;
  const int least = (t * ips + nb - 1) / nb, sp = nb / (a.n_seqs * ips), even = (mx + sp - 1) / sp;
  if (even <= least + 1) {  // the same number for every item is as good: no search, no scan
    p.sp = sp;
    p.aligned = even <= p.per + 1;
    if (p.aligned) p.per = even;
    return p;
  }
  auto fits = [&](int per) {  // do nb CTAs suffice for runs of per chunks?
    int r = 0;
    for (int s = threadIdx.x & 31; s < a.n_seqs; s += 32) r += (tt_chunks(a, s, &n) + per - 1) / per;
    return __reduce_add_sync(0xffffffffu, r) * ips <= nb;
  };
  int lo = least, hi = even;
  while (lo < hi) {
    const int mid = hi - lo > 4 ? (lo + hi) >> 1 : lo;
    if (fits(mid)) hi = mid;
    else lo = mid + 1;
  }
  if (lo <= p.per + 1) {
    p.aligned = 1;
    p.per = lo;
  }
  return p;
}

// The sequence, item, position in the item, context length and number of
// chunks at position x of the flat order; aligned (run > 0): position = run
// of the item, x = CTA.
struct Spot {
  int s, it, c, n, nch;
};
__device__ __forceinline__ Spot tt_locate(const TreeAttnDesc& a, int ips, int x, int run) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  Spot p = {a.n_seqs, 0, 0, 0, 1};
  for (int b = 0; b < a.n_seqs; b += 32) {
    const int s = b + lane;
    int n = 0;
    const int nch = s < a.n_seqs ? tt_chunks(a, s, &n) : 0;
    const int len = s >= a.n_seqs ? 0 : run ? (nch + run - 1) / run : nch + tt_setup(a);
    int inc = len * ips;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + inc > x);
    if (hit) {
      const int w = __ffs(hit) - 1;
      p.nch = __shfl_sync(0xffffffffu, nch, w);
      const int k = __shfl_sync(0xffffffffu, len, w), at = x - (before + __shfl_sync(0xffffffffu, inc, w) - k * ips);
      p.s = b + w;
      p.it = at / k;
      p.c = at % k;
      p.n = __shfl_sync(0xffffffffu, n, w);
      return p;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  return p;
}

// The run of CTA b (aligned): its item, number in the item (c), lengths.
__device__ __forceinline__ Spot tt_run(const TreeAttnDesc& a, int ips, int b, const Part& pt) {
  if (!pt.sp) return tt_locate(a, ips, b, pt.per);
  Spot p = {a.n_seqs, 0, 0, 0, 1};
  const int item = b / pt.sp;
  if (item < a.n_seqs * ips) {
    p.s = item / ips;
    p.it = item % ips;
    p.c = b % pt.sp;
    p.nch = tt_chunks(a, p.s, &p.n);
  }
  return p;
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

// The smallest e in [-118, 120] with mx <= 448 * 2^e (e4m3's largest value).
__device__ __forceinline__ int tt_exp8_of(float mx) {
  const int b = __float_as_int(mx);
  return min(max((b >> 23) - 135 + ((b & 0x7FFFFF) > 0x600000 ? 1 : 0), -118), 120);
}

// Eight elements over 2^e as the sum of two e4m3 codes each: 4 significant
// bits, then 4 of what is left.  A bf16's 8 are kept down to 2^-10 of the
// largest element's power of two; below, the second code's smallest step bounds
// the error by 2^-10 / 224 of the largest.  NaN and infinite elements give NaN.
__device__ __forceinline__ void tt_split8(const float (&v)[8], int e, uint2& hi, uint2& lo) {
  const float s = __int_as_float((127 - e) << 23);
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 y = make_float2(v[2 * i] * s, v[2 * i + 1] * s);
    y.x = fabsf(y.x) < INFINITY ? y.x : NAN;
    y.y = fabsf(y.y) < INFINITY ? y.y : NAN;
    h[i] = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
    const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)h[i], __NV_E4M3)));
    l[i] = __nv_cvt_float2_to_fp8x2(make_float2(y.x - f.x, y.y - f.y), __NV_SATFINITE, __NV_E4M3);
  }
  hi = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
  lo = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
}

// 16 e4m3 codes times f -> 16 bf16 values (two 16-byte pieces): exact, for a
// code has 4 significant bits and f is a power of two.
__device__ __forceinline__ void tt_codes_to_bf16(const uint4& c, float f, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  const unsigned long long f2 = tt_pair(f, f);
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 x = __half22float2(__half2(
        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu), __NV_E4M3)));
    float a, b;
    tt_unpair(tt_mul2(tt_pair(x.x, x.y), f2), a, b);
    o[i] = tt_pack(a, b);
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// Bits 15 and 31: a bf16 element whose exponent is all ones (NaN or infinite).
__device__ __forceinline__ uint32_t tt_odd(const uint4& x) {
  const uint32_t e[4] = {x.x, x.y, x.z, x.w};
  uint32_t odd = 0u;
#pragma unroll
  for (int k = 0; k < 4; ++k) odd |= ((e[k] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
  return odd;
}
// Those elements cleared.
__device__ __forceinline__ uint4 tt_clear_odd(const uint4& x) {
  uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if ((e[k] & 0x7F80u) == 0x7F80u) e[k] &= 0xFFFF0000u;
    if ((e[k] & 0x7F800000u) == 0x7F800000u) e[k] &= 0xFFFFu;
  }
  return make_uint4(e[0], e[1], e[2], e[3]);
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
  uint8_t* Ts = sm + Cfg::T_OFF;
  uint8_t* Rv = sm + Cfg::R_OFF;
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
      tc::mbar_init(&sh->kfull[i], 1);
      tc::mbar_init(&sh->kempty[i], NT);  // the issuers that read the slot
      tc::mbar_init(&sh->vfull[i], Q8 ? 128 : 1);
      tc::mbar_init(&sh->vempty[i], NT);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sh->tkfull[i], 128);
      tc::mbar_init(&sh->rvfull[i], 1);
      tc::mbar_init(&sh->rvempty[i], 128);
      // the product's commit, and the issuer's own arrival: what the issuer has
      // observed (scale exponents, bad rows) is visible to who waits here
      tc::mbar_init(&sh->sfull[i], 2);
      tc::mbar_init(&sh->pdone[i], 128);
      tc::mbar_init(&sh->ofull[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sh->qraw[i], 1);
      tc::mbar_init(&sh->qfull[i], Q8 || !p.q_tma ? 128 : 1);  // the rows' threads, or the copy
      tc::mbar_init(&sh->qfree[i], NT == 1 ? 2 : 1);           // the issuers that read the tile
    }
    for (int i = 0; i < kTtRing; ++i) tc::mbar_init(&sh->kfr[i], 128);
    tc::mbar_init(&sh->tkempty, NT);
    for (int i = 0; i < 4; ++i) tc::mbar_init(&sh->vraw[i], 1);
    for (int i = 0; i < 4; ++i) tc::mbar_init(&sh->mready[i], 32);
    sh->abort = 0;
    for (int i = 0; i < kTtRing * 4; ++i) sh->badv[i >> 2][i & 3] = 0u;
    tc::fence_mbar_init();
    tc::tma_prefetch_desc(&p.kc);
    tc::tma_prefetch_desc(&p.vc);
  }
  if (warp == 1) tc::tmem_alloc(&sh->tslot, 512);
  pdl_wait();
  pdl_launch_dependents();
  if (warp == 0) {
    const Part pt = tt_part(a, ips, gridDim.x, status);
    Spot sp = {0, 0, 0, 0, 1};
    int len = 0;
    if (pt.aligned) {
      sp = tt_run(a, ips, blockIdx.x, pt);
      if (sp.s < a.n_seqs && sp.c * pt.per < sp.nch) {
        sp.c *= pt.per;
        len = min(pt.per, sp.nch - sp.c);
      }
    } else {
      const int x0 = min((int)blockIdx.x * pt.per, pt.total);  // (nb * per < total + nb: no overflow)
      len = min(pt.per, pt.total - x0);
      if (len > 0) sp = tt_locate(a, ips, x0, 0);
    }
    if (lane == 0) {
      sh->s0 = sp.s;
      sh->it0 = sp.it;
      sh->c0 = sp.c;
      sh->n0 = sp.n;
      sh->len = len;
      sh->setup = pt.aligned ? 0 : tt_setup(a);
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
      int nk = 0, nv = 0, nraw = 0;  // copies issued; V tiles with rows to clear
      uint32_t parts = 0u;           // which of the last V tiles those were
      constexpr int SK = NSK, SV = Q8 ? Cfg::NRV : NSV;
      uint64_t* kf = sh->kfull;
      uint64_t* ke = sh->kempty;
      uint64_t* vf = Q8 ? sh->rvfull : sh->vfull;
      uint64_t* ve = Q8 ? sh->rvempty : sh->vempty;
      const uint64_t pol = tc::policy_evict_first();
      for (bool on = sg.begin(&a, ips, sh); on && ok; on = sg.next()) {
        const int g = sg.it / p.n_pt;
        for (int c = sg.c0; c < sg.c1 && ok; ++c) {
          const bool tree = sg.is_tree(c);
          int row = 0;
          if (!tree) {
            bool bad = false;
            row = (int)(km.row0(sg.s, c * kTtCH, &bad) + (uint32_t)g * (uint32_t)km.head_rows());
            if (bad) raise_status(status, ST_RANGE);  // reads page 0 instead
          }
          if (nk >= SK && !wait(&ke[nk % SK], (uint32_t)(nk / SK - 1))) break;
          if constexpr (Q8) {
            if (tree) {  // the converters read the tree's rows themselves; its slot stays unused
              tc::mbar_arrive(&kf[nk++ % SK]);
              continue;
            }
            tc::mbar_arrive_expect_tx(&kf[nk % SK], RAW);
            tc::tma_load_2d(Ks + (nk % SK) * RAW, &p.kc, 0, row, &kf[nk % SK], pol);
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
            const bool part = tree || sg.keys(c) < kTtCH;  // warp 3 clears rows and passes the tile on
            uint64_t* bar = part ? &sh->vraw[nraw++ & 3] : &vf[nv % SV];
            parts = parts << 1 | (part ? 1u : 0u);
            tc::mbar_arrive_expect_tx(bar, TILE);
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
              uint8_t* dst = Vs + (nv % SV) * TILE + h * (kTtCH * 128);
              if (tree) tc::tma_load_3d(dst, &p.vb, 64 * h, g, sg.s * a.rows, bar);
              else tc::tma_load_2d(dst, &p.vc, 64 * h, row, bar, pol);
            }
          }
          ++nv;
        }
      }
      // every copy has landed before the CTA's shared memory goes away
      for (int i = max(0, nk - SK); i < nk; ++i) tc::mbar_wait(&kf[i % SK], (uint32_t)(i / SK) & 1u, nullptr, lim_ns);
      for (int i = max(0, nv - SV); i < nv; ++i)
        if (!(parts >> (nv - 1 - i) & 1u)) tc::mbar_wait(&vf[i % SV], (uint32_t)(i / SV) & 1u, nullptr, lim_ns);
      for (int i = max(0, nraw - SV); i < nraw; ++i) tc::mbar_wait(&sh->vraw[i & 3], (uint32_t)(i >> 2) & 1u, nullptr, lim_ns);
    }
  } else if (warp == 1 || warp == 2) {
    // ---------------------------------------------------- MMA issue, stream t
    // The whole warp walks the stream's jobs, so that descriptors and
    // addresses stay in uniform registers; one lane issues.  A warp per
    // stream: a job's waits and commits (about 700 cycles in one thread) then
    // run beside the other stream's.
    const int t = warp - 1;
    constexpr uint32_t idS = Q8 ? tt_idesc_e4m3(kTtRows, kTtCH) : tc::idesc_bf16_f32(kTtRows, kTtCH);
    constexpr uint32_t idV = tc::idesc_bf16_f32_bmn(kTtRows, D);
    const uint32_t ut = __reduce_max_sync(0xffffffffu, (uint32_t)t);
    const uint64_t dq = tc::sdesc_sw128(tc::smem_u32(Qs) + (NT == 2 ? ut * TILE : 0u)),
                   dk = tt_sdesc<Q8 ? D : 128>(tc::smem_u32(Ks)), dt = tt_sdesc<Q8 ? D : 128>(tc::smem_u32(Ts)),
                   dv = tc::sdesc_sw128_mn(tc::smem_u32(Vs), kTtCH * 128, 1024);
    const uint32_t tm_s = __reduce_max_sync(0xffffffffu, tmem) + ut * 128u, tm_o = tm_s + 256u;
    // S of the stream's next job is issued right behind P V of the job
    // before, whose P lies in the same columns.
    Seg ss;                      // the S side's segment
    int sc = 0, c = 0;           // its chunk counter and chunk
    int s_seg = 0, q_seen = -1;  // segment; the last one whose queries have been waited for
    int t_seen = 0;              // the tree's K tiles waited for
    bool s_on = ss.begin(&a, ips, sh, true);
    if (s_on) c = ss.c0;
    auto s_next = [&]() {
      ++sc;
      if (++c == ss.c1) {
        if (tt_elect()) tc::mma_commit(&sh->qfree[tt_qi<NT>(t, s_seg)]);  // the segment's query tile has been read
        __syncwarp();
        ++s_seg;
        s_on = ss.next();
        c = ss.c0;
      }
    };
    if (NT == 1 && s_on && ut == 1u) s_next();  // (stream 1 takes the odd chunks)
    auto wait_s = [&]() {  // the operands of the next S
      if (q_seen < s_seg) {
        q_seen = s_seg;
        if (!wait_warp(&sh->qfull[tt_qi<NT>(t, s_seg)], tt_qp<NT>(s_seg))) return;
      }
      if (!wait_warp(&sh->kfull[sc % NSK], (uint32_t)(sc / NSK))) return;
      if (Q8 && ss.is_tree(c)) wait_warp(&sh->tkfull[NT == 1 ? t : 0], (uint32_t)t_seen++);
    };
    auto issue_s = [&]() {
      if (!ok) return;
      const int slot = sc % NSK;
      tc::tc_fence_after();
      const uint64_t k = dk + (uint64_t)(slot * Cfg::KT / 16);
      const bool tree = Q8 && ss.is_tree(c);
      if (tt_elect()) {
        if constexpr (Q8) {
          // 32 dims a step: the queries' high codes, then what those left
#pragma unroll
          for (int j = 0; j < D / 32; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              mma_e4m3(tm_s, dq + (uint64_t)((j >> 1) * (kTtRows * 128 / 16) + (j & 1) * 4 + h * 2),
                       (tree ? dt : k) + (uint64_t)(2 * j), idS, j + h > 0 ? 1u : 0u);
          if (tree) {
#pragma unroll
            for (int j = 0; j < D / 32; ++j)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                mma_e4m3(tm_s, dq + (uint64_t)((j >> 1) * (kTtRows * 128 / 16) + (j & 1) * 4 + h * 2),
                         dt + (uint64_t)(RAW / 16 + 2 * j), idS, 1u);
          }
        } else {
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            constexpr int kBox = kTtCH * 128 / 16;  // descriptor addresses count 16 bytes
            const uint64_t off = (uint64_t)((j >> 2) * kBox + (j & 3) * 2);
            tc::mma_bf16(tm_s, dq + off, k + off, idS, j > 0 ? 1u : 0u);
          }
        }
        tc::mma_commit(&sh->sfull[t]);
        tc::mbar_arrive(&sh->sfull[t]);
        tc::mma_commit(&sh->kempty[slot]);
        if (tree) tc::mma_commit(&sh->tkempty);
      }
      __syncwarp();
      s_next();
      if (NT == 1 && s_on) s_next();
    };
    if (s_on) {
      wait_s();
      issue_s();
    }
    int vc = 0, vj = 0;
    for (bool on = sg.begin(&a, ips, sh, true); on && ok; on = sg.next()) {
      uint32_t acc0 = 0u;  // the stream's first P V of the segment starts its accumulator
      for (int x = sg.c0; x < sg.c1 && ok; ++x, ++vc) {
        if (NT == 1 && (uint32_t)(vc & 1) != ut) continue;
        const int slot = vc % NSV, nk = sg.keys(x);
        if (!wait_warp(&sh->vfull[slot], (uint32_t)(vc / NSV))) break;
        // waited for early, so that S follows P V in the tensor pipe without a
        // gap; not across segments, whose query load may still take a while
        const bool last = x + NT >= sg.c1 + (NT == 2 ? 1 : -1);
        if (!last && s_on) wait_s();
        if (!wait_warp(&sh->pdone[t], (uint32_t)vj)) break;
        ++vj;
        tc::tc_fence_after();
        const uint64_t v = dv + (uint64_t)(slot * TILE / 16);
        if (tt_elect()) {
#pragma unroll
          for (int j = 0; j < kTtCH / 16; ++j)  // (16 keys a step; of a short chunk only those that hold some)
            if (16 * j < nk) {
              mma_ts(tm_o, tm_s + 16 * j, v + (uint64_t)(j * 128), idV, j > 0 ? 1u : acc0);
              mma_ts(tm_o, tm_s + 16 * j + 8, v + (uint64_t)(j * 128), idV, 1u);  // what P's first part left
            }
          // the stream's last job of the segment: its output is complete
          if (last) {
            tc::mma_commit(&sh->ofull[t]);
            tc::mbar_arrive(&sh->ofull[t]);
          }
        }
        __syncwarp();
        acc0 = 1u;
        if (s_on) {
          if (last) wait_s();
          issue_s();
        }
        if (tt_elect()) tc::mma_commit(&sh->vempty[slot]);  // (behind S: the softmax waits for S, nobody yet for V)
        __syncwarp();
      }
    }
  } else if (warp == 3) {
    // ---------------------------------------------------- ahead of the softmax: queries, masks, V rows to clear
    // Values of slots past the last key may be anything (unwritten cache
    // rows); a hidden tree row's may too.  0 * NaN is NaN, so such rows are
    // cleared before the product: of the tree's rows only NaN and infinite
    // elements, which the segment's end adds to the rows that see them.
    // (8-bit: the converters do it.)
    auto bar = [&](int t, int seg) { return Q8 ? &sh->qraw[t] : &sh->qfull[tt_qi<NT>(t, seg)]; };
    int n = 0, vc = 0, nraw = 0, nmask = 0, last_s = -1;
    for (bool on = sg.begin(&a, ips, sh); on && ok; ++n) {
      const int g = sg.it / p.n_pt, qv0 = (sg.it % p.n_pt) * (NT * kTtRows);
#pragma unroll 1
      for (int t = 0; t < NT; ++t) {
        if (n > 0 && !wait_warp(&sh->qfree[tt_qi<NT>(t, n - 1)], tt_qp<NT>(n - 1))) break;
        // (tokens past the sequence's last: other rows' queries or zeros, whose results are not used)
        if (p.q_tma && lane == 0) {
          tc::mbar_arrive_expect_tx(bar(t, n), TILE);
          const int tok = sg.s * a.rows + tt_div_grp(p, qv0 + t * kTtRows, grp);
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tc::tma_load_3d(Qs + t * TILE + h * (kTtRows * 128), &p.q3, 64 * h, g * grp, tok, bar(t, n));
        }
      }
      Seg nx = sg;
      const bool more = nx.next();
      if (more && p.q_tma && lane < NT * (D / 64)) {  // the next segment's queries into L2
        const int t = lane / (D / 64), h = lane % (D / 64);
        tma_prefetch_3d(&p.q3, 64 * h, nx.it / p.n_pt * grp,
                        nx.s * a.rows + tt_div_grp(p, (nx.it % p.n_pt) * (NT * kTtRows) + t * kTtRows, grp));
      }
      // the tree's ancestor masks, once per sequence, in turn into four buffers
      // (the queries of the segment before have been scored, so each stream's
      // softmax is done with every chunk of the fourth segment back)
      if (sg.c1 == sg.nch && sg.s != last_s) {
        last_s = sg.s;
        uint32_t(*mb)[4] = sh->mask[nmask & 3];
        if (a.parent)
          for (int i = lane; i < a.rows; i += 32) sh->par[i] = __ldg(a.parent + (size_t)sg.s * a.rows + i);
        __syncwarp();
        for (int i = lane; i < a.rows; i += 32) {
          uint32_t w[4] = {0u, 0u, 0u, 0u};
          bool bad = false;
          if (!tree_row_mask(a.parent ? sh->par : nullptr, i, w, &bad)) w[0] = w[1] = w[2] = w[3] = 0u;  // padding: sees nothing
          else if (a.pos) bad = (uint32_t)__ldg(a.pos + (size_t)sg.s * a.rows + i) >= (uint32_t)a.pos_end;
          if (bad) raise_status(status, ST_RANGE);
#pragma unroll
          for (int k = 0; k < 4; ++k) mb[i][k] = w[k];
        }
        ++nmask;
        __syncwarp();
        tc::mbar_arrive(&sh->mready[(nmask - 1) & 3]);
      }
      if constexpr (!Q8) {
        for (int c = sg.c0; c < sg.c1 && ok; ++c, ++vc) {
          const int nk = sg.keys(c), slot = vc % NSV;
          const bool tree = sg.is_tree(c);
          if (!tree && nk == kTtCH) continue;
          if (!wait_warp(&sh->vraw[nraw & 3], (uint32_t)(nraw >> 2))) break;
          ++nraw;
          constexpr int CPR = D / 8;
          uint8_t* vt = Vs + slot * TILE;
          auto at = [&](int i) { return reinterpret_cast<uint4*>(vt + tt_off(i / CPR, i % CPR)); };
          if (tree) {
            uint32_t any = 0u;
#pragma unroll 8
            for (int i = lane; i < nk * CPR; i += 32) any |= tt_odd(*at(i));
            if (lane < 4) sh->badv[vc % kTtRing][lane] = 0u;
            __syncwarp();
            if (__any_sync(0xffffffffu, any != 0u)) {
#pragma unroll 1
              for (int i = lane; i < nk * CPR; i += 32) {
                const uint4 x = *at(i);
                if (tt_odd(x)) {
                  *at(i) = tt_clear_odd(x);
                  atomicOr(&sh->badv[vc % kTtRing][i / CPR >> 5], 1u << (i / CPR & 31));
                }
              }
            }
          }
#pragma unroll 4
          for (int i = nk * CPR + lane; i < (nk + 15 & ~15) * CPR; i += 32) *at(i) = make_uint4(0, 0, 0, 0);
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sh->vfull[slot]);
        }
      }
      on = more;
      sg = nx;
    }
    // (a copy that was issued lands before the CTA's shared memory goes away)
    if (lane == 0 && p.q_tma && n > 0)
      for (int t = 0; t < NT; ++t)
        tc::mbar_wait(bar(t, n - 1), (Q8 ? (uint32_t)(n - 1) : tt_qp<NT>(n - 1)) & 1u, nullptr, lim_ns);
  } else if (warp < 12) {
    // ---------------------------------------------------- softmax: stream t, one query vector per thread
    const int t = (warp - 4) >> 2;
    const int r = (warp & 3) * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t ts = lane_base + t * 128, to = lane_base + 256 + t * 128;
    int nj = 0;         // jobs this stream has done
    int cc = 0;         // chunk counter
    int no[2] = {0, 0}; // segments in which each stream had a job
    int nmask = 0, last_s = -1;  // ancestor masks waited for, and their sequence
    int seg_no = 0;
    for (bool on = sg.begin(&a, ips, sh); on; on = sg.next(), ++seg_no) {
      const int g = sg.it / p.n_pt, qv0 = (sg.it % p.n_pt) * (NT * kTtRows);
      const int qv = qv0 + (NT == 2 ? t * kTtRows : 0) + r;
      const bool has_row = qv < nqv;
      const bool warp_on = __any_sync(0xffffffffu, has_row);
      const int node = has_row ? tt_div_grp(p, qv, grp) : 0;
      const int head = g * grp + (has_row ? qv - node * grp : 0);
      if ((Q8 || !p.q_tma) && (NT == 2 || t == 0)) {
        // ---- the thread's row of the query tile: loaded where it is no TMA
        // box, split into e4m3 codes in place with an 8-bit cache
        uint8_t* qd = Qs + (NT == 2 ? t * TILE : 0);
        if (p.q_tma) {
          wait(&sh->qraw[NT == 2 ? t : 0], (uint32_t)seg_no);
        } else {
          if (seg_no > 0) wait(&sh->qfree[tt_qi<NT>(t, seg_no - 1)], tt_qp<NT>(seg_no - 1));
          const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.q) +
                                                            ((size_t)sg.s * a.rows + node) * QD + (size_t)head * D);
#pragma unroll 8
          for (int ch = 0; ch < D / 8; ++ch)
            *reinterpret_cast<uint4*>(qd + tt_off(r, ch)) = has_row ? __ldg(src + ch) : make_uint4(0, 0, 0, 0);
          __syncwarp();
        }
        if constexpr (Q8) {
          // A warp's 32 rows, D / 16 lanes to a row, 16 dims to a lane: two
          // codes each, in place.  Of every 32 dims (64 bytes) the first half
          // takes the codes, the second the codes of what those left.
          constexpr int LR = D / 16, RW = 32 / LR;
          const int wr = (warp & 3) * 32, jl = (lane % LR) >> 1, hl = lane & 1;
#pragma unroll 1
          for (int r0 = wr; r0 < wr + 32 && qv - lane + (r0 - wr) < nqv; r0 += RW) {
            const int row = r0 + lane / LR;
            float v[2][8];
#pragma unroll
            for (int c = 0; c < 2; ++c)
              load8(reinterpret_cast<const __nv_bfloat16*>(qd + tt_off(row, 4 * jl + 2 * hl + c)), v[c]);
            float mx = fmaxf(tt_finite_max(v[0]), tt_finite_max(v[1]));
#pragma unroll
            for (int o = LR / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const int e = tt_exp8_of(mx);
            if (lane % LR == 0) sh->qe[seg_no & 3][NT == 2 ? t : 0][row] = (int8_t)e;
            uint2 h[2], l[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) tt_split8(v[c], e, h[c], l[c]);
            __syncwarp();  // the row has been read
            *reinterpret_cast<uint4*>(qd + tt_off(row, 4 * jl + hl)) = make_uint4(h[0].x, h[0].y, h[1].x, h[1].y);
            *reinterpret_cast<uint4*>(qd + tt_off(row, 4 * jl + 2 + hl)) = make_uint4(l[0].x, l[0].y, l[1].x, l[1].y);
          }
          __syncwarp();
        }
        tc::fence_proxy_async_smem();
        tc::mbar_arrive(&sh->qfull[tt_qi<NT>(t, seg_no)]);
      }
      const bool has_tree = sg.c1 == sg.nch;  // the segment ends with the tree's rows
      const int tree_ring = (cc + sg.c1 - 1 - sg.c0) % kTtRing;
      float m_run = -INFINITY, l_run = 0.f;
      const int nj0 = nj;
      uint32_t tm[4] = {0u, 0u, 0u, 0u};  // the row's own ancestors, once the tree's chunk comes
      auto load_mask = [&]() {
        if (last_s != sg.s) {
          last_s = sg.s;
          wait(&sh->mready[nmask & 3], (uint32_t)(nmask >> 2));
          ++nmask;
        }
        if (has_row) {
#pragma unroll
          for (int k = 0; k < 4; ++k) tm[k] = sh->mask[(nmask - 1) & 3][node][k];
        }
      };
      for (int c = sg.c0; c < sg.c1; ++c, ++cc) {
        if (NT == 1 && (cc & 1) != t) continue;
        const bool tree = sg.is_tree(c);
        const int nk = sg.keys(c);
        const bool masked = tree || nk < kTtCH;
        if (tree) load_mask();
        if (Q8) wait(&sh->kfr[cc % kTtRing], (uint32_t)(cc / kTtRing));
        wait(&sh->sfull[t], (uint32_t)nj);
        if constexpr (NT == 2) {  // the streams' softmaxes take turns
          if (t == 1) tc::named_bar(7, 256);
          else if (nj > 0) tc::named_bar(6, 256);
        }
        __syncwarp();
        tc::tc_fence_after();
        float cs = a.scale;  // score scale (log2 units)
        // A hidden score is -inf before it is scaled, so no scale may underflow to
        // 0 (NaN): a query's is 2^-106 at least, next to which scores (sums of
        // codes below 2^26, times keys' scales) are 0 all the same, and a tree
        // key's 2^-40 (kTtKeyExp).  (A floor under the products of the two, where
        // scores are hidden: 277 us instead of 265, 32 sequences x 64 rows, 8k.)
        if constexpr (Q8) cs = fmaxf(tt_scale(a.scale, sh->qe[seg_no & 3][NT == 2 ? t : 0][r]), 0x1p-106f);
        if (warp_on) {
          // keys 32 i .. of the chunk that the row sees, as bits
          auto seen = [&](int i) {
            const int n = nk - 32 * i;
            uint32_t w = n >= 32 ? 0xffffffffu : n > 0 ? (1u << n) - 1u : 0u;
            if (tree) w &= i == 0 ? tm[0] : i == 1 ? tm[1] : i == 2 ? tm[2] : tm[3];
            return w;
          };
          constexpr int W = 16, HC = Q8 ? 32 : 64;  // columns per step, per part
          auto hide = [&](float (&x)[W], int i) {  // columns W i ..
            if (masked) {
              const uint32_t w = seen(i * W >> 5) >> (W * i & 31);
#pragma unroll
              for (int k = 0; k < W; ++k) x[k] = (w >> k) & 1u ? x[k] : -INFINITY;
            }
          };
          const float4* kf4 = reinterpret_cast<const float4*>(sh->kf[cc & 3]);
          // the keys' scales of step i; read a step ahead (shared memory is busy
          // with the products' operands, and a wait for scores holds loads back)
          struct Scales {
            float4 f[Q8 ? W / 4 : 1];
          };
          auto load_kf = [&](int i, Scales& f) {
            if constexpr (Q8) {
#pragma unroll
              for (int k = 0; k < W / 4; ++k) f.f[k] = kf4[i * (W / 4) + k];
            }
          };
          auto scale2 = [&](const Scales& f, int k) {  // the score scales of columns 2 k, 2 k + 1
            const unsigned long long cs2 = tt_pair(cs, cs);
            if constexpr (Q8) {
              const float4& y = f.f[k >> 1];
              return tt_mul2(k & 1 ? tt_pair(y.z, y.w) : tt_pair(y.x, y.y), cs2);
            } else {
              return cs2;
            }
          };
          auto cols_max = [&](int i0, int n) {  // the largest score of n steps
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            float x[W];
#pragma unroll 1
            for (int i = i0; i < i0 + n; ++i) {
              Scales f;
              tmem_ld_async(ts + W * i, x);
              load_kf(i, f);
              tmem_wait(x);
#pragma unroll
              for (int k = 0; k < W; k += 2) tt_unpair(tt_mul2(tt_pair(x[k], x[k + 1]), scale2(f, k / 2)), x[k], x[k + 1]);
              hide(x, i);
#pragma unroll
              for (int k = 0; k < W; k += 2) m4[(k >> 1) & 3] = fmaxf(fmaxf(m4[(k >> 1) & 3], x[k]), x[k + 1]);
            }
            return fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          };
          unsigned long long sa, sb;
          // weights 2^(scale x + m0) of a step, as the product takes them (W / 2
          // columns of their first parts, then what those left), and their sums; `next` starts
          // the next step's loads once the scores have been taken
          auto piece = [&](float (&x)[W], const Scales& f, uint32_t* pk, float m0, auto next) {
            const unsigned long long m2 = tt_pair(m0, m0);
            unsigned long long y[W / 2];
#pragma unroll
            for (int k = 0; k < W / 2; ++k) y[k] = tt_fma2(tt_pair(x[2 * k], x[2 * k + 1]), scale2(f, k), m2);
            next();
#pragma unroll
            for (int k = 0; k < W / 2; ++k) {
              float lo, hi;
              tt_unpair(y[k], lo, hi);
              lo = tt_ex2(lo);
              hi = tt_ex2(hi);
              if (k & 1) sb = tt_add2(sb, tt_pair(lo, hi));
              else sa = tt_add2(sa, tt_pair(lo, hi));
              tt_split_bf16(lo, hi, pk[k], pk[W / 2 + k]);
            }
          };
          // the weights of the chunk's first n keys
          auto rescale_p = [&](float f, int n) {
            if (!__any_sync(0xffffffffu, f != 1.f)) return;
#pragma unroll 1
            for (int q = 0; q < n / 16; ++q) {
              float w[16];
              uint32_t v[16];
              tc::tmem_ld16(ts + 16 * q, w);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const uint32_t h = __float_as_uint(w[k]), l = __float_as_uint(w[8 + k]);
                const float lo = __uint_as_float(h << 16) + __uint_as_float(l << 16);
                const float hi = __uint_as_float(h & 0xFFFF0000u) + __uint_as_float(l & 0xFFFF0000u);
                tt_split_bf16(lo * f, hi * f, v[k], v[8 + k]);
                if (f == 1.f) v[k] = h, v[8 + k] = l;  // (halfway cases may split the other way round)
              }
              tmem_st16u(ts + 16 * q, v);
            }
          };
          auto rescale = [&](float f) {
            // O holds the stream's chunks before this one: their products
            // precede this chunk's S in the tensor pipe, so they are complete.
            if (nj > nj0 && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
              for (int q = 0; q < D / 16; ++q) {
                float o[16];
                tc::tmem_ld16(to + 16 * q, o);
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] *= f;
                tc::tmem_st16(to + 16 * q, o);
              }
            }
          };
          // a new reference, for a row that needs one: the largest of what it has
          // and of n steps' scores.  (The others keep theirs: a row's result does
          // not depend on the rows that share its warp, lanes without one included.)
          auto refer = [&](int i0, int n, bool needs) {
            const float m_new = fmaxf(cols_max(i0, n), m_run);
            if (!needs) return 1.f;
            const float alpha = m_run == -INFINITY ? 0.f : tt_ex2(m_run - m_new);
            m_run = m_new;
            return alpha;
          };
          // A part of a chunk at a time, whose weights stay in registers until
          // their sum shows that the reference suits them.  (8-bit: 16 warps'
          // 128 registers hold a quarter; what spills goes to L2, for shared
          // memory takes the first-level cache, and doubles the chunk's time.)
          const int np = (nk + HC - 1) / HC;  // parts that hold keys
          float sum0 = 0.f;
#pragma unroll 1
          for (int h = 0; h < np; ++h) {
            uint32_t pk[HC];
            float sum;
            bool again = false, over;
#pragma unroll 1
            for (;;) {
              const float m0 = m_run == -INFINITY ? 0.f : -m_run;
              sa = sb = tt_pair(0.f, 0.f);
              float x[W];
              Scales f;
              tmem_ld_async(ts + HC * h, x);
              load_kf(h * (HC / W), f);
#pragma unroll
              for (int i = 0; i < HC / W; ++i) {  // the next scores arrive while these are exponentiated
                tmem_wait(x);
                hide(x, h * (HC / W) + i);
                piece(x, f, pk + i * W, m0, [&]() {
                  if (i + 1 < HC / W) {
                    tmem_ld_async(ts + HC * h + W * (i + 1), x);
                    load_kf(h * (HC / W) + i + 1, f);
                  }
                });
              }
              float s0, s1;
              tt_unpair(tt_add2(sa, sb), s0, s1);
              sum = s0 + s1;
              // too large for the reference; or a row's first keys, which reference 0 does not suit
              over = sum > 0x1p30f || (m_run == -INFINITY && sum < 0x1p-30f);
              if (again || !__any_sync(0xffffffffu, over && has_row)) break;
              again = true;
              const float alpha = refer(h * (HC / W), HC / W, over);
              rescale(alpha);
              l_run *= alpha;
              if (h) {  // the parts before, stored already
                sum0 *= alpha;
                rescale_p(alpha, HC * h);
              }
            }
            if (!over && m_run == -INFINITY) m_run = 0.f;
            sum0 += sum;
            if (NT == 2 && h == min(1, np - 1)) named_arrive(t == 0 ? 7 : 6, 256);
#pragma unroll
            for (int i = 0; i < HC; i += 32) tmem_st32u(ts + HC * h + i, pk + i);
          }
          l_run += sum0;
        } else if constexpr (NT == 2) {
          named_arrive(t == 0 ? 7 : 6, 256);
        }
        tc::tc_fence_before();
        tc::mbar_arrive(&sh->pdone[t]);
        ++nj;
      }

      // ---- the segment's end: normalise and write, or leave a partial
      if (NT == 1 && has_tree && (nj == nj0 || ((cc - 1) & 1) != t)) load_mask();  // (the other stream had the tree)
      const bool row_ok = !has_tree || (tm[0] | tm[1] | tm[2] | tm[3]) != 0u;
      bool had[2];  // streams with a job in this segment
      had[t] = nj > nj0;
      had[t ^ 1] = NT == 2 ? false : (sg.c1 - sg.c0) > (nj - nj0);
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (had[u]) wait(&sh->ofull[u], (uint32_t)no[u]++);
      __syncwarp();
      tc::tc_fence_after();
      float M = m_run, L = l_run, f_own = 1.f, f_oth = 0.f;
      if constexpr (NT == 1) {
        sh->xm[t][r] = m_run;
        sh->xl[t][r] = l_run;
        tc::named_bar(4, 256);
        const float mo = sh->xm[t ^ 1][r], lo = sh->xl[t ^ 1][r];
        M = fmaxf(m_run, mo);
        const float ao = mo == -INFINITY ? 0.f : tt_ex2(mo - M), as = m_run == -INFINITY ? 0.f : tt_ex2(m_run - M);
        // (both streams' threads form the same sum: stream 0's term first)
        L = t == 0 ? l_run * as + lo * ao : lo * ao + l_run * as;
        f_own *= as;
        f_oth = ao;
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
        float* part = static_cast<float*>(a.work) +
                      ((size_t)2 * blockIdx.x + (sg.c0 > 0 ? 0 : 1)) * tt_slot_floats<D, NT>();
        const int prow = (NT == 2 ? t * kTtRows : 0) + r;
        // (16 bytes per lane and store, to 32 rows: more cache-line accesses than
        // rows turned among lanes first, but a quarter of the instructions, and
        // nothing else here uses the load/store unit)
        const bool write = has_row && (row_ok || a.zero_pad) && DFL_CHECK(node < a.rows, status);
        uint4* out4 = reinterpret_cast<uint4*>(a.out) + ((size_t)(sg.s * a.rows + node) * a.nq + head) * (D / 8);
        constexpr int W = NCOL < 32 ? NCOL : 32;  // columns per step
#pragma unroll 1
        for (int q = 0; q < NCOL / W; ++q) {
          const int col = col0 + W * q;
          float o[W];
#pragma unroll
          for (int k = 0; k < W; ++k) o[k] = 0.f;
          __syncwarp();  // the loads below are warp-collective
          // stream 0's term first whichever thread adds them (NT = 1)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const bool own = u == t;
            if (NT == 2 && !own) continue;
            if (!had[u]) continue;
            const float f = own ? f_own : f_oth;
#pragma unroll
            for (int e = 0; e < W / 16; ++e) {
              float x[16];
              tc::tmem_ld16(lane_base + 256 + u * 128 + col + 16 * e, x);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[16 * e + k] = fmaf(x[k], f, o[16 * e + k]);
            }
          }
          if (any_bad) {  // visible NaN or infinite values: added as they are
            for (int i = 0; i < 4; ++i)
              for (uint32_t b = bad[i]; b; b &= b - 1) {
                const int j = 32 * i + __ffs(b) - 1;
                const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(a.vb) +
                                         (((size_t)sg.s * a.rows + j) * a.nkv + g) * D + col;
#pragma unroll
                for (int k = 0; k < W; ++k) {
                  const float f = __bfloat162float(v[k]);
                  if (!(fabsf(f) < INFINITY)) o[k] += f;
                }
              }
          }
          __syncwarp();
          if (whole) {
            if (write) {
#pragma unroll
              for (int k = 0; k < W / 8; ++k)
                out4[col / 8 + k] = !row_ok ? make_uint4(0, 0, 0, 0)
                                            : make_uint4(tt_pack(o[8 * k], o[8 * k + 1]), tt_pack(o[8 * k + 2], o[8 * k + 3]),
                                                         tt_pack(o[8 * k + 4], o[8 * k + 5]),
                                                         tt_pack(o[8 * k + 6], o[8 * k + 7]));
            }
          } else if (has_row) {
            float4* p4 = reinterpret_cast<float4*>(part) + (size_t)(prow >> 7) * (kTtRows * D / 4);
#pragma unroll
            for (int k = 0; k < W / 4; ++k)
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
      // both outputs have been read before either stream goes on
      if constexpr (NT == 1) tc::named_bar(4, 256);
    }
    if (NT == 2 && t == 0 && nj > 0) tc::named_bar(6, 256);  // meets stream 1's last arrival
  } else {
    // ---------------------------------------------------- 8-bit cache: V's codes and the tree's rows to operands
    // (after a wait gave up the loops run on without work, to meet the barriers)
    if constexpr (Q8) {
      const int ct = tid - 384;
      constexpr int LPR = D / 16;                     // lanes per code row (16 codes each)
      constexpr int RPP = 128 / LPR, NP = 128 / RPP;  // rows per pass, passes
      const int cr = ct / LPR, pc = ct % LPR;
      int i = 0, nr = 0, nt = 0;              // chunks, raw chunks, trees
      float kfn = 1.f, vfn = 0.f;             // the next chunk's scales of row ct
      auto load_exp = [&](int c, int g) {
        bool badp = false;
        const size_t row = (size_t)km.row0(sg.s, c * kTtCH, &badp) + (size_t)g * km.head_rows() + ct;
        const bool in = ct < sg.keys(c);
        kfn = in ? __int_as_float((int)__ldg(a.k_exp + row) << 23) : 1.f;  // (a hidden key: any finite scale)
        vfn = in ? __int_as_float((int)__ldg(a.v_exp + row) << 23) : 0.f;
      };
      for (bool on = sg.begin(&a, ips, sh); on; on = sg.next()) {
        const int g = sg.it / p.n_pt;
        for (int c = sg.c0; c < sg.c1; ++c, ++i) {
          const int nk = sg.keys(c), slot = i % NSV;
          uint8_t* dst = Vs + slot * TILE;
          if (!sg.is_tree(c)) {
            if (c == sg.c0) load_exp(c, g);
            const float kf = kfn, vf = vfn;
            if (c + 1 < sg.c1 && !sg.is_tree(c + 1)) load_exp(c + 1, g);
            sh->kf[i & 3][ct] = kf;
            tc::mbar_arrive(&sh->kfr[i % kTtRing]);
            sh->fac[i & 1][ct] = vf;          // (its readers two chunks ago are past the last chunk's barrier)
            tc::named_bar(5, 128);
            const int rs = nr % Cfg::NRV;
            const uint8_t* raw = Rv + rs * RAW + cr * D + pc * 16;
            const float* fac = sh->fac[i & 1] + cr;
            if (i >= NSV) wait_warp(&sh->vempty[slot], (uint32_t)(i / NSV - 1));
            if (wait_warp(&sh->rvfull[rs], (uint32_t)(nr / Cfg::NRV))) {
              // all reads of the tile before the first write (one warp per
              // scheduler: nothing else hides their latency); rows past the
              // last key zero, their codes may be the NaN code
              uint4 code[NP];
              float f[NP];
#pragma unroll
              for (int b = 0; b < NP; ++b) {
                if (b * RPP >= nk) break;  // (the product reads 16 keys at a time, a pass's rows or half of them)
                code[b] = *reinterpret_cast<const uint4*>(raw + b * RPP * D);
                f[b] = fac[b * RPP];
              }
              // (the next copy into the slot is the async proxy's: without a fence
              // the last rows' reads came behind it)
              tc::fence_proxy_async_smem();
              tc::mbar_arrive(&sh->rvempty[rs]);
#pragma unroll
              for (int b = 0; b < NP; ++b) {
                if (b * RPP >= nk) break;
                const int row = b * RPP + cr;
                uint4 lo, hi;
                if (row >= nk) code[b] = make_uint4(0, 0, 0, 0);
                tt_codes_to_bf16(code[b], f[b], lo, hi);
                *reinterpret_cast<uint4*>(dst + tt_off(row, 2 * pc)) = lo;
                *reinterpret_cast<uint4*>(dst + tt_off(row, 2 * pc + 1)) = hi;
              }
              tc::fence_proxy_async_smem();
              tc::mbar_arrive(&sh->vfull[slot]);
            }
            ++nr;
          } else {
            // the tree's bf16 rows: K as two e4m3 codes with a scale per row, V
            // as it is.  Eight 16-byte pieces per thread and round, in flight
            // at once.
            constexpr int CPR = D / 8, RS = 128 / CPR, U = 8, RN = RS * U;  // rows per step, per round
            const size_t rstr = (size_t)a.nkv * D;
            const size_t off = ((size_t)sg.s * a.rows * a.nkv + g) * D + (size_t)(ct / CPR) * rstr + (ct % CPR) * 8;
            uint4 x[U];
            auto load_rows = [&](int v, int r0) {
              const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(v ? a.vb : a.kb) + off;
#pragma unroll
              for (int u = 0; u < U; ++u)  // (zeros past the last row)
                x[u] = r0 + u * RS + ct / CPR < nk ? __ldg(reinterpret_cast<const uint4*>(src + (size_t)(r0 + u * RS) * rstr))
                                                   : make_uint4(0, 0, 0, 0);
            };
            auto unpack = [](const uint4& w, float (&y)[8]) {
              const __nv_bfloat162* b2 = reinterpret_cast<const __nv_bfloat162*>(&w);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float2 f = __bfloat1622float2(b2[k]);
                y[2 * k] = f.x;
                y[2 * k + 1] = f.y;
              }
            };
            if (nt > 0) wait_warp(&sh->tkempty, (uint32_t)(nt - 1));
            if (ct >= nk) sh->kf[i & 3][ct] = 1.f;  // (a hidden key: any finite scale, for -inf times it)
#pragma unroll 1
            for (int r0 = 0; r0 < nk; r0 += RN) {
              load_rows(0, r0);
#pragma unroll
              for (int u = 0; u < U; ++u) {
                if (r0 + u * RS >= nk) break;
                const int row = r0 + u * RS + ct / CPR;
                float y[8];
                unpack(x[u], y);
                float m = tt_finite_max(y);
#pragma unroll
                for (int o = CPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                const int e = max(tt_exp8_of(m), kTtKeyExp);
                uint2 hi, lo;
                tt_split8(y, e, hi, lo);
                uint8_t* q = Ts + tt_off8<D>(row, (ct % CPR) >> 1) + (ct & 1) * 8;
                *reinterpret_cast<uint2*>(q) = hi;
                *reinterpret_cast<uint2*>(q + RAW) = lo;
                if (ct % CPR == 0 && row < nk) sh->kf[i & 3][row] = __int_as_float((127 + e) << 23);
              }
            }
            tc::fence_proxy_async_smem();
            tc::mbar_arrive(&sh->tkfull[NT == 1 ? i & 1 : 0]);
            tc::mbar_arrive(&sh->kfr[i % kTtRing]);
            ++nt;
            load_rows(1, 0);
            if (ct < 4) sh->badv[i % kTtRing][ct] = 0u;
            tc::named_bar(5, 128);
            if (i >= NSV) wait_warp(&sh->vempty[slot], (uint32_t)(i / NSV - 1));
            if (ok) {
#pragma unroll 1
              for (int r0 = 0; r0 < nk; r0 += RN) {
                if (r0 > 0) load_rows(1, r0);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                  const int row = r0 + u * RS + ct / CPR;
                  if (r0 + u * RS >= (nk + 15 & ~15)) break;  // (the product reads 16 keys at a time)
                  // a NaN or infinity must not meet a hidden row's weight 0
                  if (tt_odd(x[u])) {
                    x[u] = tt_clear_odd(x[u]);
                    atomicOr(&sh->badv[i % kTtRing][row >> 5], 1u << (row & 31));
                  }
                  *reinterpret_cast<uint4*>(dst + tt_off(row, ct % CPR)) = x[u];
                }
              }
              tc::fence_proxy_async_smem();
              tc::mbar_arrive(&sh->vfull[slot]);
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

// Joins the partials of the items that several CTAs shared.  Grid: y = the
// item's first boundary between runs (flat) or the item (aligned), so that
// only shared items' warps do anything; x = (32 rows, CW columns) of the
// item, one warp each: lanes are rows, so the partials' reads are 512
// contiguous bytes; the loads of U partials are in flight at once.
template <int D, int NT, int CW, int U>
__global__ void __launch_bounds__(128) tree_tc_merge_kernel(const __grid_constant__ TreeAttnDesc a, int n_pt, int nb) {
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int ips = a.nkv * n_pt, grp = a.nq / a.nkv, nqv = a.rows * grp;
  constexpr int CG = D / CW;
  const int w = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int cg = w % CG, rg = w / CG;
  // Which item, if any: found beside the attention kernel's last CTAs, for the
  // lengths it goes by were there before that kernel's own wait ended.
  int s = 0, it = 0, b0 = 0, b1 = 0;
  if (rg < min(NT * 4, (nqv + 31) / 32)) {
    const Part pt = tt_part(a, ips, nb, nullptr);
    if (pt.aligned) {
      const Spot sp = tt_run(a, ips, blockIdx.y, pt);
      if (sp.s < a.n_seqs && sp.c == 0) {  // an item's first run
        s = sp.s;
        it = sp.it;
        b0 = blockIdx.y;
        b1 = b0 + (sp.nch - 1) / pt.per;
      }
    } else {
      const int per = pt.per, x = (int)(blockIdx.y + 1) * per;
      if (x < pt.total) {
        const Spot sp = tt_locate(a, ips, x, 0);
        const int X = x - sp.c + tt_setup(a);  // the item's chunks are [X, X + nch)
        if (x > X && X / per == (int)blockIdx.y) {  // an item is cut here, for the first time
          s = sp.s;
          it = sp.it;
          b0 = blockIdx.y;
          b1 = (X + sp.nch - 1) / per;
        }
      }
    }
  }
  pdl_wait();  // (every CTA: who waits for this kernel waits for the attention too)
  if (b0 == b1) return;  // none, or written by its CTA
  const int g = it / n_pt, qv = (it % n_pt) * (NT * kTtRows) + rg * 32 + lane;
  if (qv - lane >= nqv) return;
  const int tile = rg >> 2, prow = (rg & 3) * 32 + lane;
  constexpr int ML = NT * kTtRows * D;
  const int mrow = ML + tile * kTtRows + prow;
  const size_t orow = (size_t)tile * (kTtRows * D) + ((size_t)(cg * (CW / 4)) * kTtRows + prow) * 4;
  float M = -INFINITY, L = 0.f, o[CW], last = 0.f;
#pragma unroll
  for (int k = 0; k < CW; ++k) o[k] = 0.f;
#pragma unroll 1
  for (int b = b0; b <= b1; b += U) {
    float4 v[U][CW / 4];
    float mb[U], lb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int bb = b + u;
      mb[u] = -INFINITY;
      lb[u] = 0.f;
#pragma unroll
      for (int k = 0; k < CW / 4; ++k) v[u][k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (bb > b1) continue;
      // slot 0: the item began in an earlier CTA
      const float* sl = static_cast<const float*>(a.work) + ((size_t)2 * bb + (bb > b0 ? 0 : 1)) * tt_slot_floats<D, NT>();
#pragma unroll
      for (int k = 0; k < CW / 4; ++k) v[u][k] = *reinterpret_cast<const float4*>(sl + orow + (size_t)4 * k * kTtRows);
      mb[u] = sl[mrow];
      lb[u] = sl[mrow + NT * kTtRows];
    }
    float Mn = M;
#pragma unroll
    for (int u = 0; u < U; ++u) Mn = fmaxf(Mn, mb[u]);
    const float x = M == -INFINITY ? 0.f : tt_ex2(M - Mn);
    M = Mn;
    L *= x;
#pragma unroll
    for (int k = 0; k < CW; ++k) o[k] *= x;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float y = mb[u] == -INFINITY ? 0.f : tt_ex2(mb[u] - M);
      L = fmaf(lb[u], y, L);
#pragma unroll
      for (int k = 0; k < CW / 4; ++k) {
        o[4 * k] = fmaf(v[u][k].x, y, o[4 * k]);
        o[4 * k + 1] = fmaf(v[u][k].y, y, o[4 * k + 1]);
        o[4 * k + 2] = fmaf(v[u][k].z, y, o[4 * k + 2]);
        o[4 * k + 3] = fmaf(v[u][k].w, y, o[4 * k + 3]);
      }
      if (b + u == b1) last = lb[u];  // the tree's partial: negative in a padding row
    }
  }
  if (qv >= nqv || (last < 0.f && !a.zero_pad)) return;
  const float inv = L > 0.f ? 1.f / L : L == L ? 0.f : L;
  const int node = qv / grp, head = g * grp + qv % grp;
  uint4* out = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.out) + ((size_t)s * a.rows + node) * a.nq * D +
                                        (size_t)head * D + cg * CW);
#pragma unroll
  for (int k = 0; k < CW / 8; ++k)
    out[k] = last < 0.f ? make_uint4(0, 0, 0, 0)
                        : make_uint4(tt_pack(o[8 * k] * inv, o[8 * k + 1] * inv), tt_pack(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                                     tt_pack(o[8 * k + 4] * inv, o[8 * k + 5] * inv),
                                     tt_pack(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
}

template <int D, int NT, bool Q8>
cudaError_t tt_launch(const TreeAttnDesc& a, int num_sms, cudaStream_t st) {
  using Cfg = TtCfg<D, NT, Q8>;
  TtTma p;
  p.a = a;
  const int nqv = a.rows * (a.nq / a.nkv);
  p.n_pt = (nqv + NT * kTtRows - 1) / (NT * kTtRows);
  const uint32_t grp = a.nq / a.nkv;
  p.grp_mul = grp >= 2 && grp <= 256 ? (uint32_t)((0x100000000ull + grp - 1) / grp) : 0u;
  const uint64_t rows = a.pages ? (uint64_t)a.pool * a.nkv * a.ps : (uint64_t)a.n_seqs * a.nkv * a.cap;
  bool okm;
  if (Q8) {
    okm = make_tmap_u8(&p.kc, a.kc, D, rows, kTtCH, true) && make_tmap_u8(&p.vc, a.vc, D, rows, kTtCH);
    p.kb = p.kc;
    p.vb = p.vc;
  } else {
    const uint64_t M = (uint64_t)a.n_seqs * a.rows;
    okm = make_tmap_bf16(&p.kc, a.kc, D, rows, kTtCH) && make_tmap_bf16(&p.vc, a.vc, D, rows, kTtCH) &&
          make_tmap3_bf16(&p.kb, a.kb, D, a.nkv, M, 1, kTtCH) && make_tmap3_bf16(&p.vb, a.vb, D, a.nkv, M, 1, kTtCH);
  }
  p.q_tma = kTtRows % grp == 0;
  if (p.q_tma)
    okm = okm && make_tmap3_bf16(&p.q3, a.q, D, a.nq, (uint64_t)a.n_seqs * a.rows, grp, kTtRows / grp);
  else
    p.q3 = p.kc;
  if (!okm) return cudaErrorInvalidValue;
  cudaError_t e =
      cudaFuncSetAttribute(tree_tc_kernel<D, NT, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_pdl(tree_tc_kernel<D, NT, Q8>, dim3(num_sms), dim3(Cfg::THREADS), Cfg::SMEM, st, p);
  if (e != cudaSuccess) return e;
  // NT = 1: narrow columns (many warps, few rows a call); NT = 2: wide ones.
  constexpr int CW = NT == 1 ? 8 : 32, U = NT == 1 ? 8 : 2;
  const int warps = (nqv < NT * kTtRows ? (nqv + 31) / 32 : NT * 4) * (D / CW);
  return launch_pdl(tree_tc_merge_kernel<D, NT, CW, U>, dim3((warps + 3) / 4, num_sms), dim3(128), 0, st, a, p.n_pt,
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
