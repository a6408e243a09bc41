// k_prompt_attn_tc.cu -- causal attention of packed prompts on the tcgen05
// tensor cores (bf16).
//
// Work: an item is (sequence, KV head, two query tiles); a tile holds tok =
// 128 / group tokens of the group's query heads (row = token * group + head),
// so that K and V of a chunk serve 2 tok tokens x group heads whatever the
// group.  An item's chunks are the 128-slot chunks of the cached context, then
// those of the sequence's own rows up to the item's last token.  The chunks of
// all items in a row are cut into equal runs, one per CTA (one CTA per SM), so
// the causal triangle, ragged lengths and few long contexts balance alike.  A
// CTA walks its run as segments (the part of one item inside the run): a whole
// item is normalised and written at once, the first and the last segment may
// leave a partial (O, m, l); the CTA that leaves an item's last one joins them,
// in their order, or a second kernel does (pt_apart).
//
// Where sequences have at most a tile of rows (single tokens, short prompts over
// long contexts) an item is one tile, whose chunks the streams take in turn:
// two chunks are under way at once, and the streams' outputs are joined from
// tensor memory at the segment's end.  An empty second tile would cost its
// products all the same: 64 single tokens over 4096 slots 171 us instead of 314
// (94% of the copy rate), one over 131072 92 instead of 162.
//
// Two streams per CTA, one per query tile, each an online softmax with its own
// score and output accumulators in tensor memory (S 128 + O D columns).  Per
// chunk and stream (128 query vectors x 128 keys):
//   S = Q K^T        tcgen05.mma, both operands in shared memory
//   P = 2^(c S - m)  one thread per query vector, written over S
//   O += P V         tcgen05.mma, P from tensor memory, V MN-major
// The streams' softmaxes take turns, so that one stream's products run beside
// the other's softmax.  Bound: the chain of a stream.  A chunk of both streams
// takes 4.1k cycles (8k tokens, 32 / 8 heads), its products 3.0k (61 a product,
// the tensor core's rate); the chain is softmax 1750, store and hand-over 290,
// P V 980, the next S 520, commits and wake-ups 500.  8k tokens: 552 us at the
// power limit, 1.0 PFLOP/s of the formula's, 1.5 of those executed (512 to 515 in
// short loops, where the other figures were taken: without any softmax arithmetic
// 444; scores in steps of 16 columns instead of 32: 560).  Slower too: scores of
// 64 keys ahead in two buffers a stream without turns (584 where this then took 558: a product 64
// columns wide takes almost as long as one of 128); P V of a chunk's first half
// beside the softmax of its second (563, 548); two threads a row (619, 548);
// the output by four warps of its own (553, 509: with 512 threads 128 registers
// are left to each).
// The reference m stays while the weights suit bf16 (which has fp32's
// exponents) and the sums: it starts at 0 where a row's first half chunk sums to
// 2^-30 at least, and stays while all of the row's weights sum to 2^30 at most,
// so the usual chunk needs no maximum and no rescaling of O.  Otherwise the half
// chunk is done again with a new reference: its maximum, or log2 of the row's
// sum so far, which is no less than the maximum of what the row has seen.  Sums
// of outputs are thus at most 2^30 max|v|, and 2^39 max|v| where the parts of all
// CTAs are joined: values up to 2^88 do not overflow on the way, over any number
// of keys.  (2^22 instead of 2^30, for values up to 2^96, takes new references
// more often: 8k tokens with scores of standard deviation 1 / 3 / 4: 515 / 531 /
// 536 us with 2^30, 515 / 546 / 1018 with 2^22.)
//
// The softmax is no rounding point: the weights enter their product as two
// bf16 operands, P = P_hi + P_lo (2^-16 relative), whose products share V's
// tile and the accumulator.  The sum l uses the unrounded weights.
//
// What a row does not see may hold anything.  Scores are hidden by selection;
// values meet a weight of 0, and 0 * NaN is NaN, so one warp goes over the V
// tiles that some row of the item sees in part: rows behind the context's or
// the item's end are cleared, NaN and infinite elements of the others are
// cleared and noted, and added to the rows that see them when the segment ends.
//
// Roles: warp 0 K/V copies; warps 1, 2 the products of stream 0, 1; warp 3
// query copies and V tiles; warps 4..11 the softmax, a query vector per thread.
#include <math.h>

#include <algorithm>

#include "attn_tc.cuh"
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "prompt_attn.cuh"
#include "tc_ptx.cuh"
#include "tmap.h"

namespace dfl {

namespace {

constexpr int kPtCH = 128;    // keys per chunk
constexpr int kPtRows = 128;  // query vectors per tile
constexpr int kPtRing = 8;    // chunks whose bad rows are kept
constexpr float kPtMost = 0x1p30f, kPtFew = 0x1p-30f;  // sums of weights that a reference suits (header)
// Positions of a run at least: shorter ones share an item of few chunks among
// many CTAs (seven prompts of up to 33 rows over 131 slots: 12.0 us with 1, 10.1
// with 4, 14.4 with 6).
constexpr int kPtLeast = 4;
constexpr int kPtLeastOne = 2;  // of items of one tile (16 rows over 2048 slots: 19.5 / 16.2 / 16.8 / 18.8 us with 1 / 2 / 4 / 6)
// Positions an item has before its chunks', for what it costs besides them (16
// prompts of 229 to 3401 tokens: 681 / 660 / 680 / 698 us with 1 / 2 / 3 / 4).
constexpr int kPtSetup = 2;

struct PtTma {
  CUtensorMap kc, vc;  // cache rows [..][D], boxes of 64 dims x 128 rows
  CUtensorMap kb, vb;  // own rows [M][nkv][D]
  CUtensorMap q3;      // queries [M][nq][D], box 64 dims x group x tok
  PromptAttnDesc a;
  int grp, tok;        // query heads per KV head, tokens per tile
  uint32_t grp_mul;    // ceil(2^32 / grp) for 2 <= grp, else 0
  int apart;           // shared items are joined by a kernel of their own
};

// The shared item that begins in a CTA, for that kernel.
struct PtItem {
  int row0, n;  // the item's first row, its tokens (0: none)
  int g, b1;    // KV head; the CTA with its last part
};

// r / grp, r < 128.
__device__ __forceinline__ int pt_div_grp(const PtTma& p, int r) {
  return p.grp_mul ? (int)__umulhi((uint32_t)r, p.grp_mul) : r;
}

// TWO: an item has two query tiles, one a stream; otherwise one, whose chunks
// the streams take in turn.
template <int D, bool TWO>
struct PtCfg {
  static constexpr int TILE = kPtCH * D * 2;
  static constexpr int NS = D == 64 ? 4 : 2;  // K slots, V slots
  // Slots of a ring.  With one tile each stream has a ring of its own: who waits
  // on a slot's barrier by parity must have seen its phase before.
  static constexpr int R = TWO ? NS : NS / 2;
  static constexpr int THREADS = 384;
  static constexpr int K_OFF = 2 * TILE;  // behind the streams' query tiles; of one tile: this item's and the next one's
  static constexpr int V_OFF = K_OFF + NS * TILE;
  static constexpr int O_OFF = V_OFF + NS * TILE;  // 2 KB a softmax warp, where it turns its output rows
  static constexpr int M_OFF = O_OFF + 8 * 2048;   // the streams' maxima and sums, [2][2][128] (one tile)
  static constexpr int X_OFF = M_OFF + (TWO ? 0 : 2048);
  static constexpr int X_BYTES = 2048;
  static constexpr size_t SMEM = X_OFF + X_BYTES + 1024;
  static_assert(SMEM <= 232448, "shared memory of one CTA");
};

// sum of floor((a i + b) / m) over i < n (Euclid's steps: few for m = 128).
__device__ __forceinline__ int pt_floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  uint32_t sum = 0;
  for (;;) {
    if (n == 0) return (int)sum;
    if (a >= m) {
      sum += (uint32_t)(((uint64_t)n * (n - 1) >> 1) * (a / m));
      a %= m;
    }
    if (b >= m) {
      sum += n * (b / m);
      b %= m;
    }
    const uint32_t y = a * n + b;
    if (y < m) return (int)sum;
    n = y / m;
    b = y % m;
    const uint32_t x = m;
    m = a;
    a = x;
  }
}

struct PtSeq {
  int row0, n, ctx;  // first row, rows, cached positions
  int cc, T;         // context chunks, items per KV head
  __device__ __forceinline__ void set(const PromptAttnDesc& a, int tt, int r0, int r1, int c) {
    row0 = r0;
    n = r1 - r0;
    ctx = min(max(c, 0), a.max_pos);
    cc = (ctx + kPtCH - 1) / kPtCH;
    T = (n + tt - 1) / tt;
  }
  __device__ __forceinline__ int end(int tt, int t) const { return min(n, (t + 1) * tt); }  // behind item t's last token
  __device__ __forceinline__ int chunks(int tt, int t) const { return cc + (end(tt, t) + kPtCH - 1) / kPtCH; }
  // Positions of items 0 .. t-1 of a KV head.
  __device__ __forceinline__ int before(int tt, int t) const {
    if (t <= 0) return 0;
    const int u = t == T ? t - 1 : t;  // (whole items)
    const int x = u * (kPtSetup + cc) + pt_floor_sum(u, kPtCH, tt, tt + kPtCH - 1);
    return t == T ? x + kPtSetup + chunks(tt, T - 1) : x;
  }
};

struct PtShared {  // after the tiles
  uint32_t badv[kPtRing][4];  // own rows whose V holds a NaN or infinity, by chunk counter
  int odd[kPtRing];           // are there such rows?
  int s0, g0, t0, c0, len;    // the CTA's run: first item, position in it, number of positions
  PtSeq q;                    // the first item's sequence
  int x0, per;                // its first position, positions of a run
  int last;                   // this CTA's partial was its item's last one
  int good;                   // row_start is in order
  uint64_t kfull[4], kempty[4], vfull[4], vempty[4], vraw[4];  // (vraw: a ring of its own)
  uint64_t sfull[2], pdone[2], ofull[2], qfull[2], qfree[2];
  uint32_t tslot;
  int abort;
};

__device__ __forceinline__ PtSeq pt_seq(const PromptAttnDesc& a, int tt, int s, bool* far) {
  const int c = a.base_pos ? __ldg(a.base_pos + s) : 0;
  PtSeq q;
  q.set(a, tt, __ldg(a.row_start + s), __ldg(a.row_start + s + 1), c);
  *far |= q.ctx != c;
  return q;
}

// All positions (one warp); none where row_start leaves [0, M] or decreases.
// status (or null): told of that, and of contexts out of range.  mine: the
// sequence of this lane, of the first 32, and len its positions.
__device__ __forceinline__ int pt_total(const PromptAttnDesc& a, int tt, uint32_t* status, bool* good, PtSeq* mine,
                                        int* len) {
  int t = 0;
  *len = 0;
  bool bad = false, far = false;
  mine->set(a, tt, 0, 0, 0);
  for (int s = threadIdx.x & 31; s < a.n_seqs; s += 32) {
    const PtSeq q = pt_seq(a, tt, s, &far);
    bad |= q.row0 < 0 || q.row0 > a.M || q.n < 0 || q.n > a.M - q.row0;
    if (!bad) t += q.before(tt, q.T) * a.nkv;
    if (s < 32) {
      *mine = q;
      *len = t;
    }
  }
  if ((bad || far) && status) raise_status(status, ST_RANGE);
  *good = !__any_sync(0xffffffffu, bad);
  return *good ? __reduce_add_sync(0xffffffffu, t) : 0;
}

// The item at position x of the flat order, and the position c in it (one
// warp; x below pt_total's result, mine and its length from there).
struct PtSpot {
  int s, g, t, c;
  PtSeq q;
};
__device__ __forceinline__ PtSpot pt_locate(const PromptAttnDesc& a, int tt, int x, const PtSeq& mine, int mine_len) {
  const int lane = threadIdx.x & 31;
  PtSpot p;
  p.s = a.n_seqs;
  p.g = p.t = p.c = 0;
  p.q.set(a, tt, 0, 0, 0);
  int first = 0;
  for (int b = 0; b < a.n_seqs; b += 32) {
    PtSeq q = mine;
    int len = mine_len;
    if (b > 0) {
      bool far = false;
      q.set(a, tt, 0, 0, 0);
      if (b + lane < a.n_seqs) q = pt_seq(a, tt, b + lane, &far);
      len = q.before(tt, q.T) * a.nkv;
    }
    int inc = len;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, first + inc > x);
    if (!hit) {
      first += __shfl_sync(0xffffffffu, inc, 31);
      continue;
    }
    const int w = __ffs(hit) - 1;
    x -= first + __shfl_sync(0xffffffffu, inc - len, w);
    p.s = b + w;
    p.q.row0 = __shfl_sync(0xffffffffu, q.row0, w);
    p.q.n = __shfl_sync(0xffffffffu, q.n, w);
    p.q.ctx = __shfl_sync(0xffffffffu, q.ctx, w);
    p.q.cc = __shfl_sync(0xffffffffu, q.cc, w);
    p.q.T = __shfl_sync(0xffffffffu, q.T, w);
    const int one = __shfl_sync(0xffffffffu, len, w) / a.nkv;  // positions of a KV head
    p.g = x / one;
    x %= one;
    int lo = 0, hi = p.q.T;  // the item lies in [lo, hi): 32 places at a time
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, at = lo + lane * step;
      const unsigned le = __ballot_sync(0xffffffffu, at < hi && p.q.before(tt, at) <= x);
      lo += (__popc(le) - 1) * step;
      hi = min(hi, lo + step);
    }
    p.t = lo;
    p.c = x - p.q.before(tt, lo);
    return p;
  }
  return p;
}

// A CTA's run walked segment by segment; every role keeps its own copy.  UNI: a
// whole warp walks, loaded values go through a reduction, which the compiler
// knows to be the same in every lane.
template <bool UNI>
struct PtSeg {
  const PromptAttnDesc& a;
  const int tt;        // tokens per item
  int left;            // positions of the run not yet walked
  int s, g, t;         // the item
  PtSeq q;
  int end, nch;        // behind the item's last token; its chunks
  int c0, c1;          // the segment's chunks
  __device__ __forceinline__ PtSeg(const PromptAttnDesc& a_, int tt_) : a(a_), tt(tt_) {}
  __device__ __forceinline__ static int same(int x) { return UNI ? __reduce_max_sync(0xffffffffu, x) : x; }
  __device__ __forceinline__ void load() {
    q.set(a, tt, same(__ldg(a.row_start + s)), same(__ldg(a.row_start + s + 1)),
          a.base_pos ? same(__ldg(a.base_pos + s)) : 0);
  }
  __device__ __forceinline__ void item() {
    end = q.end(tt, t);
    nch = q.chunks(tt, t);
  }
  // The part of the current item from position v on, at most `left` positions.
  __device__ __forceinline__ void take(int v) {
    const int n = min(nch + kPtSetup - v, left);
    c0 = max(0, v - kPtSetup);
    c1 = max(0, v + n - kPtSetup);
    left -= n;
  }
  __device__ __forceinline__ bool begin(const PtShared* sh) {
    left = same(sh->len);
    if (left <= 0) return false;
    s = same(sh->s0);
    g = same(sh->g0);
    t = same(sh->t0);
    q.row0 = same(sh->q.row0);
    q.n = same(sh->q.n);
    q.ctx = same(sh->q.ctx);
    q.cc = same(sh->q.cc);
    q.T = same(sh->q.T);
    item();
    take(same(sh->c0));
    return c1 > c0 || next();
  }
  __device__ __forceinline__ bool next() {
    do {
      if (left <= 0) return false;
      if (++t == q.T) {
        t = 0;
        if (++g == a.nkv) {
          g = 0;
          do {
            if (++s >= a.n_seqs) return false;
            load();
          } while (q.T == 0);
        }
      }
      item();
      take(0);
    } while (c1 <= c0);
    return true;
  }
  __device__ __forceinline__ bool own(int c) const { return c >= q.cc; }
  __device__ __forceinline__ int key0(int c) const { return (c - q.cc) * kPtCH; }  // an own chunk's first row
  // Keys of the chunk that some row of the item sees.
  __device__ __forceinline__ int keys(int c) const { return min(kPtCH, own(c) ? end - key0(c) : q.ctx - c * kPtCH); }
  // Does some row of the item see the chunk in part?
  __device__ __forceinline__ bool masked(int c) const {
    return own(c) ? key0(c) + kPtCH - 1 > t * tt : q.ctx - c * kPtCH < kPtCH;
  }
};

// Where a segment's partial lies: slot 0 of CTA b when the item began in an
// earlier CTA, slot 1 when it ends in a later one.  A slot holds D / 4 column
// groups of [128 rows] float4 per tile, then maxima and sums.
template <int D>
__host__ __device__ constexpr size_t pt_slot_floats() {
  return (size_t)2 * kPtRows * (D + 2);
}

// The CTAs' items, behind the slots.
template <int D>
__host__ __device__ __forceinline__ PtItem* pt_items(void* work, int ctas) {
  return reinterpret_cast<PtItem*>(static_cast<float*>(work) + (size_t)2 * ctas * pt_slot_floats<D>());
}

// Joins the partials that CTAs b0 .. b1 left of an item, in their order, by
// warp `warp` of `warps`: a warp takes 32 rows and CW columns at a time, lanes
// are rows, so its reads are 512 contiguous bytes; the loads of U partials are
// in flight at once.
template <int D, bool TWO, int CW, int U>
__device__ __forceinline__ void pt_join(const PtTma& p, const PtItem& it, int b0, int warp, int warps) {
  constexpr int CG = D / CW;
  const int b1 = it.b1;
  const PromptAttnDesc& a = p.a;
  if (!DFL_CHECK(b0 >= 0 && b1 < (int)gridDim.x && it.g >= 0 && it.g < a.nkv, a.status)) return;
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int w = warp; w < (TWO ? 8 : 4) * CG; w += warps) {
    const int rg = w / CG, cg = w % CG, tile = TWO ? rg >> 2 : 0, r = (rg & 3) * 32 + lane;
    const int rt = pt_div_grp(p, r), token = tile * p.tok + rt;
    const bool has_row = rt < p.tok && token < it.n;
    if (!__any_sync(0xffffffffu, has_row)) continue;
    if (!has_row || !DFL_CHECK(it.row0 >= 0 && it.row0 + token < a.M, a.status)) continue;
    const int mrow = 2 * kPtRows * D + tile * kPtRows + r;
    const size_t orow = (size_t)tile * (kPtRows * D) + ((size_t)(cg * (CW / 4)) * kPtRows + r) * 4;
    float M = -INFINITY, L = 0.f, o[CW];
#pragma unroll
    for (int k = 0; k < CW; ++k) o[k] = 0.f;
#pragma unroll 1
    for (int b = b0; b <= b1; b += U) {
      float4 v[U][CW / 4];
      float mb[U], lb[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        mb[u] = -INFINITY;
        lb[u] = 0.f;
#pragma unroll
        for (int k = 0; k < CW / 4; ++k) v[u][k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (b + u > b1) continue;
        // slot 0: the item began in an earlier CTA
        const float* sl =
            static_cast<const float*>(a.work) + ((size_t)2 * (b + u) + (b + u > b0 ? 0 : 1)) * pt_slot_floats<D>();
#pragma unroll
        for (int k = 0; k < CW / 4; ++k)
          v[u][k] = __ldcg(reinterpret_cast<const float4*>(sl + orow + (size_t)4 * k * kPtRows));
        mb[u] = __ldcg(sl + mrow);
        lb[u] = __ldcg(sl + mrow + 2 * kPtRows);
      }
      float Mn = M;
#pragma unroll
      for (int u = 0; u < U; ++u) Mn = fmaxf(Mn, mb[u]);
      const float y = M == -INFINITY ? 0.f : tt_ex2(M - Mn);
      M = Mn;
      L *= y;
#pragma unroll
      for (int k = 0; k < CW; ++k) o[k] *= y;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float e = mb[u] == -INFINITY ? 0.f : tt_ex2(mb[u] - M);
        L = fmaf(lb[u], e, L);
#pragma unroll
        for (int k = 0; k < CW / 4; ++k) {
          o[4 * k] = fmaf(v[u][k].x, e, o[4 * k]);
          o[4 * k + 1] = fmaf(v[u][k].y, e, o[4 * k + 1]);
          o[4 * k + 2] = fmaf(v[u][k].z, e, o[4 * k + 2]);
          o[4 * k + 3] = fmaf(v[u][k].w, e, o[4 * k + 3]);
        }
      }
    }
    const float inv = 1.f / L;  // (every row sees itself: 0 is a row whose scores are all -inf, NaN as 0 / 0)
    uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) +
                                          ((size_t)(it.row0 + token) * a.nq + it.g * p.grp + r - rt * p.grp) * D + cg * CW);
#pragma unroll
    for (int k = 0; k < CW / 8; ++k)
      out[k] = make_uint4(tt_pack(o[8 * k] * inv, o[8 * k + 1] * inv), tt_pack(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                          tt_pack(o[8 * k + 4] * inv, o[8 * k + 5] * inv),
                          tt_pack(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
  }
}

template <int D, bool TWO>
__global__ void __launch_bounds__(PtCfg<D, TWO>::THREADS, 1) prompt_tc_kernel(const __grid_constant__ PtTma p) {
  using Cfg = PtCfg<D, TWO>;
  constexpr int TILE = Cfg::TILE, R = Cfg::R;
  constexpr int STEP = TWO ? 1 : 2;  // a stream's next chunk
  extern __shared__ __align__(1024) uint8_t pt_smem[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(pt_smem) + 1023) & ~uintptr_t(1023));
  uint8_t* Qs = sm;
  uint8_t* Ks = sm + Cfg::K_OFF;
  uint8_t* Vs = sm + Cfg::V_OFF;
  PtShared* sh = reinterpret_cast<PtShared*>(sm + Cfg::X_OFF);
  static_assert(sizeof(PtShared) <= Cfg::X_BYTES, "exchange area");
  volatile int* abort = &sh->abort;

  const PromptAttnDesc& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int grp = p.grp, tt = (TWO ? 2 : 1) * p.tok;
  uint32_t* status = a.status;

  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(&sh->kfull[i], 1);
      tc::mbar_init(&sh->kempty[i], TWO ? 2 : 1);  // the issuers that use it
      tc::mbar_init(&sh->vfull[i], 1);
      tc::mbar_init(&sh->vempty[i], TWO ? 2 : 1);
      tc::mbar_init(&sh->vraw[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sh->sfull[i], 1);
      tc::mbar_init(&sh->pdone[i], 128);
      // the product's commit, and the issuer's own arrival: what the issuer has
      // observed (bad rows) is visible to who waits here
      tc::mbar_init(&sh->ofull[i], 2);
      tc::mbar_init(&sh->qfull[i], 1);
      tc::mbar_init(&sh->qfree[i], TWO ? 1 : 2);
    }
    sh->abort = 0;
    tc::fence_mbar_init();
    tc::tma_prefetch_desc(&p.kb);
    tc::tma_prefetch_desc(&p.vb);
    tc::tma_prefetch_desc(&p.kc);
    tc::tma_prefetch_desc(&p.vc);
    tc::tma_prefetch_desc(&p.q3);
  }
  if (warp == 1) tc::tmem_alloc(&sh->tslot, 512);
  pdl_wait();
  pdl_launch_dependents();
  if (warp == 0) {
    bool good;
    PtSeq mine;
    int mine_len;
    const int total = pt_total(a, tt, blockIdx.x == 0 ? status : nullptr, &good, &mine, &mine_len);
    const int per = max(TWO ? kPtLeast : kPtLeastOne, (total + (int)gridDim.x - 1) / (int)gridDim.x);
    const int x0 = (int)min((long long)blockIdx.x * per, (long long)total), len = min(per, total - x0);
    PtSpot sp;
    sp.s = sp.g = sp.t = sp.c = 0;
    sp.q = mine;
    if (len > 0) sp = pt_locate(a, tt, x0, mine, mine_len);
    if (lane == 0) {
      sh->s0 = sp.s;
      sh->g0 = sp.g;
      sh->t0 = sp.t;
      sh->c0 = sp.c;
      sh->len = sp.s < a.n_seqs ? len : 0;
      sh->q = sp.q;
      sh->x0 = x0;
      sh->per = per;
      sh->good = good;
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (a.pos || a.zero_pad)
    prompt_layer_rows<__nv_bfloat16>(a, sh->good, blockIdx.x * Cfg::THREADS + tid, (long long)gridDim.x * Cfg::THREADS);
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
  if (warp == 0) {
    // ---------------------------------------------------- K/V copies
    if (lane == 0 && !stall) {
      int nk[2] = {0, 0}, nv[2] = {0, 0}, nraw = 0;  // copies issued, by ring; V tiles that warp 3 goes over
      uint32_t parts[2] = {0u, 0u};                  // which of the last V tiles those were
      auto copy = [&](const PtSeg<false>& sg, int c, uint8_t* dst, const CUtensorMap* mo, const CUtensorMap* mc,
                      uint64_t* bar) {
        const bool own = sg.own(c);
        int row = own ? sg.q.row0 + sg.key0(c) : 0;
        if (!own) {
          bool bad = false;
          row = (int)(km.row0(sg.s, c * kPtCH, &bad) + (uint32_t)sg.g * (uint32_t)km.head_rows());
          if (bad) raise_status(status, ST_RANGE);  // reads page 0 instead
        }
        if (!DFL_CHECK((uint32_t)row < (own ? (uint32_t)a.M : (uint32_t)(a.pages ? a.pool : a.n_seqs) * a.nkv * km.head_rows()),
                       status))
          row = 0;
        tc::mbar_arrive_expect_tx(bar, TILE);
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          if (own) tc::tma_load_3d(dst + h * (kPtCH * 128), mo, 64 * h, sg.g, row, bar);
          else tma_load_2d_plain(dst + h * (kPtCH * 128), mc, 64 * h, row, bar);
        }
      };
      auto ring = [&](const PtSeg<false>& sg, int c) { return TWO ? 0 : (c - sg.c0) & 1; };
      auto copy_k = [&](const PtSeg<false>& sg, int c) {
        const int x = ring(sg, c), slot = x * R + nk[x] % R;
        if (nk[x] >= R && !wait(&sh->kempty[slot], (uint32_t)(nk[x] / R - 1))) return false;
        copy(sg, c, Ks + slot * TILE, &p.kb, &p.kc, &sh->kfull[slot]);
        ++nk[x];
        return true;
      };
      auto copy_v = [&](const PtSeg<false>& sg, int c) {
        const int x = ring(sg, c), slot = x * R + nv[x] % R;
        if (nv[x] >= R && !wait(&sh->vempty[slot], (uint32_t)(nv[x] / R - 1))) return false;
        const bool part = sg.masked(c);  // warp 3 goes over it and passes it on
        parts[x] = parts[x] << 1 | (part ? 1u : 0u);
        copy(sg, c, Vs + slot * TILE, &p.vb, &p.vc, part ? &sh->vraw[nraw++ & 3] : &sh->vfull[slot]);
        ++nv[x];
        return true;
      };
      PtSeg<false> sg(a, tt);
      bool on = sg.begin(sh);
      if constexpr (TWO) {
        for (; on && ok; on = sg.next())
          for (int c = sg.c0; c < sg.c1 && ok; ++c)
            if (!copy_k(sg, c) || !copy_v(sg, c)) break;
      } else {
        // K(c + 1) before V(c), the order in which their slots come free: after
        // the scores of chunk c - 1, after the other stream's output of c - 2
        PtSeg<false> kg(sg);
        bool k_on = on;
        int c = sg.c0, k = sg.c0;
        auto step = [](PtSeg<false>& g, int& i, bool& go) {
          if (++i == g.c1) {
            go = g.next();
            i = g.c0;
          }
        };
        if (k_on && copy_k(kg, k)) step(kg, k, k_on);
        while (on && ok) {
          if (k_on) {
            if (!copy_k(kg, k)) break;
            step(kg, k, k_on);
          }
          if (!copy_v(sg, c)) break;
          step(sg, c, on);
        }
      }
      // every copy has landed before the CTA's shared memory goes away
#pragma unroll
      for (int x = 0; x < (TWO ? 1 : 2); ++x) {
        for (int i = max(0, nk[x] - R); i < nk[x]; ++i)
          tc::mbar_wait(&sh->kfull[x * R + i % R], (uint32_t)(i / R) & 1u, nullptr, lim_ns);
        for (int i = max(0, nv[x] - R); i < nv[x]; ++i)
          if (!(parts[x] >> (nv[x] - 1 - i) & 1u))
            tc::mbar_wait(&sh->vfull[x * R + i % R], (uint32_t)(i / R) & 1u, nullptr, lim_ns);
      }
      for (int i = max(0, nraw - Cfg::NS); i < nraw; ++i)
        tc::mbar_wait(&sh->vraw[i & 3], (uint32_t)(i >> 2) & 1u, nullptr, lim_ns);
    }
  } else if (warp == 1 || warp == 2) {
    // ---------------------------------------------------- MMA issue, stream t
    // The whole warp walks the stream's jobs, so that descriptors and
    // addresses stay in uniform registers; one lane issues.
    const int t = warp - 1;
    constexpr uint32_t idS = tc::idesc_bf16_f32(kPtRows, kPtCH);
    constexpr uint32_t idV = tc::idesc_bf16_f32_bmn(kPtRows, D);
    const uint32_t ut = __reduce_max_sync(0xffffffffu, (uint32_t)t);
    const uint64_t dq = tc::sdesc_sw128(tc::smem_u32(Qs) + (TWO ? ut * TILE : 0u)), dk = tc::sdesc_sw128(tc::smem_u32(Ks)),
                   dv = tc::sdesc_sw128_mn(tc::smem_u32(Vs), kPtCH * 128, 1024);
    const uint32_t tm_s = __reduce_max_sync(0xffffffffu, tmem) + ut * 128u, tm_o = tm_s + 256u;
    // S of the stream's next job is issued right behind P V of the job
    // before, whose P lies in the same columns.
    PtSeg<true> ss(a, tt), sg(a, tt);  // the S side's segment, the P V side's
    int sc = 0, c = 0;           // its chunk counter and chunk
    int s_seg = 0, q_seen = -1;  // segment; the last one whose queries have been waited for
    bool s_on = ss.begin(sh);
    if (s_on) c = ss.c0 + (TWO ? 0 : t);
    const int ring = TWO ? 0 : (int)ut * R;  // the stream's first slot
    auto qt = [&]() { return TWO ? t : s_seg & 1; };  // query buffer, and its phase
    auto qph = [&]() { return (uint32_t)(TWO ? s_seg : s_seg >> 1); };
    auto next_seg = [&]() {
      ++s_seg;
      s_on = ss.next();
      c = ss.c0 + (TWO ? 0 : t);
    };
    auto wait_s = [&]() {  // the operands of the next S
      if constexpr (!TWO) {
        while (s_on && c >= ss.c1) {  // the segment's one chunk is the other stream's
          q_seen = s_seg;
          if (!wait_warp(&sh->qfull[qt()], qph())) return;
          if (lane == 0) tc::mbar_arrive(&sh->qfree[qt()]);
          next_seg();
        }
        if (!s_on) return;
      }
      if (q_seen < s_seg) {
        q_seen = s_seg;
        if (!wait_warp(&sh->qfull[qt()], qph())) return;
      }
      wait_warp(&sh->kfull[ring + sc % R], (uint32_t)(sc / R));
    };
    auto issue_s = [&]() {
      if (!ok || (!TWO && !s_on)) return;
      const int slot = ring + sc % R;
      tc::tc_fence_after();
      const uint64_t k = dk + (uint64_t)(slot * TILE / 16), q = TWO ? dq : dq + (uint64_t)((s_seg & 1) * TILE / 16);
      const bool q_last = c + STEP >= ss.c1;
      if (tt_elect()) {
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          constexpr int kBox = kPtCH * 128 / 16;  // descriptor addresses count 16 bytes
          const uint64_t off = (uint64_t)((j >> 2) * kBox + (j & 3) * 2);
          tc::mma_bf16(tm_s, q + off, k + off, idS, j > 0 ? 1u : 0u);
        }
        tc::mma_commit(&sh->sfull[t]);
        tc::mma_commit(&sh->kempty[slot]);
        if (q_last) tc::mma_commit(&sh->qfree[qt()]);  // the segment's query tile has been read
      }
      __syncwarp();
      ++sc;
      c += STEP;
      if (q_last) next_seg();
    };
    if (s_on) {
      wait_s();
      issue_s();
    }
    int vc = 0;
    for (bool on = sg.begin(sh); on && ok; on = sg.next()) {
      uint32_t acc0 = 0u;  // the segment's first P V starts the accumulator
      for (int x = sg.c0 + (TWO ? 0 : t); x < sg.c1 && ok; x += STEP, ++vc) {
        const int slot = ring + vc % R, nk = sg.keys(x);
        if (!wait_warp(&sh->vfull[slot], (uint32_t)(vc / R))) break;
        // waited for early, so that S follows P V in the tensor pipe without a
        // gap; not across segments, whose query load may still take a while, nor
        // of one tile, where K comes late (single tokens over 1000 slots, heads of
        // 64: 37 us, 39 with the wait; over 4096 162 and 158)
        const bool last = x + STEP >= sg.c1;
        if (TWO && !last && s_on) wait_s();
        if (!wait_warp(&sh->pdone[t], (uint32_t)vc)) break;
        tc::tc_fence_after();
        const uint64_t v = dv + (uint64_t)(slot * TILE / 16);
        if (tt_elect()) {
#pragma unroll
          for (int j = 0; j < kPtCH / 16; ++j)  // (16 keys a step; of a short chunk only those that hold some)
            if (16 * j < nk) {
              mma_ts(tm_o, tm_s + 16 * j, v + (uint64_t)(j * 128), idV, j > 0 ? 1u : acc0);
              mma_ts(tm_o, tm_s + 16 * j + 8, v + (uint64_t)(j * 128), idV, 1u);  // what P's first part left
            }
          if (last) {  // the segment's output is complete
            tc::mma_commit(&sh->ofull[t]);
            tc::mbar_arrive(&sh->ofull[t]);
          }
        }
        __syncwarp();
        acc0 = 1u;
        // V's slot is given back behind S, for which the softmax waits; but ahead
        // of a wait that may pass over segments, whose V comes into the slot
        if (!TWO && tt_elect()) tc::mma_commit(&sh->vempty[slot]);
        if (s_on) {
          if (!TWO || last) wait_s();
          issue_s();
        }
        if (TWO && tt_elect()) tc::mma_commit(&sh->vempty[slot]);
        __syncwarp();
      }
    }
  } else if (warp == 3) {
    // ---------------------------------------------------- queries, V tiles seen in part
    PtSeg<false> sg(a, tt);
    int n = 0, vc = 0, v0 = 0, v1 = 0, nraw = 0, loads = 0;  // (loads: to buffers 0 and 1 in turn)
    const uint32_t qbytes = (uint32_t)(D / 64) * (uint32_t)(grp * p.tok) * 128u;
    // (tokens past the sequence's last: other rows' queries or zeros, whose results are not used)
    auto load_q = [&](const PtSeg<false>& x, int b, int t) {
      if (lane == 0) {
        ++loads;
        tc::mbar_arrive_expect_tx(&sh->qfull[b], qbytes);
        const int tok = x.q.row0 + x.t * tt + t * p.tok;
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          tc::tma_load_3d(Qs + b * TILE + h * (kPtRows * 128), &p.q3, 64 * h, x.g * grp, tok, &sh->qfull[b]);
      }
    };
    for (bool on = sg.begin(sh); on && ok; on = sg.next(), ++n) {
      PtSeg<false> nx(sg);
      if constexpr (TWO) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (n > 0 && !wait_warp(&sh->qfree[t], (uint32_t)(n - 1))) break;
          load_q(sg, t, t);
        }
        if (nx.next() && lane < 2 * (D / 64))  // the next segment's queries into L2
          tma_prefetch_3d(&p.q3, 64 * (lane >> 1), nx.g * grp, nx.q.row0 + nx.t * tt + (lane & 1) * p.tok);
      } else {
        if (n == 0) load_q(sg, 0, 0);
        if (nx.next()) {  // the next segment's, in the buffer of the one before (200 short items, heads of 64: 60 us without)
          if (n > 0 && !wait_warp(&sh->qfree[(n + 1) & 1], (uint32_t)((n - 1) >> 1))) break;
          load_q(nx, (n + 1) & 1, 0);
        }
      }
      for (int c = sg.c0; c < sg.c1 && ok; ++c, ++vc) {
        if (!sg.masked(c)) continue;
        const int nk = sg.keys(c), i0 = c - sg.c0;
        const int slot = TWO ? vc % R : (i0 & 1) * R + ((i0 & 1 ? v1 : v0) + (i0 >> 1)) % R;
        if (!wait_warp(&sh->vraw[nraw & 3], (uint32_t)(nraw >> 2))) break;
        ++nraw;
        constexpr int CPR = D / 8;
        uint8_t* vt = Vs + slot * TILE;
        auto at = [&](int i) { return reinterpret_cast<uint4*>(vt + tt_off(i / CPR, i % CPR)); };
        if (sg.own(c)) {
          const int first = max(0, sg.t * tt + 1 - sg.key0(c)) * CPR;  // (rows before it are seen by every row of the item)
          uint32_t any = 0u;
#pragma unroll 8
          for (int i = first + lane; i < nk * CPR; i += 32) any |= tt_odd(*at(i));
          const bool odd = __any_sync(0xffffffffu, any != 0u);
          if (lane == 0) sh->odd[vc % kPtRing] = odd;
          if (odd) {
            if (lane < 4) sh->badv[vc % kPtRing][lane] = 0u;
            __syncwarp();
#pragma unroll 1
            for (int i = first + lane; i < nk * CPR; i += 32) {
              const uint4 x = *at(i);
              if (tt_odd(x)) {
                *at(i) = tt_clear_odd(x);
                atomicOr(&sh->badv[vc % kPtRing][i / CPR >> 5], 1u << (i / CPR & 31));
              }
            }
          }
        }
#pragma unroll 4
        for (int i = nk * CPR + lane; i < ((nk + 15) & ~15) * CPR; i += 32) *at(i) = make_uint4(0, 0, 0, 0);
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh->vfull[slot]);
      }
      if (!ok) break;
      v0 += (sg.c1 - sg.c0 + 1) >> 1;
      v1 += (sg.c1 - sg.c0) >> 1;
    }
    // the query copies have landed before the CTA's shared memory goes away
    for (int t = 0; t < 2; ++t)
      if (loads > t) tc::mbar_wait(&sh->qfull[t], (uint32_t)((loads - t + 1) / 2 - 1) & 1u, nullptr, lim_ns);
  } else {
    // ---------------------------------------------------- softmax, stream t
    const int t = (warp - 4) >> 2, r = tid & 127;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t ts = lane_base + (uint32_t)t * 128u, to = ts + 256u;
    const int rt = pt_div_grp(p, r);  // the row's token of the tile
    const bool in_tile = rt < p.tok;
    PtSeg<false> sg(a, tt);
    int nj = 0, no = 0;                    // the stream's chunks; segments (of one tile: of stream 0)
    int nch = 0, no1 = 0;                  // one tile: all chunks; stream 1's segments
    if (p.apart && tid == 128) pt_items<D>(a.work, gridDim.x)[blockIdx.x].n = 0;  // (no shared item begins here)
    // (after a wait gave up the loops run on without work, to meet the barriers)
    for (bool on = sg.begin(sh); on; on = sg.next()) {
      const int token = sg.t * tt + (TWO ? t * p.tok : 0) + rt;  // of the sequence
      const bool has_row = in_tile && token < sg.q.n;
      const bool warp_on = __any_sync(0xffffffffu, has_row);
      float m_run = -INFINITY, l_run = 0.f;
      const int nj0 = nj;
      // keys of own chunk c that the row sees
      auto own_seen = [&](int c) { return min(kPtCH, max(0, token + 1 - sg.key0(c))); };
      for (int c = sg.c0 + (TWO ? 0 : t); c < sg.c1; c += STEP) {
        const int nk = sg.keys(c);
        const int see = sg.own(c) ? own_seen(c) : nk;
        const int all = sg.own(c) ? sg.t * tt + (TWO ? t * p.tok : 0) + 1 - sg.key0(c) : nk;  // keys that every row of the tile sees
        wait(&sh->sfull[t], (uint32_t)nj);
        // the streams' softmaxes take turns
        if (TWO) {
          if (t == 1) tc::named_bar(7, 256);
          else if (nj > 0) tc::named_bar(6, 256);
        }
        __syncwarp();
        tc::tc_fence_after();
        if (warp_on) {
          constexpr int W = 32, HC = 64;  // columns per step, per part
          auto hide = [&](float (&x)[W], int i) {  // columns W i ..
            if (all < W * (i + 1)) {
              const int n = see - W * i;
              const uint32_t w = n >= W ? 0xffffffffu : n > 0 ? (1u << n) - 1u : 0u;
#pragma unroll
              for (int k = 0; k < W; ++k) x[k] = (w >> k) & 1u ? x[k] : -INFINITY;
            }
          };
          const unsigned long long cs2 = tt_pair(a.scale, a.scale);
          auto cols_max = [&](int i0, int n) {  // the largest score of n steps
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            float x[W];
#pragma unroll 1
            for (int i = i0; i < i0 + n; ++i) {
              tmem_ld_async(ts + W * i, x);
              tmem_wait(x);
#pragma unroll
              for (int k = 0; k < W; k += 2) tt_unpair(tt_mul2(tt_pair(x[k], x[k + 1]), cs2), x[k], x[k + 1]);
              hide(x, i);
#pragma unroll
              for (int k = 0; k < W; k += 2) m4[(k >> 1) & 3] = fmaxf(fmaxf(m4[(k >> 1) & 3], x[k]), x[k + 1]);
            }
            return fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          };
          unsigned long long sa, sb;
          // weights 2^(scale x + m0) of a step, as the product takes them (of 16
          // keys 8 columns of first parts, then what those left), and their sums;
          // `next` starts the next step's loads once the scores have been taken
          auto piece = [&](float (&x)[W], uint32_t* pk, float m0, auto next) {
            const unsigned long long m2 = tt_pair(m0, m0);
            unsigned long long y[W / 2];
#pragma unroll
            for (int k = 0; k < W / 2; ++k) y[k] = tt_fma2(tt_pair(x[2 * k], x[2 * k + 1]), cs2, m2);
            next();
#pragma unroll
            for (int k = 0; k < W / 2; ++k) {
              float lo, hi;
              tt_unpair(y[k], lo, hi);
              lo = tt_ex2(lo);
              hi = tt_ex2(hi);
              if (k & 1) sb = tt_add2(sb, tt_pair(lo, hi));
              else sa = tt_add2(sa, tt_pair(lo, hi));
              tt_split_bf16(lo, hi, pk[(k & ~7) * 2 + (k & 7)], pk[(k & ~7) * 2 + (k & 7) + 8]);
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
          // a new reference, for a row that needs one: log2 of its sum l so far, or
          // the largest of n steps' scores.  (The others keep theirs: a row's result
          // does not depend on the rows that share its warp, lanes without one included.)
          auto refer = [&](int i0, int n, float l, bool needs) {
            const float m_new = fmaxf(cols_max(i0, n), m_run == -INFINITY ? m_run : m_run + tt_lg2(l));
            if (!needs) return 1.f;
            const float alpha = m_run == -INFINITY ? 0.f : tt_ex2(m_run - m_new);
            m_run = m_new;
            return alpha;
          };
          // A half chunk at a time, whose weights stay in registers until their
          // sum shows that the reference suits them.
          const int np = (nk + HC - 1) / HC;  // halves that hold keys
          float sum0 = 0.f;
#pragma unroll 1
          for (int h = 0; h < np; ++h) {
            uint32_t pk[HC];
            float sum;
            bool again = false, over;
#pragma unroll 1
            for (;;) {
              const float m0 = m_run == -INFINITY ? 0.f : -m_run, room = kPtMost - (l_run + sum0);
              sa = sb = tt_pair(0.f, 0.f);
              float x[W];
              tmem_ld_async(ts + HC * h, x);
#pragma unroll
              for (int i = 0; i < HC / W; ++i) {  // the next scores arrive while these are exponentiated
                tmem_wait(x);
                hide(x, h * (HC / W) + i);
                piece(x, pk + i * W, m0, [&]() {
                  if (i + 1 < HC / W) tmem_ld_async(ts + HC * h + W * (i + 1), x);
                });
              }
              float s0, s1;
              tt_unpair(tt_add2(sa, sb), s0, s1);
              sum = s0 + s1;
              // too much for the reference; or a row's first keys, which reference 0 does not suit
              over = sum > room || (m_run == -INFINITY && sum < kPtFew);
              if (again || !__any_sync(0xffffffffu, over && has_row)) break;
              again = true;
              const float alpha = refer(h * (HC / W), HC / W, l_run + sum0, over);
              rescale(alpha);
              l_run *= alpha;
              if (h) {  // the half before, stored already
                sum0 *= alpha;
                rescale_p(alpha, HC * h);
              }
            }
            if (!over && m_run == -INFINITY) m_run = 0.f;
            sum0 += sum;
            if (TWO && h == min(1, np - 1)) named_arrive(t == 0 ? 7 : 6, 256);
#pragma unroll
            for (int i = 0; i < HC; i += 32) tmem_st32u(ts + HC * h + i, pk + i);
          }
          l_run += sum0;
        } else if (TWO) {
          named_arrive(t == 0 ? 7 : 6, 256);
        }
        tc::tc_fence_before();
        tc::mbar_arrive(&sh->pdone[t]);
        ++nj;
      }

      // ---- the segment's end: normalise and write, or leave a partial.  What
      // does not depend on the last product comes before the wait for it.
      const bool whole = sg.c0 == 0 && sg.c1 == sg.nch;
      // A whole item's rows are turned in shared memory, so that four lanes
      // store 64 bytes of a row: lane i has piece i % 4 of rows i / 4 + 8 k.
      uint4* stage = reinterpret_cast<uint4*>(sm + Cfg::O_OFF + (warp - 4) * 2048);
      uint32_t piece_at[4];  // in 16-byte pieces of `out` (the host checks that they fit)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int rr = (warp & 3) * 32 + 8 * k + (lane >> 2), tk = pt_div_grp(p, rr), at = sg.t * tt + (TWO ? t * p.tok : 0) + tk;
        const bool write = tk < p.tok && at < sg.q.n && DFL_CHECK(sg.q.row0 + at < a.M, status);
        piece_at[k] = write ? ((uint32_t)(sg.q.row0 + at) * a.nq + sg.g * grp + rr - tk * grp) * (D / 8) + (lane & 3)
                            : 0xffffffffu;
      }
      const int cb = max(sg.c0, max(sg.q.cc, sg.c1 - 3));  // (an item's tokens reach into three chunks at most)
      float f = 1.f, f1 = 0.f;  // factors of the stream's output; of one tile: of stream 0's and stream 1's
      if constexpr (TWO) {
        if (whole) f = 1.f / l_run;  // (as in pt_join)
        wait(&sh->ofull[t], (uint32_t)no++);
      } else {
        float* ml = reinterpret_cast<float*>(sm + Cfg::M_OFF);
        ml[t * 256 + r] = m_run;
        ml[t * 256 + 128 + r] = l_run;
        wait(&sh->ofull[0], (uint32_t)no++);
        if (sg.c1 - sg.c0 > 1) wait(&sh->ofull[1], (uint32_t)no1++);
        tc::named_bar(1, 256);
        const float m0 = ml[r], m1 = ml[256 + r];
        m_run = fmaxf(m0, m1);
        f = m0 == -INFINITY ? 0.f : tt_ex2(m0 - m_run);
        f1 = m1 == -INFINITY ? 0.f : tt_ex2(m1 - m_run);
        l_run = fmaf(ml[128 + r], f, ml[384 + r] * f1);
        if (whole) {
          f /= l_run;
          f1 /= l_run;
        }
      }
      __syncwarp();
      tc::tc_fence_after();
      if (warp_on) {
        // visible NaN or infinite values of chunks seen in part
        const int cj0 = (TWO ? nj0 : nch) - sg.c0;
        auto bad_of = [&](int c, int i) {
          const int n = (has_row ? own_seen(c) : 0) - 32 * i;
          const uint32_t w = n >= 32 ? 0xffffffffu : n > 0 ? (1u << n) - 1u : 0u;
          return w & sh->badv[(cj0 + c) % kPtRing][i];
        };
        bool any_bad = false;
        for (int c = cb; c < sg.c1; ++c) any_bad |= sg.masked(c) && sh->odd[(cj0 + c) % kPtRing] != 0;
        float* part = static_cast<float*>(a.work) +
                      ((size_t)2 * blockIdx.x + (sg.c0 > 0 ? 0 : 1)) * pt_slot_floats<D>();
        const int prow = (TWO ? t * kPtRows : 0) + r;
        constexpr int W = 32;  // columns per step
#pragma unroll 1
        for (int q = 0; q < D / W / STEP; ++q) {  // (of one tile each stream takes half of the columns)
          const int col = W * q + (TWO ? 0 : t * (D / 2));
          float o[W];
          __syncwarp();  // the load below is warp-collective
          if constexpr (TWO) {
            tc::tmem_ld32(to + col, o);
#pragma unroll
            for (int k = 0; k < W; ++k) o[k] *= f;
          } else {
            tc::tmem_ld32(lane_base + 256u + col, o);
#pragma unroll
            for (int k = 0; k < W; ++k) o[k] *= f;
            if (sg.c1 - sg.c0 > 1) {
              float y[W];
              tc::tmem_ld32(lane_base + 384u + col, y);
#pragma unroll
              for (int k = 0; k < W; ++k) o[k] = fmaf(y[k], f1, o[k]);
            }
          }
          if (any_bad)  // added as they are
            for (int c = cb; c < sg.c1; ++c)
              if (sg.masked(c) && sh->odd[(cj0 + c) % kPtRing])
                for (int i = 0; i < 4; ++i)
                  for (uint32_t b = bad_of(c, i); b; b &= b - 1) {
                    const int vrow = sg.q.row0 + sg.key0(c) + 32 * i + __ffs(b) - 1;
                    if (!DFL_CHECK(vrow >= 0 && vrow < a.M, status)) continue;
                    const __nv_bfloat16* v =
                        static_cast<const __nv_bfloat16*>(a.vb) + ((size_t)vrow * a.nkv + sg.g) * D + col;
#pragma unroll
                    for (int k = 0; k < W; ++k) {
                      const float x = __bfloat162float(v[k]);
                      if (!(fabsf(x) < INFINITY)) o[k] += x;
                    }
                  }
          __syncwarp();
          if (whole) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              stage[lane * 4 + (k ^ ((lane >> 1) & 3))] =
                  make_uint4(tt_pack(o[8 * k], o[8 * k + 1]), tt_pack(o[8 * k + 2], o[8 * k + 3]),
                             tt_pack(o[8 * k + 4], o[8 * k + 5]), tt_pack(o[8 * k + 6], o[8 * k + 7]));
            __syncwarp();
            uint4 y[4];  // (all read before the first is stored: the stores may alias)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int rr = 8 * k + (lane >> 2);
              y[k] = stage[rr * 4 + ((lane & 3) ^ ((rr >> 1) & 3))];
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (piece_at[k] != 0xffffffffu) reinterpret_cast<uint4*>(a.out)[piece_at[k] + col / 8] = y[k];
          } else if (has_row) {
            float4* p4 = reinterpret_cast<float4*>(part) + (TWO ? (size_t)t * (kPtRows * D / 4) : 0);
#pragma unroll
            for (int k = 0; k < W / 4; ++k)
              p4[(size_t)(col / 4 + k) * kPtRows + r] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
        }
        if (!whole && has_row && (TWO || t == 0)) {
          float* ml = part + (size_t)2 * kPtRows * D;
          ml[prow] = m_run;
          ml[2 * kPtRows + prow] = l_run;
        }
      }
      if (!TWO) tc::tc_fence_before();
      if (sg.c0 > 0 || sg.c1 < sg.nch) {  // the item is shared
        const int first = sg.c0 > 0 ? sh->x0 - sh->c0 : sh->x0 + sh->len - sg.c1 - kPtSetup;  // the item's first position
        const int b0 = (first + kPtSetup) / sh->per, b1 = (first + kPtSetup + sg.nch - 1) / sh->per;
        const PtItem it{sg.q.row0 + sg.t * tt, sg.end - sg.t * tt, sg.g, b1};
        if (p.apart) {
          if (sg.c0 == 0 && tid == 128) pt_items<D>(a.work, gridDim.x)[blockIdx.x] = it;
        } else {  // who leaves the last partial joins them
          __threadfence();
          tc::named_bar(1, 256);
          if (tid == 128) {
            uint32_t* ctr = a.counters + (DFL_CHECK(b0 >= 0 && b0 < (int)gridDim.x, status) ? b0 : blockIdx.x);
            const uint32_t before = atomicAdd(ctr, 1u);
            sh->last = before == (uint32_t)(b1 - b0);
            if (sh->last) *ctr = 0u;  // (ready for the next launch)
            __threadfence();
          }
          tc::named_bar(1, 256);
          if (sh->last) pt_join<D, TWO, 16, 4>(p, it, b0, warp - 4, 8);
        }
      }
      // (sh->last has been read; of one tile, the streams' outputs, maxima and sums)
      if (!TWO || !p.apart) tc::named_bar(1, 256);
      nch += sg.c1 - sg.c0;
    }
    if (TWO && t == 0 && nj > 0) tc::named_bar(6, 256);  // meets stream 1's last arrival
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

// Joins every shared item: CTA (b, y) takes every gridDim.y-th share of the one
// that begins in CTA b of the kernel before.
template <int D, bool TWO>
__global__ void __launch_bounds__(256) prompt_join_kernel(const __grid_constant__ PtTma p) {
  pdl_wait();
  pdl_launch_dependents();
  const int4 x = __ldcg(reinterpret_cast<const int4*>(pt_items<D>(p.a.work, gridDim.x)) + blockIdx.x);
  const PtItem it{x.x, x.y, x.z, x.w};
  if (it.n > 0) pt_join<D, TWO, 8, 8>(p, it, blockIdx.x, blockIdx.y * 8 + (threadIdx.x >> 5), gridDim.y * 8);
}

// Are shared items joined by a kernel of their own?  Within the kernel one CTA
// reads an item's partials (65 GB/s), while the second launch costs 3 us but
// spreads them over all SMs: from 256 KB an item on, or 16 partials, by what is
// known here of the lengths.  In the kernel / apart: 64 rows over 8000 slots 51
// / 26 us, 32 over 4000 28 / 17.5, 1 over 8000 18.3 / 17.2; 5 rows over nothing
// 7.1 / 10.8, 200 sequences of 5 rows over 300 53 / 57.
bool pt_apart(const PromptAttnDesc& a, int num_sms, int tt) {
  const double rows = (double)a.M / a.n_seqs, grp = a.nq / a.nkv;
  const double items = (double)a.nkv * std::max((double)a.n_seqs, (double)a.M / tt);
  const double chunks = ((double)a.max_pos + rows) / kPtCH + 1;
  const double parts = std::min(num_sms / items, chunks / kPtLeastOne);
  return parts >= 16 || parts * std::min(rows, (double)tt) * grp * a.d * 4 >= 256 * 1024;
}

template <int D, bool TWO>
cudaError_t pt_launch(const PromptAttnDesc& a, int num_sms, cudaStream_t st) {
  using Cfg = PtCfg<D, TWO>;
  PtTma p;
  p.a = a;
  p.grp = a.nq / a.nkv;
  p.tok = kPtRows / p.grp;
  p.grp_mul = p.grp >= 2 ? (uint32_t)((0x100000000ull + p.grp - 1) / p.grp) : 0u;
  const uint64_t M = (uint64_t)a.M;
  bool okm = make_tmap3_bf16(&p.kb, a.kb, D, a.nkv, M, 1, kPtCH) && make_tmap3_bf16(&p.vb, a.vb, D, a.nkv, M, 1, kPtCH) &&
             make_tmap3_bf16(&p.q3, a.q, D, a.nq, M, p.grp, p.tok);
  p.kc = p.kb;
  p.vc = p.vb;
  if (a.kc) {
    const uint64_t rows = a.pages ? (uint64_t)a.pool * a.nkv * a.ps : (uint64_t)a.n_seqs * a.nkv * a.cap;
    okm = okm && make_tmap_bf16(&p.kc, a.kc, D, rows, kPtCH) && make_tmap_bf16(&p.vc, a.vc, D, rows, kPtCH);
  }
  if (!okm) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(prompt_tc_kernel<D, TWO>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg::SMEM);
  if (e != cudaSuccess) return e;
  p.apart = pt_apart(a, num_sms, p.tok * (TWO ? 2 : 1)) ? 1 : 0;
  e = launch_pdl(prompt_tc_kernel<D, TWO>, dim3(num_sms), dim3(Cfg::THREADS), Cfg::SMEM, st, p);
  if (e != cudaSuccess || !p.apart) return e;
  return launch_pdl(prompt_join_kernel<D, TWO>, dim3(num_sms, TWO ? D / 8 : D / 16), dim3(256), 0, st, p);
}

}  // namespace

size_t prompt_tc_workspace(const PromptAttnDesc& a, int num_sms) {
  return (size_t)num_sms * (2 * 2 * kPtRows * (a.d + 2) * sizeof(float) + sizeof(PtItem));
}

cudaError_t launch_prompt_tc(const PromptAttnDesc& a, int num_sms, cudaStream_t st) {
  // Items of two tiles where sequences have more rows than a tile on average (one
  // / two tiles, 32 rows a tile: 8 sequences of 16 rows over 4000 slots 37 / 54
  // us, of 32 40 / 57, of 33 57 / 48, of 64 59 / 53; 16 of 1 to 64 over 1000 34 /
  // 38; a prompt of 2000 73 / 58).
  const bool two = (long long)a.M > (long long)a.n_seqs * (kPtRows / (a.nq / a.nkv));
  if (two) return a.d == 128 ? pt_launch<128, true>(a, num_sms, st) : pt_launch<64, true>(a, num_sms, st);
  return a.d == 128 ? pt_launch<128, false>(a, num_sms, st) : pt_launch<64, false>(a, num_sms, st);
}

}  // namespace dfl
