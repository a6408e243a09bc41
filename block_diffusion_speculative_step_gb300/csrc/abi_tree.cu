// abi_tree.cu -- the C ABI of tree verification: host-side argument checks and
// launches of dflash_tree_attention, dflash_tree_build, dflash_tree_accept,
// dflash_kv_write and dflash_kv_read.  Every check runs before the first
// launch of a call; no exception crosses the ABI.
#include <string.h>

#include "abi_common.h"
#include "abi_tree.h"
#include "common.cuh"
#include "internal.h"

using namespace dfl;

namespace dfl {

// Shapes of a tree attention problem (also the layer's DFLASH_ATTN_TREE mode).
int check_tree_shape(const dflash_dims& d, int S, int rows, int max_pos, const dflash_kv& kv, const char* who) {
  DF_CHECK(S > 0 && rows > 0, "%s: n_seqs and rows must be positive", who);
  DF_CHECK(rows <= DFLASH_MAX_TREE, "%s: a tree holds at most %d rows", who, DFLASH_MAX_TREE);
  DF_CHECK(kv.capacity > 0, "%s: kv capacity must be positive", who);
  DF_CHECK(kv.window == 0, "%s: tree attention takes no window", who);
  DF_CHECK((kv.k_exp == nullptr) == (kv.v_exp == nullptr), "%s: k_exp and v_exp must both be set or both be NULL", who);
  int rc = check_kv_pages(kv, who);
  if (rc) return rc;
  DF_CHECK(max_pos >= 0 && max_pos <= kv.capacity, "%s: max_pos %d must be in [0, capacity %d]", who, max_pos,
           kv.capacity);
  const long long vecs =
      kv.pages ? (long long)kv.pool_pages * kv.page_size * d.n_kv_heads : (long long)S * kv.capacity * d.n_kv_heads;
  DF_CHECK(vecs < (1ll << 31), "%s: the cache holds 2^31 or more rows", who);
  DF_CHECK((long long)S * rows * d.n_q_heads < (1ll << 31) / 128, "%s: too many query vectors", who);
  DF_CHECK((long long)S * d.n_kv_heads * ((rows * (d.n_q_heads / d.n_kv_heads) + 127) / 128) * (max_pos / 128 + 4) <
               (1ll << 27),
           "%s: too many (sequence, KV head, 128-slot chunk) pieces", who);
  DF_CHECK(S <= 65535 && d.n_q_heads <= 4096, "%s: n_seqs must be at most 65535, n_q_heads at most 4096", who);
  return DFLASH_OK;
}

// Device pointers that the kernels read with 16-byte accesses.
static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int check_tree_kv(const dflash_kv& kv, const char* who) {
  DF_CHECK(kv.k && kv.v, "%s: NULL cache pointer", who);
  DF_CHECK(aligned16(kv.k) && aligned16(kv.v), "%s: cache pointers must be 16-byte aligned", who);
  return DFLASH_OK;
}

TreeAttnDesc tree_attn_desc(const dflash_dims& d, int S, int rows, int max_pos, const dflash_kv& kv, float scale) {
  TreeAttnDesc t;
  memset(&t, 0, sizeof(t));
  t.dtype = d.dtype;
  t.n_seqs = S;
  t.rows = rows;
  t.nq = d.n_q_heads;
  t.nkv = d.n_kv_heads;
  t.d = d.head_dim;
  t.kc = kv.k;
  t.vc = kv.v;
  t.k_exp = kv.k_exp;
  t.v_exp = kv.v_exp;
  t.cap = kv.capacity;
  t.pages = kv.pages;
  t.ps = kv.page_size;
  t.max_pages = kv.max_pages;
  t.pool = kv.pool_pages;
  t.max_pos = max_pos;
  t.scale = (scale == 0.f ? 1.f / sqrtf((float)d.head_dim) : scale) * 1.4426950408889634f;
  return t;
}

}  // namespace dfl

extern "C" {

// ------------------------------------------------------------- attention

static int check_tree_attention_shape(const dflash_tree_attention_args* a, const char* who) {
  DF_CHECK(a != nullptr, "%s: NULL args", who);
  int rc = check_dims(a->dims, who);
  if (rc) return rc;
  DF_CHECK(a->scale >= 0.f && a->scale < 1e30f, "%s: scale must be >= 0 and finite", who);
  return check_tree_shape(a->dims, a->n_seqs, a->rows, a->max_pos, a->kv, who);
}

int dflash_tree_attention(const dflash_tree_attention_args* a, void* ws, size_t ws_bytes, dflash_stream_t stream) {
  const char* who = "dflash_tree_attention";
  int rc = check_tree_attention_shape(a, who);
  if (rc) return rc;
  DF_CHECK(a->base_pos && a->q && a->kb && a->vb && a->out, "%s: NULL pointer", who);
  rc = check_tree_kv(a->kv, who);
  if (rc) return rc;
  DF_CHECK(aligned16(a->q) && aligned16(a->kb) && aligned16(a->vb) && aligned16(a->out),
           "%s: q, kb, vb and out must be 16-byte aligned", who);
  const int sms = num_sms();
  TreeAttnDesc t = tree_attn_desc(a->dims, a->n_seqs, a->rows, a->max_pos, a->kv, a->scale);
  rc = check_ws(ws, ws_bytes, kReservedBytes + tree_attn_workspace(t, sms), who);
  if (rc) return rc;
  t.base_pos = a->base_pos;
  t.parent = a->parent;
  t.q = a->q;
  t.kb = a->kb;
  t.vb = a->vb;
  t.out = a->out;
  t.work = static_cast<char*>(ws) + kReservedBytes;
  t.status = header(ws).status;
  DF_LAUNCH((cudaStream_t)stream, TF_ATTN, 0, launch_tree_attention(t, sms, (cudaStream_t)stream));
  return DFLASH_OK;
}

// ----------------------------------------------------------------- build

static int check_tree_build_shape(const dflash_tree_build_args* a, const char* who) {
  DF_CHECK(a != nullptr, "%s: NULL args", who);
  DF_CHECK(a->n_seqs > 0 && a->rows > 0 && a->rows <= DFLASH_MAX_TREE, "%s: need n_seqs > 0 and 0 < rows <= %d", who,
           DFLASH_MAX_TREE);
  DF_CHECK(a->levels > 0 && a->topk > 0, "%s: levels and topk must be positive", who);
  return DFLASH_OK;
}

int dflash_tree_build(const dflash_tree_build_args* a, void* ws, size_t ws_bytes, dflash_stream_t stream) {
  const char* who = "dflash_tree_build";
  int rc = check_tree_build_shape(a, who);
  if (rc) return rc;
  DF_CHECK(a->parent && a->rank && a->cand && a->anchor && a->base_pos && a->parent_out && a->tokens_out && a->pos_out,
           "%s: NULL pointer", who);
  rc = check_ws(ws, ws_bytes, kReservedBytes, who);
  if (rc) return rc;
  TreeBuildDesc t;
  t.n_seqs = a->n_seqs;
  t.rows = a->rows;
  t.levels = a->levels;
  t.topk = a->topk;
  t.parent = a->parent;
  t.rank = a->rank;
  t.cand = a->cand;
  t.anchor = a->anchor;
  t.base_pos = a->base_pos;
  t.parent_out = a->parent_out;
  t.tokens_out = a->tokens_out;
  t.pos_out = a->pos_out;
  t.status = header(ws).status;
  DF_LAUNCH((cudaStream_t)stream, TF_PATH, 0, launch_tree_build(t, (cudaStream_t)stream));
  return DFLASH_OK;
}

// ---------------------------------------------------------------- accept

static int check_tree_accept_shape(const dflash_tree_accept_args* a, const char* who) {
  DF_CHECK(a != nullptr, "%s: NULL args", who);
  DF_CHECK(a->dims.vocab > 0 && a->dims.vocab < (1 << 24), "%s: vocab must be in [1, 2^24)", who);
  DF_CHECK(a->n_seqs > 0 && a->rows > 0 && a->rows <= DFLASH_MAX_TREE, "%s: need n_seqs > 0 and 0 < rows <= %d", who,
           DFLASH_MAX_TREE);
  DF_CHECK(a->n_seqs <= (1 << 16), "%s: n_seqs must be at most 65536", who);
  DF_CHECK(a->temperature >= 0.f && a->temperature < 1e30f, "%s: temperature must be >= 0 and finite", who);
  DF_CHECK(a->temperature == 0.f || a->temperature >= 1e-6f, "%s: temperature must be 0 or at least 1e-6", who);
  DF_CHECK(a->levels >= 0, "%s: levels must be >= 0", who);
  return DFLASH_OK;
}

int dflash_tree_accept(const dflash_tree_accept_args* a, void* ws, size_t ws_bytes, dflash_stream_t stream) {
  const char* who = "dflash_tree_accept";
  int rc = check_tree_accept_shape(a, who);
  if (rc) return rc;
  DF_CHECK(a->tokens && a->accept_len && a->path && a->out_tokens, "%s: NULL pointer", who);
  if (a->temperature > 0.f)
    DF_CHECK(a->target_logits && a->u && a->noise, "%s: sampling needs target_logits, u and noise", who);
  else
    DF_CHECK(a->target_argmax, "%s: temperature 0 needs target_argmax", who);
  DF_CHECK(!a->draft_logits || a->levels > 0, "%s: draft_logits needs levels > 0", who);
  DF_CHECK(a->base_pos || !(a->update_base_pos || a->commit_base), "%s: update_base_pos and commit_base need base_pos",
           who);
  rc = check_ws(ws, ws_bytes, kReservedBytes, who);
  if (rc) return rc;
  TreeAcceptDesc t;
  memset(&t, 0, sizeof(t));
  t.n_seqs = a->n_seqs;
  t.rows = a->rows;
  t.levels = a->levels;
  t.V = a->dims.vocab;
  t.invT = a->temperature > 0.f ? 1.f / a->temperature : 0.f;
  t.parent = a->parent;
  t.tokens = a->tokens;
  t.target = a->target_logits;
  t.argmax = a->target_argmax;
  t.draft = a->draft_logits;
  t.u = a->u;
  t.noise = a->noise;
  t.base_pos = a->base_pos;
  t.update_base = a->update_base_pos;
  t.accept_len = a->accept_len;
  t.path = a->path;
  t.out_tokens = a->out_tokens;
  t.next_anchor = a->next_anchor;
  t.commit_base = a->commit_base;
  t.commit_count = a->commit_count;
  t.status = header(ws).status;
  DF_LAUNCH((cudaStream_t)stream, TF_SAMPLE, 0, launch_tree_accept(t, num_sms(), (cudaStream_t)stream));
  return DFLASH_OK;
}

// ------------------------------------------------------------ cache rows

// The checks shared by the write and the read.
static int check_kv_rows(const dflash_dims& d, int n_layers, const dflash_kv* kv, int S, int rows, const char* who) {
  int rc = check_dims(d, who);
  if (rc) return rc;
  DF_CHECK(n_layers > 0 && n_layers <= DFLASH_KV_MAX_LAYERS, "%s: n_layers must be in [1, %d]", who,
           DFLASH_KV_MAX_LAYERS);
  DF_CHECK(S > 0 && rows > 0, "%s: n_seqs and rows must be positive", who);
  DF_CHECK((long long)S * rows < (1ll << 27) / d.n_kv_heads, "%s: n_seqs * rows * n_kv_heads must be below 2^27", who);
  DF_CHECK(kv != nullptr, "%s: kv_layers is NULL", who);
  for (int j = 0; j < n_layers; ++j) {
    const dflash_kv& c = kv[j];
    rc = check_kv_pages(c, who);
    if (rc) return rc;
    DF_CHECK(c.capacity > 0 && (c.window == 0 || c.window == c.capacity),
             "%s: capacity must be positive, a window ring needs capacity == window", who);
    DF_CHECK((c.k_exp == nullptr) == (c.v_exp == nullptr), "%s: k_exp and v_exp must both be set or both be NULL", who);
    DF_CHECK(c.capacity == kv[0].capacity && c.window == kv[0].window && !c.pages == !kv[0].pages &&
                 c.page_size == kv[0].page_size && c.max_pages == kv[0].max_pages && c.pool_pages == kv[0].pool_pages &&
                 !c.k_exp == !kv[0].k_exp,
             "%s: every layer's cache must share one geometry", who);
  }
  const dflash_kv& c = kv[0];
  const long long vecs =
      c.pages ? (long long)c.pool_pages * c.page_size * d.n_kv_heads : (long long)S * c.capacity * d.n_kv_heads;
  DF_CHECK(vecs < (1ll << 31), "%s: the cache holds 2^31 or more rows", who);
  return DFLASH_OK;
}

static KvRowsDesc kv_rows_desc(const dflash_dims& d, int n_layers, const dflash_kv& c, int S, int rows,
                               const int32_t* base_pos, const int32_t* valid, void* ws) {
  KvRowsDesc k;
  memset(&k, 0, sizeof(k));
  k.dtype = d.dtype;
  k.n_layers = n_layers;
  k.S = S;
  k.rows = rows;
  k.nkv = d.n_kv_heads;
  k.d = d.head_dim;
  k.base_pos = base_pos;
  k.valid = valid;
  k.cap = c.capacity;
  k.window = c.window;
  k.ps = c.page_size;
  k.max_pages = c.max_pages;
  k.pool = c.pool_pages;
  k.status = header(ws).status;
  return k;
}

int dflash_kv_write(const dflash_kv_write_args* a, void* ws, size_t ws_bytes, dflash_stream_t stream) {
  const char* who = "dflash_kv_write";
  DF_CHECK(a != nullptr, "%s: NULL args", who);
  int rc = check_kv_rows(a->dims, a->n_layers, a->kv_layers, a->n_seqs, a->rows, who);
  if (rc) return rc;
  DF_CHECK(a->kb && a->vb && a->base_pos, "%s: NULL pointer", who);
  KvRowsLayers l;
  memset(&l, 0, sizeof(l));
  for (int j = 0; j < a->n_layers; ++j) {
    const dflash_kv& c = a->kv_layers[j];
    DF_CHECK(a->kb[j] && a->vb[j] && c.k && c.v, "%s: NULL layer %d pointer", who, j);
    DF_CHECK(aligned16(a->kb[j]) && aligned16(a->vb[j]) && aligned16(c.k) && aligned16(c.v),
             "%s: layer %d pointers must be 16-byte aligned", who, j);
    l.src_k[j] = a->kb[j];
    l.src_v[j] = a->vb[j];
    l.dst_k[j] = c.k;
    l.dst_v[j] = c.v;
    l.k_exp[j] = c.k_exp;
    l.v_exp[j] = c.v_exp;
    l.pages[j] = c.pages;
  }
  rc = check_ws(ws, ws_bytes, kReservedBytes, who);
  if (rc) return rc;
  KvRowsDesc k = kv_rows_desc(a->dims, a->n_layers, a->kv_layers[0], a->n_seqs, a->rows, a->base_pos, a->valid, ws);
  k.row_index = a->row_index;
  DF_LAUNCH((cudaStream_t)stream, TF_PAGE, 0, launch_kv_write(k, l, (cudaStream_t)stream));
  return DFLASH_OK;
}

int dflash_kv_read(const dflash_kv_read_args* a, void* ws, size_t ws_bytes, dflash_stream_t stream) {
  const char* who = "dflash_kv_read";
  DF_CHECK(a != nullptr, "%s: NULL args", who);
  int rc = check_kv_rows(a->dims, a->n_layers, a->kv_layers, a->n_seqs, a->rows, who);
  if (rc) return rc;
  DF_CHECK(a->k_out && a->v_out && a->base_pos, "%s: NULL pointer", who);
  KvRowsLayers l;
  memset(&l, 0, sizeof(l));
  for (int j = 0; j < a->n_layers; ++j) {
    const dflash_kv& c = a->kv_layers[j];
    DF_CHECK(a->k_out[j] && a->v_out[j] && c.k && c.v, "%s: NULL layer %d pointer", who, j);
    DF_CHECK(aligned16(a->k_out[j]) && aligned16(a->v_out[j]) && aligned16(c.k) && aligned16(c.v),
             "%s: layer %d pointers must be 16-byte aligned", who, j);
    l.src_k[j] = c.k;
    l.src_v[j] = c.v;
    l.dst_k[j] = a->k_out[j];
    l.dst_v[j] = a->v_out[j];
    l.k_exp[j] = c.k_exp;
    l.v_exp[j] = c.v_exp;
    l.pages[j] = c.pages;
  }
  rc = check_ws(ws, ws_bytes, kReservedBytes, who);
  if (rc) return rc;
  const KvRowsDesc k =
      kv_rows_desc(a->dims, a->n_layers, a->kv_layers[0], a->n_seqs, a->rows, a->base_pos, a->valid, ws);
  DF_LAUNCH((cudaStream_t)stream, TF_PAGE, 0, launch_kv_read(k, l, (cudaStream_t)stream));
  return DFLASH_OK;
}

}  // extern "C"

namespace dfl {

size_t tree_op_workspace(int op, const void* args, const char* who) {
  switch (op) {
    case DFLASH_OP_TREE_ATTENTION: {
      const dflash_tree_attention_args* a = static_cast<const dflash_tree_attention_args*>(args);
      if (check_tree_attention_shape(a, who)) return 0;
      return kReservedBytes +
             tree_attn_workspace(tree_attn_desc(a->dims, a->n_seqs, a->rows, a->max_pos, a->kv, a->scale), num_sms());
    }
    case DFLASH_OP_TREE_BUILD:
      return check_tree_build_shape(static_cast<const dflash_tree_build_args*>(args), who) ? 0 : kReservedBytes;
    case DFLASH_OP_TREE_ACCEPT:
      return check_tree_accept_shape(static_cast<const dflash_tree_accept_args*>(args), who) ? 0 : kReservedBytes;
    case DFLASH_OP_KV_WRITE: {
      const dflash_kv_write_args* a = static_cast<const dflash_kv_write_args*>(args);
      return check_kv_rows(a->dims, a->n_layers, a->kv_layers, a->n_seqs, a->rows, who) ? 0 : kReservedBytes;
    }
    case DFLASH_OP_KV_READ: {
      const dflash_kv_read_args* a = static_cast<const dflash_kv_read_args*>(args);
      return check_kv_rows(a->dims, a->n_layers, a->kv_layers, a->n_seqs, a->rows, who) ? 0 : kReservedBytes;
    }
  }
  return 0;
}

}  // namespace dfl
