// abi_prompt.cu -- the C ABI of the prompt operators: host-side argument checks
// and launches of dflash_qk_norm_rope, dflash_prompt_attention and
// dflash_token_logprobs.  Every check runs before the first launch of a call;
// no exception crosses the ABI.
#include "abi_prompt.h"

#include <math.h>
#include <string.h>

#include "common.cuh"

using namespace dfl;

namespace dfl {

// A cache of dims.dtype without a window, as the prompt operators take it.
static int check_plain_cache(const dflash_kv& kv, int S, int nkv, const char* who) {
  if (kv.k_exp || kv.v_exp) return fail(DFLASH_ERR_UNSUPPORTED, "%s: the cache cannot be an 8-bit one", who);
  DF_CHECK(kv.capacity > 0, "%s: kv capacity must be positive", who);
  DF_CHECK(kv.window == 0, "%s: the cache takes no window", who);
  const int rc = check_kv_pages(kv, who);
  if (rc) return rc;
  const long long vecs =
      kv.pages ? (long long)kv.pool_pages * kv.page_size * nkv : (long long)S * kv.capacity * nkv;
  DF_CHECK(vecs < (1ll << 31), "%s: the cache holds 2^31 or more rows", who);
  return DFLASH_OK;
}

int check_prompt_shape(const dflash_dims& d, int S, int M, bool context, int max_pos, const dflash_kv& kv,
                       const char* who) {
  DF_CHECK(S > 0 && M > 0, "%s: n_seqs and n_rows must be positive", who);
  if (context) {
    const int rc = check_plain_cache(kv, S, d.n_kv_heads, who);
    if (rc) return rc;
    DF_CHECK(max_pos >= 0 && max_pos <= kv.capacity, "%s: max_pos %d must be in [0, capacity %d]", who, max_pos,
             kv.capacity);
  }
  const int grp = d.n_q_heads / d.n_kv_heads;
  if (grp > 128) return fail(DFLASH_ERR_UNSUPPORTED, "%s: at most 128 query heads per KV head", who);
  DF_CHECK((long long)M * d.n_q_heads < (1ll << 31) / 16, "%s: too many query vectors", who);
  // pieces (128 query vectors x KV head x 128 keys) of one sequence of all rows, and what every sequence adds
  const double tiles = (double)M * grp / 64 + S, mean = max_pos * (context ? 1.0 / 64 : 0.0) + M / 128.0 + 8;
  if (tiles * d.n_kv_heads * mean >= (double)(1u << 31) || S > (1 << 16))
    return fail(DFLASH_ERR_UNSUPPORTED, "%s: too many (query tile, KV head, 128-key chunk) pieces", who);
  return DFLASH_OK;
}

PromptAttnDesc prompt_attn_desc(const dflash_dims& d, int S, int M, bool context, int max_pos, const dflash_kv& kv,
                                float scale) {
  PromptAttnDesc p;
  memset(&p, 0, sizeof(p));
  p.dtype = d.dtype;
  p.n_seqs = S;
  p.M = M;
  p.nq = d.n_q_heads;
  p.nkv = d.n_kv_heads;
  p.d = d.head_dim;
  if (context) {
    p.kc = kv.k;
    p.vc = kv.v;
    p.cap = kv.capacity;
    p.pages = kv.pages;
    p.ps = kv.page_size;
    p.max_pages = kv.max_pages;
    p.pool = kv.pool_pages;
    p.max_pos = max_pos;
  }
  p.scale = (scale == 0.f ? 1.f / sqrtf((float)d.head_dim) : scale) * 1.4426950408889634f;
  return p;
}

QkNormDesc qk_norm_desc(const dflash_dims& d, int M, int rows, const dflash_kv* cache) {
  QkNormDesc q;
  memset(&q, 0, sizeof(q));
  q.dtype = d.dtype;
  q.M = M;
  q.rows = rows;
  q.nq = d.n_q_heads;
  q.nkv = d.n_kv_heads;
  q.d = d.head_dim;
  q.eps = d.rms_eps;
  q.stride = (long long)(d.n_q_heads + 2 * d.n_kv_heads) * d.head_dim;
  if (cache) {
    q.cache = 1;
    q.k = cache->k;
    q.v = cache->v;
    q.cap = cache->capacity;
    q.pages = cache->pages;
    q.ps = cache->page_size;
    q.max_pages = cache->max_pages;
    q.pool = cache->pool_pages;
  }
  return q;
}

}  // namespace dfl

extern "C" {

// ------------------------------------------------- head norms and rotation

static int check_qk_norm_shape(const dflash_qk_norm_rope_args* a, const char* who) {
  DF_CHECK(a != nullptr, "%s: NULL args", who);
  int rc = check_dims(a->dims, who);
  if (rc) return rc;
  DF_CHECK(a->n_seqs > 0 && a->rows > 0, "%s: n_seqs and rows must be positive", who);
  const long long heads = a->dims.n_q_heads + 2ll * a->dims.n_kv_heads;
  DF_CHECK((long long)a->n_seqs * a->rows * heads < (1ll << 31), "%s: too many heads in all", who);
  DF_CHECK(a->qkv_dtype == DFLASH_F32 || a->qkv_dtype == DFLASH_BF16, "%s: qkv_dtype %d not F32/BF16", who,
           a->qkv_dtype);
  DF_CHECK(a->qkv_stride == 0 || (a->qkv_stride >= heads * a->dims.head_dim && a->qkv_stride % 8 == 0 &&
                                  a->qkv_stride < (1ll << 40)),
           "%s: qkv_stride must be 0 or a multiple of 8 that holds every head", who);
  DF_CHECK(a->rope_max_pos > 0, "%s: rope_max_pos must be positive", who);
  return DFLASH_OK;
}

int dflash_qk_norm_rope(const dflash_qk_norm_rope_args* a, void* ws, size_t ws_bytes, dflash_stream_t stream) {
  const char* who = "dflash_qk_norm_rope";
  int rc = check_qk_norm_shape(a, who);
  if (rc) return rc;
  DF_CHECK(a->base_pos && a->qkv && a->rope_cs && a->q, "%s: NULL pointer", who);
  DF_CHECK((a->kb == nullptr) == (a->vb == nullptr), "%s: kb and vb must both be set or both be NULL", who);
  const bool cache = a->kb == nullptr;
  if (cache) {
    rc = check_plain_cache(a->kv, a->n_seqs, a->dims.n_kv_heads, who);
    if (rc) return rc;
    DF_CHECK(a->kv.k && a->kv.v, "%s: NULL cache pointer (and no kb / vb)", who);
  }
  DF_CHECK(aligned16(a->qkv) && aligned16(a->q) && aligned16(a->kb) && aligned16(a->vb) && aligned16(a->q_norm) &&
               aligned16(a->k_norm) && aligned16(a->rope_cs) && (!cache || (aligned16(a->kv.k) && aligned16(a->kv.v))),
           "%s: pointers must be 16-byte aligned", who);
  rc = check_ws(ws, ws_bytes, kReservedBytes, who);
  if (rc) return rc;
  QkNormDesc q = qk_norm_desc(a->dims, a->n_seqs * a->rows, a->rows, cache ? &a->kv : nullptr);
  q.src_dtype = a->qkv_dtype;
  q.base_pos = a->base_pos;
  q.qkv = a->qkv;
  if (a->qkv_stride) q.stride = a->qkv_stride;
  q.q_norm = a->q_norm;
  q.k_norm = a->k_norm;
  q.rope_cs = a->rope_cs;
  q.rope_max_pos = a->rope_max_pos;
  q.q = a->q;
  if (!cache) {
    q.k = a->kb;
    q.v = a->vb;
  }
  q.status = header(ws).status;
  const double heads = (double)q.M * (q.nq + 2 * q.nkv) * q.d;
  DF_LAUNCH((cudaStream_t)stream, TF_ROPE, heads * (elem_size(q.dtype) + elem_size(q.src_dtype)),
            launch_qk_norm(q, (cudaStream_t)stream));
  return DFLASH_OK;
}

// ------------------------------------------------------------- attention

static int check_prompt_attention_shape(const dflash_prompt_attention_args* a, const char* who) {
  DF_CHECK(a != nullptr, "%s: NULL args", who);
  int rc = check_dims(a->dims, who);
  if (rc) return rc;
  DF_CHECK(a->scale >= 0.f && a->scale < 1e30f, "%s: scale must be >= 0 and finite", who);
  return check_prompt_shape(a->dims, a->n_seqs, a->n_rows, a->base_pos != nullptr, a->max_pos, a->kv, who);
}

int dflash_prompt_attention(const dflash_prompt_attention_args* a, void* ws, size_t ws_bytes, dflash_stream_t stream) {
  const char* who = "dflash_prompt_attention";
  int rc = check_prompt_attention_shape(a, who);
  if (rc) return rc;
  DF_CHECK(a->row_start && a->q && a->kb && a->vb && a->out, "%s: NULL pointer", who);
  DF_CHECK(aligned16(a->q) && aligned16(a->kb) && aligned16(a->vb) && aligned16(a->out),
           "%s: q, kb, vb and out must be 16-byte aligned", who);
  if (a->base_pos) {
    DF_CHECK(a->kv.k && a->kv.v, "%s: NULL cache pointer", who);
    DF_CHECK(aligned16(a->kv.k) && aligned16(a->kv.v), "%s: cache pointers must be 16-byte aligned", who);
  }
  const int sms = num_sms();
  PromptAttnDesc p =
      prompt_attn_desc(a->dims, a->n_seqs, a->n_rows, a->base_pos != nullptr, a->max_pos, a->kv, a->scale);
  rc = check_ws(ws, ws_bytes, kReservedBytes + prompt_attn_workspace(p, sms), who);
  if (rc) return rc;
  p.row_start = a->row_start;
  p.base_pos = a->base_pos;
  p.q = a->q;
  p.kb = a->kb;
  p.vb = a->vb;
  p.out = a->out;
  p.work = static_cast<char*>(ws) + kReservedBytes;
  p.counters = header(ws).counters + kCtrAttn;
  p.status = header(ws).status;
  DF_LAUNCH((cudaStream_t)stream, TF_ATTN, 0, launch_prompt_attention(p, sms, (cudaStream_t)stream));
  return DFLASH_OK;
}

// ------------------------------------------------------ log probabilities

static int check_logprobs_shape(const dflash_token_logprobs_args* a, const char* who) {
  DF_CHECK(a != nullptr, "%s: NULL args", who);
  DF_CHECK(a->dims.vocab > 0 && a->dims.vocab < (1 << 28), "%s: vocab must be in [1, 2^28)", who);
  DF_CHECK(a->n_rows > 0 && a->n_rows <= (1 << 24), "%s: n_rows must be in [1, 2^24]", who);
  DF_CHECK(a->temperature >= 1e-6f && a->temperature < 1e30f, "%s: temperature must be at least 1e-6 and finite", who);
  DF_CHECK(a->topk >= 0 && a->topk <= DFLASH_MAX_LOGPROBS && a->topk <= a->dims.vocab,
           "%s: topk must be in [0, %d] and at most the vocabulary", who, DFLASH_MAX_LOGPROBS);
  return DFLASH_OK;
}

int dflash_token_logprobs(const dflash_token_logprobs_args* a, void* ws, size_t ws_bytes, dflash_stream_t stream) {
  const char* who = "dflash_token_logprobs";
  int rc = check_logprobs_shape(a, who);
  if (rc) return rc;
  DF_CHECK(a->logits, "%s: logits is NULL", who);
  DF_CHECK((reinterpret_cast<uintptr_t>(a->logits) & 3) == 0, "%s: logits must be 4-byte aligned", who);
  DF_CHECK((a->tokens == nullptr) == (a->logprob == nullptr), "%s: tokens and logprob go together", who);
  DF_CHECK(a->topk == 0 || (a->top_ids && a->top_logprobs), "%s: topk needs top_ids and top_logprobs", who);
  DF_CHECK(a->logprob || a->entropy || a->topk > 0, "%s: no output", who);
  rc = check_ws(ws, ws_bytes, kReservedBytes, who);
  if (rc) return rc;
  LogprobDesc d;
  memset(&d, 0, sizeof(d));
  d.M = a->n_rows;
  d.V = a->dims.vocab;
  d.topk = a->topk;
  d.invT = 1.f / a->temperature;
  d.logits = a->logits;
  d.tokens = a->tokens;
  d.logprob = a->logprob;
  d.entropy = a->entropy;
  d.top_ids = a->top_ids;
  d.top_logprobs = a->top_logprobs;
  d.status = header(ws).status;
  DF_LAUNCH((cudaStream_t)stream, TF_SAMPLE, (double)d.M * d.V * 4,
            launch_token_logprobs(d, num_sms(), (cudaStream_t)stream));
  return DFLASH_OK;
}

}  // extern "C"

namespace dfl {

size_t prompt_op_workspace(int op, const void* args, const char* who) {
  switch (op) {
    case DFLASH_OP_QK_NORM_ROPE:
      return check_qk_norm_shape(static_cast<const dflash_qk_norm_rope_args*>(args), who) ? 0 : kReservedBytes;
    case DFLASH_OP_PROMPT_ATTENTION: {
      const dflash_prompt_attention_args* a = static_cast<const dflash_prompt_attention_args*>(args);
      if (check_prompt_attention_shape(a, who)) return 0;
      return kReservedBytes + prompt_attn_workspace(prompt_attn_desc(a->dims, a->n_seqs, a->n_rows, a->base_pos != nullptr,
                                                                     a->max_pos, a->kv, a->scale),
                                                    num_sms());
    }
    case DFLASH_OP_TOKEN_LOGPROBS:
      return check_logprobs_shape(static_cast<const dflash_token_logprobs_args*>(args), who) ? 0 : kReservedBytes;
  }
  return 0;
}

}  // namespace dfl
