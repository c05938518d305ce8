// w4_serve_api.cu -- the C entry points of the paged 8-bit cache, the attention over it and the draft
// verification (include/w4.h): argument checks on the host, then one launch call each.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/w4.h"
#include "w4_internal.h"
#include "w4_serve.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int launched(cudaError_t e) { return e == cudaErrorNotSupported ? W4_ERR_UNSUPPORTED : w4::cuda_status(e); }

// The cache's fields, with the strides that 0 stands for filled in.
int check_cache(const w4_kv_cache* c, w4::KvView* v) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || !c->page_table) return W4_ERR_NULL;
  if (c->num_pages < 1 || c->kv_heads < 1 || c->table_stride < 1) return W4_ERR_SHAPE;
  const int P = c->page_tokens;
  if (P != 16 && P != 32 && P != 64 && P != 128) return W4_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128) return W4_ERR_UNSUPPORTED;
  const int64_t page_bytes = (int64_t)c->kv_heads * P * c->head_dim;
  const int64_t ps = c->page_stride ? c->page_stride : page_bytes;
  const int64_t ss = c->scale_stride ? c->scale_stride : c->kv_heads;
  if (ps < page_bytes || ss < c->kv_heads) return W4_ERR_SHAPE;
  if (page_bytes > INT32_MAX || ps >= ((int64_t)1 << 40)) return W4_ERR_UNSUPPORTED;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || (ps & 15) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
      !aligned(c->page_table, 4))
    return W4_ERR_ALIGN;
  *v = w4::KvView{c->k, c->v, c->k_scale, c->v_scale, c->page_table, (long long)ps, (long long)ss, c->num_pages,
                  c->kv_heads, P, c->head_dim, c->table_stride};
  return W4_OK;
}

// What describes the ragged batch.
int check_batch(const w4::KvView& c, const int32_t* q_start, const int32_t* kv_len, int tokens, int batch, int q_heads,
                int max_q) {
  if (!q_start || !kv_len) return W4_ERR_NULL;
  if (tokens < 0 || batch < 1 || q_heads < 1 || q_heads % c.kv_heads != 0 || max_q < 0) return W4_ERR_SHAPE;
  if (batch > W4_MAX_SEQS || q_heads / c.kv_heads > W4_MAX_GROUP) return W4_ERR_UNSUPPORTED;
  if (tokens > (1 << 28) / q_heads) return W4_ERR_UNSUPPORTED;     // rows are counted in 32 bits
  if (!aligned(q_start, 4) || !aligned(kv_len, 4)) return W4_ERR_ALIGN;
  return W4_OK;
}

// A row stride in elements: 0 stands for `dense`.
int check_stride(int64_t given, int64_t dense, long long* out) {
  *out = given ? given : dense;
  if (*out < dense) return W4_ERR_SHAPE;
  return (*out & 7) ? W4_ERR_ALIGN : W4_OK;
}

}  // namespace

extern "C" {

int w4_kv_append(const w4_kv_cache* cache, const uint16_t* q, const uint16_t* k, const uint16_t* v, uint16_t* q_out,
                 const float* rope_cos, const float* rope_sin, const int32_t* positions, const int32_t* q_start,
                 const int32_t* kv_len, int tokens, int batch, int q_heads, int max_q, int max_position,
                 int rotary_dim, int interleaved, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                 int64_t q_out_stride, w4_stream_t stream) {
  w4::AppendArgs a;
  int s = check_cache(cache, &a.c);
  if (s != W4_OK) return s;
  if (!k || !v || !q != !q_out) return W4_ERR_NULL;
  if ((s = check_batch(a.c, q_start, kv_len, tokens, batch, q_heads, max_q)) != W4_OK) return s;
  const int D = a.c.dim;
  if (rotary_dim < 0 || rotary_dim > D || rotary_dim % 16 != 0) return W4_ERR_SHAPE;
  if (rotary_dim > 0 && (!rope_cos || !rope_sin)) return W4_ERR_NULL;
  if (rotary_dim > 0 && max_position < 1) return W4_ERR_SHAPE;
  const int64_t dq = (int64_t)q_heads * D, dkv = (int64_t)a.c.kv_heads * D;
  if ((s = check_stride(q_stride, dq, &a.q_stride)) != W4_OK || (s = check_stride(k_stride, dkv, &a.k_stride)) != W4_OK ||
      (s = check_stride(v_stride, dkv, &a.v_stride)) != W4_OK ||
      (s = check_stride(q_out_stride, dq, &a.q_out_stride)) != W4_OK)
    return s;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) ||
      (rotary_dim > 0 && (!aligned(rope_cos, 16) || !aligned(rope_sin, 16))) || !aligned(positions, 4))
    return W4_ERR_ALIGN;
  if (tokens == 0 || max_q == 0) return W4_OK;
  a.q = reinterpret_cast<const __half*>(q);
  a.k = reinterpret_cast<const __half*>(k);
  a.v = reinterpret_cast<const __half*>(v);
  a.q_out = reinterpret_cast<__half*>(q_out);
  a.cos = rope_cos;
  a.sin = rope_sin;
  a.positions = positions;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.tokens = tokens;
  a.batch = batch;
  a.q_heads = q_heads;
  a.max_q = max_q < tokens ? max_q : tokens;
  a.max_position = max_position;
  a.rotary_dim = rotary_dim;
  a.interleaved = interleaved ? 1 : 0;
  return launched(w4::launch_kv_append(a, reinterpret_cast<cudaStream_t>(stream)));
}

int w4_kv_append_block(const w4_kv_append_args* p) {
  if (!p) return W4_ERR_NULL;
  return w4_kv_append(p->cache, p->q, p->k, p->v, p->q_out, p->rope_cos, p->rope_sin, p->positions, p->q_start,
                      p->kv_len, p->tokens, p->batch, p->q_heads, p->max_q, p->max_position, p->rotary_dim,
                      p->interleaved, p->q_stride, p->k_stride, p->v_stride, p->q_out_stride, p->stream);
}

int64_t w4_attn_workspace_bytes(int tokens, int batch, int q_heads, int kv_heads, int head_dim) {
  if (tokens < 0 || batch < 1 || q_heads < 1 || kv_heads < 1 || (head_dim != 64 && head_dim != 128)) return 0;
  return w4::attn_workspace_bytes(tokens, batch, q_heads, kv_heads, head_dim);
}

int w4_attn_kv8(const w4_kv_cache* cache, const uint16_t* q, uint16_t* out, float* lse, const int32_t* q_start,
                const int32_t* kv_len, int tokens, int batch, int q_heads, int max_q, float softmax_scale, int causal,
                int window, int64_t q_stride, int64_t out_stride, void* workspace, int64_t workspace_bytes,
                w4_stream_t stream) {
  w4::AttnArgs a;
  int s = check_cache(cache, &a.c);
  if (s != W4_OK) return s;
  if (!q || !out || !workspace) return W4_ERR_NULL;
  if ((s = check_batch(a.c, q_start, kv_len, tokens, batch, q_heads, max_q)) != W4_OK) return s;
  if (window < 0 || !std::isfinite(softmax_scale) || softmax_scale <= 0.f) return W4_ERR_SHAPE;
  const int64_t dq = (int64_t)q_heads * a.c.dim;
  if ((s = check_stride(q_stride, dq, &a.q_stride)) != W4_OK || (s = check_stride(out_stride, dq, &a.out_stride)) != W4_OK)
    return s;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 16)) return W4_ERR_ALIGN;
  if (workspace_bytes < w4::attn_workspace_bytes(tokens, batch, q_heads, a.c.kv_heads, a.c.dim)) return W4_ERR_SHAPE;
  if (tokens == 0 || max_q == 0) return W4_OK;
  a.q = reinterpret_cast<const __half*>(q);
  a.out = reinterpret_cast<__half*>(out);
  a.lse = lse;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.tokens = tokens;
  a.batch = batch;
  a.q_heads = q_heads;
  a.max_q = max_q < tokens ? max_q : tokens;
  a.scale = softmax_scale;
  a.causal = causal ? 1 : 0;
  a.window = window;
  a.workspace = workspace;
  return launched(w4::launch_attn(a, reinterpret_cast<cudaStream_t>(stream)));
}

int w4_attn_kv8_block(const w4_attn_kv8_args* p) {
  if (!p) return W4_ERR_NULL;
  return w4_attn_kv8(p->cache, p->q, p->out, p->lse, p->q_start, p->kv_len, p->tokens, p->batch, p->q_heads, p->max_q,
                     p->softmax_scale, p->causal, p->window, p->q_stride, p->out_stride, p->workspace,
                     p->workspace_bytes, p->stream);
}

int64_t w4_spec_verify_workspace_bytes(int batch, int drafts, int vocab) {
  if (batch < 1 || drafts < 1 || drafts > W4_MAX_DRAFTS || vocab < 1) return 0;
  return w4::verify_workspace_bytes(batch, drafts, vocab);
}

int w4_spec_verify(const uint16_t* target, const uint16_t* draft, const int32_t* draft_tokens, const float* u,
                   const float* e, int32_t* tokens, int32_t* accepted, float* logprob, int batch, int drafts,
                   int vocab, float temperature, const int32_t* n_drafts, int64_t target_stride,
                   int64_t draft_stride, void* workspace, int64_t workspace_bytes, w4_stream_t stream) {
  if (!target || !draft_tokens || !tokens || !accepted || !workspace) return W4_ERR_NULL;
  if (!(temperature >= 0.f) || !std::isfinite(temperature)) return W4_ERR_SHAPE;
  if (temperature > 0.f && (!u || !e)) return W4_ERR_NULL;
  if (batch < 1 || drafts < 1 || vocab < 1) return W4_ERR_SHAPE;
  // below 1e-4 the exponents leave FP32's range: that is temperature 0
  if (drafts > W4_MAX_DRAFTS || vocab > (1 << 24) || batch > (1 << 20) || (temperature > 0.f && temperature < 1e-4f))
    return W4_ERR_UNSUPPORTED;
  w4::VerifyArgs a;
  a.target_stride = target_stride ? target_stride : vocab;
  a.draft_stride = draft_stride ? draft_stride : vocab;
  if (a.target_stride < vocab || a.draft_stride < vocab) return W4_ERR_SHAPE;
  if (!aligned(target, 2) || !aligned(draft, 2) || !aligned(draft_tokens, 4) || !aligned(u, 4) || !aligned(e, 4) ||
      !aligned(tokens, 4) || !aligned(accepted, 4) || !aligned(logprob, 4) || !aligned(n_drafts, 4) ||
      !aligned(workspace, 16))
    return W4_ERR_ALIGN;
  if (workspace_bytes < w4::verify_workspace_bytes(batch, drafts, vocab)) return W4_ERR_SHAPE;
  a.target = reinterpret_cast<const __half*>(target);
  a.draft = reinterpret_cast<const __half*>(draft);
  a.draft_tokens = draft_tokens;
  a.u = u;
  a.e = e;
  a.tokens = tokens;
  a.accepted = accepted;
  a.logprob = logprob;
  a.batch = batch;
  a.drafts = drafts;
  a.vocab = vocab;
  a.temperature = temperature;
  a.n_drafts = n_drafts;
  a.workspace = workspace;
  return launched(w4::launch_verify(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
