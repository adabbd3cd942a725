// C ABI of the serving operators (include/mpk.h): checks of arguments and
// launches.  Nothing is allocated and nothing throws.
#include <cuda_runtime.h>

#include <cmath>

#include "graph_state.h"
#include "launch.h"
#include "mpk.h"
#include "serve.h"

using namespace mpk;

namespace {

mpk_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return MPK_OK;
  cudaGetLastError();   // a failed launch leaves no error behind
  return e == cudaErrorMemoryAllocation ? MPK_ERR_OOM : MPK_ERR_CUDA;
}
bool off(const void* p, unsigned a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0;
}
// a row of `width` 16-bit values every `stride`, in 16-byte steps
bool bad_rows(const void* p, int64_t stride, int64_t width) {
  return !p || off(p, 16) || stride < width || stride % 8;
}

mpk_status check_shape(const mpk_attn_shape* s) {
  if (!s || s->n_q_heads < 1 || s->n_kv_heads < 1 || s->page_size < 1 ||
      s->max_pages_per_seq < 1 || s->n_q_heads % s->n_kv_heads)
    return MPK_ERR_INVALID_ARG;
  if (s->head_dim != 32 && s->head_dim != 64 && s->head_dim != 128)
    return MPK_ERR_UNSUPPORTED;
  if ((int64_t)s->page_size * s->max_pages_per_seq > 0x40000000)
    return MPK_ERR_UNSUPPORTED;         // positions are 32-bit numbers
  return MPK_OK;
}
mpk_status check_batch(const mpk_token_batch* t) {
  if (!t || t->batch < 1 || t->n_tokens < 0) return MPK_ERR_INVALID_ARG;
  if (t->batch > (1 << 20)) return MPK_ERR_UNSUPPORTED;
  if (t->q_start) return off(t->q_start, 4) ? MPK_ERR_INVALID_ARG : MPK_OK;
  if (t->tokens_per_seq < 0 ||
      (int64_t)t->batch * t->tokens_per_seq > t->n_tokens)
    return MPK_ERR_INVALID_ARG;
  return MPK_OK;
}

mpk_status fill_paged(const mpk_attn_shape* s, const mpk_token_batch* t,
                      const mpk_kv_cache* kv, int layer, uint32_t* d_status,
                      PagedArgs* p) {
  mpk_status st = check_shape(s);
  if (st != MPK_OK) return st;
  st = check_batch(t);
  if (st != MPK_OK) return st;
  if (!kv || !kv->k_pool || !kv->v_pool || !kv->page_table ||
      !kv->seq_lens || kv->num_pages < 1 || layer < 0 ||
      off(kv->k_pool, 16) || off(kv->v_pool, 16) || off(kv->page_table, 4) ||
      off(kv->seq_lens, 4) || off(d_status, 4))
    return MPK_ERR_INVALID_ARG;
  // rows of the pool are 32-bit numbers (2^32 of them are more than the
  // memory: 64 bytes each at least)
  const double rows = (double)kv->num_pages * s->n_kv_heads * s->page_size;
  if (rows > 4294967295.0) return MPK_ERR_UNSUPPORTED;
  const int64_t stride = (int64_t)kv->num_pages * s->n_kv_heads *
                         s->page_size * s->head_dim;
  p->k = static_cast<uint16_t*>(kv->k_pool) + layer * stride;
  p->v = static_cast<uint16_t*>(kv->v_pool) + layer * stride;
  p->page_table = kv->page_table;
  p->seq_lens = kv->seq_lens;
  p->q_start = t->q_start;
  p->tokens_per_seq = t->tokens_per_seq;
  p->batch = t->batch;
  p->n_tokens = t->n_tokens;
  p->num_pages = kv->num_pages;
  p->page_size = s->page_size;
  p->max_pages = s->max_pages_per_seq;
  p->page_div = fast_div((uint32_t)s->page_size);
  p->grp_div = fast_div((uint32_t)(s->n_q_heads / s->n_kv_heads));
  p->Hq = s->n_q_heads;
  p->Hkv = s->n_kv_heads;
  p->d = s->head_dim;
  p->status = d_status;
  return MPK_OK;
}

}  // namespace

extern "C" {

mpk_status mpk_rope_table(const mpk_rope_scaling* s, int64_t first_pos,
                          int n_pos, float* d_table, void* cuda_stream) {
  if (!s || !d_table || off(d_table, 4) || first_pos < 0 || n_pos < 0 ||
      s->rotary_dim < 2 || s->rotary_dim % 2 || !(s->theta > 0.0) ||
      s->scaling < MPK_ROPE_PLAIN || s->scaling > MPK_ROPE_RAMP)
    return MPK_ERR_INVALID_ARG;
  if (s->scaling != MPK_ROPE_PLAIN && !(s->factor > 0.0))
    return MPK_ERR_INVALID_ARG;
  if (s->scaling >= MPK_ROPE_BANDS &&
      !(s->low > 0.0 && s->high > s->low && s->old_ctx > 0.0))
    return MPK_ERR_INVALID_ARG;
  if (s->scaling == MPK_ROPE_RAMP && s->theta == 1.0)
    return MPK_ERR_INVALID_ARG;
  if (n_pos == 0) return MPK_OK;
  RopeTableArgs a{};
  a.out = d_table;
  a.first_pos = first_pos;
  a.n_pos = n_pos;
  a.rot = s->rotary_dim;
  a.scaling = s->scaling;
  a.theta = s->theta;
  a.factor = s->factor;
  a.low = s->low;
  a.high = s->high;
  a.old_ctx = s->old_ctx;
  a.attn_factor = s->attn_factor == 0.0 ? 1.0 : s->attn_factor;
  return from_cuda(launch_rope_table(a, static_cast<cudaStream_t>(cuda_stream)));
}

mpk_status mpk_kv_append(const mpk_attn_shape* shape,
                         const mpk_token_batch* tok, const mpk_kv_cache* kv,
                         int layer, const void* d_q, int64_t q_stride,
                         const void* d_k, int64_t k_stride, const void* d_v,
                         int64_t v_stride, const void* d_q_norm,
                         const void* d_k_norm, float eps,
                         const mpk_rope* rope, void* d_q_out,
                         int64_t q_out_stride, uint32_t* d_status,
                         void* cuda_stream) {
  AppendArgs a{};
  mpk_status st = fill_paged(shape, tok, kv, layer, d_status, &a.p);
  if (st != MPK_OK) return st;
  if (a.p.n_tokens == 0) return MPK_OK;   // (empty tensors have no address)
  const int64_t wq = (int64_t)a.p.Hq * a.p.d, wk = (int64_t)a.p.Hkv * a.p.d;
  if (bad_rows(d_k, k_stride, wk) || bad_rows(d_v, v_stride, wk) ||
      (d_q_out && (bad_rows(d_q, q_stride, wq) ||
                   bad_rows(d_q_out, q_out_stride, wq))) ||
      off(d_q_norm, 16) || off(d_k_norm, 16) || !(eps >= 0.f))
    return MPK_ERR_INVALID_ARG;
  if (rope && rope->rotary_dim != 0) {
    if (rope->rotary_dim < 0 || !rope->table || off(rope->table, 16) ||
        rope->n_pos < 1)
      return MPK_ERR_INVALID_ARG;
    if (rope->rotary_dim % 16 || rope->rotary_dim > a.p.d)
      return MPK_ERR_UNSUPPORTED;
    a.table = rope->table;
    a.n_pos = rope->n_pos;
    a.rot = rope->rotary_dim;
    a.interleaved = rope->interleaved ? 1 : 0;
  }
  a.q = static_cast<const uint16_t*>(d_q);
  a.k = static_cast<const uint16_t*>(d_k);
  a.v = static_cast<const uint16_t*>(d_v);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_norm = static_cast<const uint16_t*>(d_q_norm);
  a.k_norm = static_cast<const uint16_t*>(d_k_norm);
  a.eps = eps;
  a.q_out = static_cast<uint16_t*>(d_q_out);
  a.q_out_stride = q_out_stride;
  return from_cuda(launch_append(a, static_cast<cudaStream_t>(cuda_stream)));
}

// Sizes that the attention's 32-bit row and unit numbers hold.
static bool attend_too_large(const PagedArgs& p) {
  return (int64_t)p.n_tokens * p.Hq > 0x3fffffff ||
         (int64_t)p.batch * p.Hkv > 0x3fffffff;
}

size_t mpk_prefix_attention_workspace(const mpk_attn_shape* shape,
                                      const mpk_token_batch* tok,
                                      int n_groups) {
  if (check_shape(shape) != MPK_OK || !tok || tok->batch < 1 ||
      tok->batch > (1 << 20) || tok->n_tokens < 0 || n_groups < 0 ||
      n_groups > tok->batch)
    return 0;
  AttendArgs a{};
  a.p.batch = tok->batch;
  a.p.n_tokens = tok->n_tokens;
  a.p.page_size = shape->page_size;
  a.p.max_pages = shape->max_pages_per_seq;
  a.p.Hq = shape->n_q_heads;
  a.p.Hkv = shape->n_kv_heads;
  a.p.d = shape->head_dim;
  a.n_groups = n_groups;
  if (attend_too_large(a.p)) return 0;
  // enough for whichever launches the call chooses
  a.scale_log2 = 1.f;
  a.p.num_pages = 1;
  const size_t x = attend_workspace(&a, nullptr);
  a.scale_log2 = -1.f;
  const size_t y = attend_workspace(&a, nullptr);
  return x > y ? x : y;
}

mpk_status mpk_prefix_attention(const mpk_attn_shape* shape,
                                const mpk_token_batch* tok,
                                const mpk_prefix_groups* groups,
                                const mpk_kv_cache* kv, int layer,
                                const void* d_q, int64_t q_stride, float scale,
                                void* d_out, int64_t out_stride, float* d_lse,
                                void* d_workspace, size_t workspace_bytes,
                                uint32_t* d_status, void* cuda_stream) {
  AttendArgs a{};
  mpk_status st = fill_paged(shape, tok, kv, layer, d_status, &a.p);
  if (st != MPK_OK) return st;
  if (a.p.n_tokens == 0) return MPK_OK;
  const int64_t wq = (int64_t)a.p.Hq * a.p.d;
  if (bad_rows(d_q, q_stride, wq) || bad_rows(d_out, out_stride, wq) ||
      d_out == d_q || off(d_lse, 4) || !std::isfinite(scale))
    return MPK_ERR_INVALID_ARG;
  if (groups) {
    if (groups->n_groups < 1 || groups->n_groups > a.p.batch ||
        !groups->group_start || !groups->prefix_len ||
        off(groups->group_start, 4) || off(groups->prefix_len, 4))
      return MPK_ERR_INVALID_ARG;
    a.n_groups = groups->n_groups;
    a.group_start = groups->group_start;
    a.prefix_len = groups->prefix_len;
  }
  if (attend_too_large(a.p)) return MPK_ERR_UNSUPPORTED;
  const double s = scale != 0.f ? (double)scale
                                : 1.0 / std::sqrt((double)a.p.d);
  a.scale_log2 = (float)(s * 1.4426950408889634074);
  if (!d_workspace || off(d_workspace, 256) ||
      workspace_bytes < attend_workspace(&a, static_cast<char*>(d_workspace)))
    return MPK_ERR_INVALID_ARG;
  a.q = static_cast<const uint16_t*>(d_q);
  a.q_stride = q_stride;
  a.out = static_cast<uint16_t*>(d_out);
  a.out_stride = out_stride;
  a.lse = d_lse;
  return from_cuda(launch_attend(a, static_cast<cudaStream_t>(cuda_stream)));
}

static bool verify_sizes(const mpk_token_batch* t, int vocab) {
  return vocab >= 1 && vocab < (1 << 30) && t->n_tokens <= 65535 &&
         t->batch <= 65535;
}

size_t mpk_verify_drafts_workspace(const mpk_token_batch* tok, int vocab) {
  if (!tok || tok->batch < 1 || tok->n_tokens < 0 || !verify_sizes(tok, vocab))
    return 0;
  VerifyArgs a{};
  a.batch = tok->batch;
  a.n_tokens = tok->n_tokens;
  a.vocab = vocab;
  return verify_workspace(&a, nullptr);
}

static mpk_status check_verify(const mpk_token_batch* tok,
                               const mpk_verify_args* v,
                               const uint32_t* d_status) {
  mpk_status st = check_batch(tok);
  if (st != MPK_OK) return st;
  const bool none = tok->n_tokens == 0;   // outputs alone are written
  if (!v || v->vocab < 1 || v->max_out < 1 || (!none && !v->tokens) ||
      (!none && !v->logits) || (!none && !v->uniform) || !v->noise ||
      !v->n_accepted || !v->out_tokens || v->logits_stride < v->vocab || v->noise_stride < v->vocab ||
      (v->draft && v->draft_stride < v->vocab) || off(v->tokens, 4) ||
      off(v->logits, 4) || off(v->draft, 4) || off(v->temperature, 4) ||
      off(v->uniform, 4) || off(v->noise, 4) || off(v->n_accepted, 4) ||
      off(v->out_tokens, 4) || off(v->logprobs, 4) || off(v->next_tokens, 4) ||
      off(v->seq_lens, 4) || off(v->seq_lens_out, 4) || off(d_status, 4))
    return MPK_ERR_INVALID_ARG;
  if (!verify_sizes(tok, v->vocab) || v->max_out > 128)
    return MPK_ERR_UNSUPPORTED;
  if (!tok->q_start && tok->tokens_per_seq > v->max_out)
    return MPK_ERR_INVALID_ARG;
  return MPK_OK;
}

mpk_status mpk_verify_drafts(const mpk_token_batch* tok,
                             const mpk_verify_args* v, void* d_workspace,
                             size_t workspace_bytes, uint32_t* d_status,
                             void* cuda_stream) {
  const mpk_status st = check_verify(tok, v, d_status);
  if (st != MPK_OK) return st;
  VerifyArgs a{};
  a.batch = tok->batch;
  a.n_tokens = tok->n_tokens;
  a.vocab = v->vocab;
  a.max_out = v->max_out;
  a.draft = v->draft;
  a.draft_is_logits = v->draft_is_logits;
  a.q_start = tok->q_start;
  a.tokens_per_seq = tok->tokens_per_seq;
  if (!d_workspace || off(d_workspace, 256) ||
      workspace_bytes < verify_workspace(&a, static_cast<char*>(d_workspace)))
    return MPK_ERR_INVALID_ARG;
  a.tokens = v->tokens;
  a.logits = v->logits;
  a.logits_stride = v->logits_stride;
  a.draft = v->draft;
  a.draft_stride = v->draft_stride;
  a.draft_is_logits = v->draft_is_logits;
  a.temperature = v->temperature;
  a.uniform = v->uniform;
  a.noise = v->noise;
  a.noise_stride = v->noise_stride;
  a.n_accepted = v->n_accepted;
  a.out_tokens = v->out_tokens;
  a.logprobs = v->logprobs;
  a.next_tokens = v->next_tokens;
  a.seq_lens = v->seq_lens;
  a.seq_lens_out = v->seq_lens_out;
  a.status = d_status;
  return from_cuda(launch_verify(a, static_cast<cudaStream_t>(cuda_stream)));
}

// The graph's heads and cache geometry.
static mpk_attn_shape graph_shape(const mpk_graph* g) {
  const mpk_model_shape& s = g->bg.cfg.shape;
  return mpk_attn_shape{s.n_q_heads, s.n_kv_heads, s.head_dim, s.page_size,
                        s.max_pages_per_seq};
}

size_t mpk_verify_step_workspace(const mpk_graph* g,
                                 const mpk_token_batch* tok, int n_groups) {
  if (!g || !tok || g->bg.cfg.shape.chain_ffn > 0 ||
      tok->n_tokens != g->bg.cfg.batch)
    return 0;
  // the attention's workspace is free again when the drafts are judged
  const mpk_attn_shape s = graph_shape(g);
  const size_t a = mpk_prefix_attention_workspace(&s, tok, n_groups);
  const size_t b = mpk_verify_drafts_workspace(tok, g->bg.cfg.shape.vocab);
  return a == 0 || b == 0 ? 0 : a > b ? a : b;
}

mpk_status mpk_verify_step(mpk_graph* g, const mpk_token_batch* tok,
                           const mpk_prefix_groups* groups,
                           const mpk_kv_cache* kv, const mpk_verify_args* v,
                           float* d_logits, void* d_workspace,
                           size_t workspace_bytes, void* cuda_stream) {
  if (!g || !v || !d_logits || !v->tokens) return MPK_ERR_INVALID_ARG;
  if (!g->bound) return MPK_ERR_NOT_BOUND;
  const mpk_model_shape& s = g->bg.cfg.shape;
  if (s.chain_ffn > 0) return MPK_ERR_UNSUPPORTED;
  const mpk_attn_shape shape = graph_shape(g);
  mpk_status st = check_batch(tok);
  if (st != MPK_OK) return st;
  if (tok->n_tokens != g->bg.cfg.batch || tok->batch > tok->n_tokens)
    return MPK_ERR_INVALID_ARG;
  uint32_t* status = g->d_status.p;
  PagedArgs probe{};                    // what the launches below would refuse
  st = fill_paged(&shape, tok, kv, 0, status, &probe);
  if (st != MPK_OK) return st;
  const size_t need =
      mpk_verify_step_workspace(g, tok, groups ? groups->n_groups : 0);
  if (need == 0 || !d_workspace || off(d_workspace, 256) ||
      workspace_bytes < need)
    return MPK_ERR_INVALID_ARG;
  mpk_verify_args judge = *v;
  judge.vocab = s.vocab;
  judge.logits = d_logits;
  judge.logits_stride = s.vocab;
  judge.seq_lens = kv->seq_lens;
  st = check_verify(tok, &judge, status);
  if (st != MPK_OK) return st;
  if (cudaSetDevice(g->device) != cudaSuccess) return MPK_ERR_CUDA;
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  KernelParams P = g->params;
  StepArgs a{};
  a.tokens = v->tokens;
  a.logits = d_logits;
  a.timeout_ns = g->timeout_ns;
  a.n_steps = 1;
  a.k_pool = static_cast<uint16_t*>(kv->k_pool);
  a.v_pool = static_cast<uint16_t*>(kv->v_pool);
  a.page_table = kv->page_table;
  a.seq_lens = kv->seq_lens;
  a.num_pages = kv->num_pages;
  a.epoch = g->epoch;
  P.step = a;
  const int64_t wq = (int64_t)s.n_q_heads * s.head_dim,
                wk = (int64_t)s.n_kv_heads * s.head_dim, row = wq + 2 * wk;
  const mpk_rope rope{g->d_rope.p, P.dims.max_ctx, s.head_dim, 0};
  for (size_t o = 0; o < g->bg.ops.size(); ++o) {
    const BOp& op = g->bg.ops[o];
    if (op.kind == MPK_TASK_ARGMAX) continue;
    if (op.kind != MPK_TASK_ATTN) {
      const cudaError_t e =
          launch_kpo_op(P, g->h_op_first[o], op.n, g->smem, stream);
      if (e != cudaSuccess) return from_cuda(e);
      continue;
    }
    char* layer = P.act.base + (int64_t)op.layer * P.act.layer_stride;
    uint16_t* q = reinterpret_cast<uint16_t*>(layer + P.act.o_qkv);
    const uint16_t* const* w =
        g->h_layer_ptrs.data() + (size_t)op.layer * MPK_LAYER_NTENSORS;
    st = mpk_kv_append(&shape, tok, kv, op.layer, q, row, q + wq, row,
                       q + wq + wk, row, s.qk_norm ? w[MPK_W_QNORM] : nullptr,
                       s.qk_norm ? w[MPK_W_KNORM] : nullptr, s.rms_eps, &rope,
                       q, row, status, cuda_stream);
    if (st != MPK_OK) return st;
    st = mpk_prefix_attention(&shape, tok, groups, kv, op.layer, q, row, 0.f,
                              layer + P.act.o_attn, wq, nullptr, d_workspace,
                              workspace_bytes, status, cuda_stream);
    if (st != MPK_OK) return st;
  }
  return mpk_verify_drafts(tok, &judge, d_workspace, workspace_bytes, status,
                           cuda_stream);
}

}  // extern "C"
