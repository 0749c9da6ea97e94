// Host entry points of whole prompts, their scores and a cache that is short
// of memory: argument checks of prompt attention, token log probabilities, the
// 4-bit cache, and eviction.
#include "pw_host.h"

using namespace pw;

struct pw_kv4_s {
  Kv4View view;
  KvView plain;   // what the attention kernels' shared parts read of it: shape and error word
};

namespace {

inline size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
inline bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255) == 0; }

// Rows that tensor copies read: strides (of more than one row) at least a row, below 2^39 bytes.
bool bad_strides(const pw_rows& r, int T, int heads, int d) {
  const long long lim = 1ll << 38;
  return (T > 1 && (r.token_stride < d || r.token_stride >= lim)) || (heads > 1 && (r.head_stride < d || r.head_stride >= lim));
}

// The kernels count tiles of keys x rows in 32 bits.
bool too_many_tiles(int batch, int q_len, int G, int hkv, long long keys) {
  return (double)batch * ((double)keys / 64 + 3) * ((double)q_len * G / 16 + 1) * hkv > 2e9;
}

}  // namespace

extern "C" pw_status pw_prompt_attend(const pw_heads* heads, const pw_prompt_desc* a, void* stream) {
  if (!heads || !a || bad_tokens(a->tokens) || a->batch < 0) return PW_ERR_INVALID_ARG;
  const pw_status st = check_heads(*heads);
  if (st != PW_OK) return st;
  if (a->batch > kMaxBatch) return PW_ERR_UNSUPPORTED;
  if (!std::isfinite(a->scale) || !aligned4(a->lse) || !aligned4(a->err)) return PW_ERR_INVALID_ARG;
  if (a->tokens > 0 && a->batch > 0) {
    for (const pw_rows* r : {&a->q, &a->k, &a->v, &a->out})
      if (bad_rows(r)) return PW_ERR_INVALID_ARG;
    if (bad_strides(a->q, a->tokens, heads->n_heads, heads->head_dim)) return PW_ERR_INVALID_ARG;
    for (const pw_rows* r : {&a->k, &a->v})
      if (bad_strides(*r, a->tokens, heads->n_kv_heads, heads->head_dim)) return PW_ERR_INVALID_ARG;
    if (!a->offsets || !aligned4(a->offsets)) return PW_ERR_INVALID_ARG;
  }
  if (host_sim()) return PW_ERR_UNSUPPORTED;
  if (a->tokens == 0 || a->batch == 0) return PW_OK;
  Range range("pw_prompt_attend");
  PromptParams P = {};
  P.q = a->q;
  P.k = a->k;
  P.v = a->v;
  P.out = a->out;
  P.lse = a->lse;
  P.offsets = a->offsets;
  P.err = a->err;
  P.T = a->tokens;
  P.B = a->batch;
  P.hq = heads->n_heads;
  P.hkv = heads->n_kv_heads;
  P.G = P.hq / P.hkv;
  P.scale = a->scale;
  return launched(launch_prompt(P, heads->dtype, heads->head_dim, as_stream(stream)));
}

extern "C" pw_status pw_prompt_check_device(void* stream) {
  if (host_sim()) return PW_ERR_UNSUPPORTED;
  int* word = nullptr;
  const cudaError_t e = prompt_error_word(&word);
  return e == cudaSuccess ? read_error(word, as_stream(stream)) : record_cuda_error(e);
}

extern "C" pw_status pw_token_logprobs(const pw_logprob_desc* a, void* stream) {
  if (!a || bad_tokens(a->T) || a->V < 1 || a->V > (1 << 24)) return PW_ERR_INVALID_ARG;
  if (a->dtype != PW_F16 && a->dtype != PW_BF16 && a->dtype != PW_F32) return PW_ERR_INVALID_ARG;
  if (a->n_top < 0 || a->n_top > a->V) return PW_ERR_INVALID_ARG;
  if (a->n_top > kMaxTop) return PW_ERR_UNSUPPORTED;
  const uintptr_t element = a->dtype == PW_F32 ? 3 : 1;
  if (a->T > 0) {
    if (!a->logits || (reinterpret_cast<uintptr_t>(a->logits) & element)) return PW_ERR_INVALID_ARG;
    for (const void* p : {(const void*)a->tokens, (const void*)a->logprobs})
      if (!p || !aligned4(p)) return PW_ERR_INVALID_ARG;
    if (a->n_top > 0 && (!a->top_ids || !a->top_logprobs)) return PW_ERR_INVALID_ARG;
    for (const void* p : {(const void*)a->entropy, (const void*)a->top_ids, (const void*)a->top_logprobs, (const void*)a->err})
      if (!aligned4(p)) return PW_ERR_INVALID_ARG;
  }
  if (host_sim()) return PW_ERR_UNSUPPORTED;
  if (a->T == 0) return PW_OK;
  Range range("pw_token_logprobs");
  const LogprobParams P = {a->logits,  a->row_stride, a->T,       a->V,       a->n_top,       a->tokens,
                           a->logprobs, a->entropy,    a->top_ids, a->top_logprobs, a->err};
  return launched(launch_logprobs(P, a->dtype, as_stream(stream)));
}

// ---- the cache in 4 bits ---------------------------------------------------------

extern "C" pw_status pw_kv4_create(const pw_kv4_desc* desc, void* k, void* v, void* k_steps, void* v_steps, int32_t* err,
                                   pw_kv4_t* out) {
  if (!desc || !k || !v || !k_steps || !v_steps || !err || !out) return PW_ERR_INVALID_ARG;
  const pw_status st = check_heads(desc->heads);
  if (st != PW_OK) return st;
  const int pt = desc->page_tokens;
  if (pt < 8 || pt > 1024 || (pt & (pt - 1)) || desc->n_pages < 1 || (long long)desc->n_pages * pt > 0x7fffffffll)
    return PW_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_steps) || !aligned16(v_steps) || !aligned4(err)) return PW_ERR_INVALID_ARG;
  Kv4View w = {};
  w.k = static_cast<char*>(k);
  w.v = static_cast<char*>(v);
  w.ks = static_cast<char*>(k_steps);
  w.vs = static_cast<char*>(v_steps);
  w.err = err;
  w.dtype = desc->heads.dtype;
  w.hq = desc->heads.n_heads;
  w.hkv = desc->heads.n_kv_heads;
  w.d = desc->heads.head_dim;
  while ((1 << w.page_shift) < pt) ++w.page_shift;
  w.n_pages = desc->n_pages;
  KvView p = {};
  p.err = err;
  p.dtype = w.dtype;
  p.hq = w.hq;
  p.hkv = w.hkv;
  p.d = w.d;
  p.page_shift = w.page_shift;
  p.n_pages = w.n_pages;
  auto* kv = new (std::nothrow) pw_kv4_s{w, p};
  if (!kv) return PW_ERR_OOM;
  *out = kv;
  return PW_OK;
}

extern "C" pw_status pw_kv4_destroy(pw_kv4_t kv) {
  if (!kv) return PW_ERR_INVALID_ARG;
  delete kv;
  return PW_OK;
}

extern "C" pw_status pw_kv4_check_device(pw_kv4_t kv, void* stream) {
  if (!kv) return PW_ERR_INVALID_ARG;
  if (host_sim()) return PW_ERR_UNSUPPORTED;
  return read_error(kv->view.err, as_stream(stream));
}

namespace {
pw_status rows4(pw_kv4_t kv, const int32_t* slots, int T, const pw_rows* k, const pw_rows* v, bool load, void* stream) {
  if (!kv || bad_tokens(T)) return PW_ERR_INVALID_ARG;
  if (T > 0 && (!slots || !aligned4(slots) || bad_rows(k) || bad_rows(v))) return PW_ERR_INVALID_ARG;
  if (host_sim()) return PW_ERR_UNSUPPORTED;
  if (T == 0) return PW_OK;
  Range range(load ? "pw_kv4_load" : "pw_kv4_append");
  const Row4Params P = {kv->view, *k, *v, slots, T};
  return launched(launch_rows4(P, load, as_stream(stream)));
}
}  // namespace

extern "C" pw_status pw_kv4_append(pw_kv4_t kv, const int32_t* slots, int T, const pw_rows* k, const pw_rows* v, void* stream) {
  return rows4(kv, slots, T, k, v, false, stream);
}

extern "C" pw_status pw_kv4_load(pw_kv4_t kv, const int32_t* slots, int T, const pw_rows* k, const pw_rows* v, void* stream) {
  return rows4(kv, slots, T, k, v, true, stream);
}

extern "C" pw_status pw_kv4_attend_workspace_size(pw_kv4_t kv, int batch, int q_len, size_t* bytes) {
  if (!kv || !bytes || batch < 0 || q_len < 1 || q_len > kMaxQLen) return PW_ERR_INVALID_ARG;
  if (batch > kMaxBatch) return PW_ERR_UNSUPPORTED;
  *bytes = attend4_ws_bytes(kv->plain, batch, q_len);
  return PW_OK;
}

extern "C" pw_status pw_kv4_attend(pw_kv4_t kv, const pw_attend_desc* a, void* ws, size_t ws_bytes, void* stream) {
  if (!kv || !a) return PW_ERR_INVALID_ARG;
  const KvView& w = kv->plain;
  size_t need = 0;
  const pw_status st = pw_kv4_attend_workspace_size(kv, a->batch, a->q_len, &need);
  if (st != PW_OK) return st;
  if (a->n_groups != 0) return a->n_groups < 0 ? PW_ERR_INVALID_ARG : PW_ERR_UNSUPPORTED;
  if (!std::isfinite(a->scale) || a->table_stride < 0) return PW_ERR_INVALID_ARG;
  const long long keys = (long long)a->table_stride << w.page_shift;
  if (keys > kMostKeys) return PW_ERR_INVALID_ARG;
  if (a->batch > 0) {
    if (bad_rows(&a->q) || bad_rows(&a->out) || !aligned4(a->lse)) return PW_ERR_INVALID_ARG;
    if (!a->lens || !aligned4(a->lens) || !aligned4(a->table) || (a->table_stride > 0 && !a->table)) return PW_ERR_INVALID_ARG;
    if (!ws || !aligned256(ws)) return PW_ERR_INVALID_ARG;
    if (ws_bytes < need) return PW_ERR_OOM;
  }
  if (too_many_tiles(a->batch, a->q_len, w.hq / w.hkv, w.hkv, keys)) return PW_ERR_UNSUPPORTED;
  if (host_sim()) return PW_ERR_UNSUPPORTED;
  if (a->batch == 0) return PW_OK;
  Range range("pw_kv4_attend");
  AttendParams P = {};
  P.kv = w;
  P.q = a->q;
  P.out = a->out;
  P.lse = a->lse;
  P.B = a->batch;
  P.ql = a->q_len;
  P.G = w.hq / w.hkv;
  P.scale = a->scale;
  P.table = a->table;
  P.table_stride = a->table_stride;
  P.lens = a->lens;
  return launched(launch_attend4(P, kv->view, ws, as_stream(stream)));
}

// ---- eviction --------------------------------------------------------------------

extern "C" pw_status pw_kv_weigh(pw_kv_t kv, const pw_weigh_desc* a, void* stream) {
  if (!kv || !a) return PW_ERR_INVALID_ARG;
  const KvView& w = kv->view;
  if (a->batch < 0 || a->q_len < 1 || a->q_len > kMaxQLen || a->table_stride < 0 || a->mass_stride < 0) return PW_ERR_INVALID_ARG;
  if (a->batch > kMaxBatch) return PW_ERR_UNSUPPORTED;
  if (!std::isfinite(a->scale) || !std::isfinite(a->decay)) return PW_ERR_INVALID_ARG;
  if (((long long)a->table_stride << w.page_shift) > kMostKeys || a->mass_stride > kMostKeys) return PW_ERR_INVALID_ARG;
  if (a->batch > 0) {
    if (bad_rows(&a->q) || !a->lse || !aligned4(a->lse) || !a->lens || !aligned4(a->lens)) return PW_ERR_INVALID_ARG;
    if (!aligned4(a->table) || (a->table_stride > 0 && !a->table)) return PW_ERR_INVALID_ARG;
    if (!aligned4(a->mass) || !aligned4(a->out) || (a->mass_stride > 0 && (!a->mass || !a->out))) return PW_ERR_INVALID_ARG;
  }
  if (host_sim()) return PW_ERR_UNSUPPORTED;
  if (a->batch == 0) return PW_OK;
  Range range("pw_kv_weigh");
  WeighParams P = {};
  P.kv = w;
  P.q = a->q;
  P.lse = a->lse;
  P.B = a->batch;
  P.ql = a->q_len;
  P.G = w.hq / w.hkv;
  P.scale = a->scale;
  P.decay = a->decay;
  P.table = a->table;
  P.table_stride = a->table_stride;
  P.lens = a->lens;
  P.mass = a->mass;
  P.out = a->out;
  P.mass_stride = a->mass_stride;
  return launched(launch_weigh(P, as_stream(stream)));
}

extern "C" pw_status pw_kv_evict_workspace_size(pw_kv_t kv, int batch, int budget, size_t* bytes) {
  if (!kv || !bytes || batch < 0 || budget < 1 || budget > (1 << 24)) return PW_ERR_INVALID_ARG;
  if (batch > kMaxBatch) return PW_ERR_UNSUPPORTED;
  *bytes = up256((size_t)batch * budget * 8) + up256((size_t)batch * 4);
  return PW_OK;
}

extern "C" pw_status pw_kv_evict(pw_kv_t kv, const pw_evict_desc* a, void* ws, size_t ws_bytes, void* stream) {
  if (!kv || !a) return PW_ERR_INVALID_ARG;
  const KvView& w = kv->view;
  size_t need = 0;
  const pw_status st = pw_kv_evict_workspace_size(kv, a->batch, a->budget, &need);
  if (st != PW_OK) return st;
  if (a->recent < 0 || a->table_stride < 0 || a->new_stride < 0 || a->mass_stride < 0) return PW_ERR_INVALID_ARG;
  const long long old_cap = (long long)a->table_stride << w.page_shift, new_cap = (long long)a->new_stride << w.page_shift;
  if (old_cap > kMostKeys || new_cap > kMostKeys || a->mass_stride > kMostKeys) return PW_ERR_INVALID_ARG;
  // what stays has to fit into the new table's row
  long long most = old_cap < a->mass_stride ? old_cap : a->mass_stride;
  if (most > a->budget) most = a->budget;
  if (new_cap < most) return PW_ERR_INVALID_ARG;
  if (a->batch > 0) {
    if (!a->lens || !aligned4(a->lens) || !a->new_lens || !aligned4(a->new_lens) || !aligned4(a->kept)) return PW_ERR_INVALID_ARG;
    for (const int32_t* t : {a->table, a->new_table})
      if (!aligned4(t) || (most > 0 && !t)) return PW_ERR_INVALID_ARG;
    for (const float* t : {a->mass, (const float*)a->new_mass})
      if (!aligned4(t) || (a->mass_stride > 0 && !t)) return PW_ERR_INVALID_ARG;
    if (!ws || !aligned256(ws)) return PW_ERR_INVALID_ARG;
    if (ws_bytes < need) return PW_ERR_OOM;
  }
  if (host_sim()) return PW_ERR_UNSUPPORTED;
  if (a->batch == 0) return PW_OK;
  Range range("pw_kv_evict");
  EvictParams P = {};
  P.kv = w;
  P.B = a->batch;
  P.budget = a->budget;
  P.recent = a->recent;
  P.table = a->table;
  P.table_stride = a->table_stride;
  P.lens = a->lens;
  P.mass = a->mass;
  P.mass_stride = a->mass_stride;
  P.new_table = a->new_table;
  P.new_stride = a->new_stride;
  P.new_lens = a->new_lens;
  P.new_mass = a->new_mass;
  P.kept = a->kept;
  char* at = static_cast<char*>(ws);
  P.ws_moves = reinterpret_cast<int2*>(at);
  P.ws_left = reinterpret_cast<int*>(at + up256((size_t)a->batch * a->budget * 8));
  return launched(launch_evict(P, as_stream(stream)));
}
