// Host entry points around the layer: argument checks of the head norm and
// rotation, the paged KV cache, its attention and draft verification.
#include "pw_serve.h"

#include <cmath>
#include <new>

using namespace pw;

struct pw_kv_s {
  KvView view;
  KvMapSet maps;
};

namespace {

struct Range {
  explicit Range(const char* name) { range_push(name); }
  ~Range() { range_pop(); }
};

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }
inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }
inline pw_status launched(cudaError_t e) { return e == cudaSuccess ? PW_OK : record_cuda_error(e); }
inline bool bad_tokens(int T) { return T < 0 || T > (1 << 20); }

pw_status check_heads(const pw_heads& h) {
  if (h.dtype != PW_F16 && h.dtype != PW_BF16) return PW_ERR_INVALID_ARG;
  if (h.n_heads < 1 || h.n_kv_heads < 1 || h.n_heads > 16384 || h.n_heads % h.n_kv_heads != 0)
    return PW_ERR_INVALID_ARG;
  if (h.n_heads / h.n_kv_heads > kMaxGroup) return PW_ERR_UNSUPPORTED;
  if (h.head_dim != 64 && h.head_dim != 128) return PW_ERR_UNSUPPORTED;
  return PW_OK;
}

// A set of head rows that a call reads or writes: 16-byte aligned rows.
bool bad_rows(const pw_rows* r) {
  return !r || !r->ptr || !aligned16(r->ptr) || (r->token_stride & 7) || (r->head_stride & 7);
}

pw_status check_rotary(const pw_rotary& r, int d) {
  if (r.rot_dim < 0 || r.rot_dim > d || (r.rot_dim & 15)) return PW_ERR_INVALID_ARG;
  if (r.rot_dim > 0 && (!r.cos_sin || !aligned16(r.cos_sin) || r.max_pos < 1)) return PW_ERR_INVALID_ARG;
  if (r.interleaved != 0 && r.interleaved != 1) return PW_ERR_INVALID_ARG;
  if (!aligned16(r.q_weight) || !aligned16(r.k_weight)) return PW_ERR_INVALID_ARG;
  if (!(r.eps >= 0.f) || !std::isfinite(r.eps)) return PW_ERR_INVALID_ARG;
  return PW_OK;
}

void set_rotary(RopeParams& P, const pw_rotary* r, const int32_t* positions) {
  if (!r) return;
  P.cos_sin = r->cos_sin;
  P.positions = positions;
  P.qw = r->q_weight;
  P.kw = r->k_weight;
  P.eps = r->eps;
  P.max_pos = r->max_pos;
  P.rot = r->rot_dim;
  P.interleaved = r->interleaved;
}

}  // namespace

extern "C" pw_status pw_qk_norm_rope(const pw_heads* heads, const pw_rotary* rot, const int32_t* positions, int T,
                                     const pw_rows* q, const pw_rows* k, const pw_rows* q_out, const pw_rows* k_out,
                                     int32_t* err, void* stream) {
  if (!heads || !rot || bad_tokens(T)) return PW_ERR_INVALID_ARG;
  pw_status st = check_heads(*heads);
  if (st != PW_OK) return st;
  if ((st = check_rotary(*rot, heads->head_dim)) != PW_OK) return st;
  const bool hasq = q && q->ptr, hask = k && k->ptr;
  if (!aligned4(err) || (!hasq && !hask && T > 0)) return PW_ERR_INVALID_ARG;
  if (T > 0) {
    if (rot->rot_dim > 0 && (!positions || !aligned4(positions))) return PW_ERR_INVALID_ARG;
    if (hasq && (bad_rows(q) || bad_rows(q_out))) return PW_ERR_INVALID_ARG;
    if (hask && (bad_rows(k) || bad_rows(k_out))) return PW_ERR_INVALID_ARG;
  }
  if (host_sim()) return PW_ERR_UNSUPPORTED;
  if (T == 0) return PW_OK;
  Range range("pw_qk_norm_rope");
  RopeParams P = {};
  set_rotary(P, rot, positions);
  P.T = T;
  P.hq = hasq ? heads->n_heads : 0;
  P.hk = hask ? heads->n_kv_heads : 0;
  if (hasq) P.q = *q, P.q_out = *q_out;
  if (hask) P.k = *k, P.k_out = *k_out;
  P.err = err;
  return launched(launch_rope(P, heads->dtype, heads->head_dim, as_stream(stream)));
}

extern "C" pw_status pw_kv_create(const pw_kv_desc* desc, void* k, void* v, int32_t* err, pw_kv_t* out) {
  if (!desc || !k || !v || !err || !out) return PW_ERR_INVALID_ARG;
  pw_status st = check_heads(desc->heads);
  if (st != PW_OK) return st;
  const int pt = desc->page_tokens;
  if (pt < 8 || pt > 1024 || (pt & (pt - 1)) || desc->n_pages < 1 ||
      (long long)desc->n_pages * pt > 0x7fffffffll)
    return PW_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned4(err)) return PW_ERR_INVALID_ARG;
  const long long d = desc->heads.head_dim, lim = 1ll << 38;  // strides below 2^39 bytes
  for (long long s : {desc->page_stride, desc->head_stride, desc->token_stride})
    if (s < d || (s & 7) || s >= lim) return PW_ERR_INVALID_ARG;
  KvView w = {};
  w.k = static_cast<char*>(k);
  w.v = static_cast<char*>(v);
  w.err = err;
  w.dtype = desc->heads.dtype;
  w.hq = desc->heads.n_heads;
  w.hkv = desc->heads.n_kv_heads;
  w.d = desc->heads.head_dim;
  while ((1 << w.page_shift) < pt) ++w.page_shift;
  w.n_pages = desc->n_pages;
  w.page_stride = desc->page_stride;
  w.head_stride = desc->head_stride;
  w.token_stride = desc->token_stride;
  KvMapSet maps = {};
  if (!host_sim()) {
    const cudaError_t e = encode_kv_maps(w, &maps);
    if (e != cudaSuccess) return record_cuda_error(e);
  }
  auto* kv = new (std::nothrow) pw_kv_s{w, maps};
  if (!kv) return PW_ERR_OOM;
  *out = kv;
  return PW_OK;
}

extern "C" pw_status pw_kv_destroy(pw_kv_t kv) {
  if (!kv) return PW_ERR_INVALID_ARG;
  delete kv;
  return PW_OK;
}

extern "C" pw_status pw_kv_check_device(pw_kv_t kv, void* stream) {
  if (!kv) return PW_ERR_INVALID_ARG;
  if (host_sim()) return PW_ERR_UNSUPPORTED;
  int err = 0;
  cudaStream_t s = as_stream(stream);
  cudaError_t e = cudaMemcpyAsync(&err, kv->view.err, sizeof(int), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && err != 0) {
    e = cudaMemsetAsync(kv->view.err, 0, sizeof(int), s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  if (e != cudaSuccess) return record_cuda_error(e);
  return err == 0 ? PW_OK : err == kErrTimeout ? PW_ERR_TIMEOUT : PW_ERR_DEVICE_CHECK;
}

extern "C" pw_status pw_kv_append(pw_kv_t kv, const pw_rotary* rot, const int32_t* positions, const int32_t* slots,
                                  int T, const pw_rows* k, const pw_rows* v, const pw_rows* q, const pw_rows* q_out,
                                  void* stream) {
  if (!kv || bad_tokens(T)) return PW_ERR_INVALID_ARG;
  const KvView& w = kv->view;
  if (rot) {
    const pw_status st = check_rotary(*rot, w.d);
    if (st != PW_OK) return st;
  }
  const bool hasq = q && q->ptr;
  if (T > 0) {
    if (!slots || !aligned4(slots) || bad_rows(k) || bad_rows(v)) return PW_ERR_INVALID_ARG;
    if (rot && rot->rot_dim > 0 && (!positions || !aligned4(positions))) return PW_ERR_INVALID_ARG;
    if (hasq && (bad_rows(q) || bad_rows(q_out))) return PW_ERR_INVALID_ARG;
    if (!hasq && q_out && q_out->ptr) return PW_ERR_INVALID_ARG;
  }
  if (host_sim()) return PW_ERR_UNSUPPORTED;
  if (T == 0) return PW_OK;
  Range range("pw_kv_append");
  RopeParams P = {};
  set_rotary(P, rot, positions);
  P.T = T;
  P.hq = hasq ? w.hq : 0;
  P.hk = P.hv = w.hkv;
  if (hasq) P.q = *q, P.q_out = *q_out;
  P.k = *k;
  P.v = *v;
  P.err = w.err;
  P.slots = slots;
  P.kv = w;
  return launched(launch_rope(P, w.dtype, w.d, as_stream(stream)));
}

extern "C" pw_status pw_kv_attend_workspace_size(pw_kv_t kv, int batch, int q_len, int n_groups, size_t* bytes) {
  if (!kv || !bytes || batch < 0 || q_len < 1 || q_len > kMaxQLen || n_groups < 0) return PW_ERR_INVALID_ARG;
  if (batch > kMaxBatch || n_groups > kMaxBatch) return PW_ERR_UNSUPPORTED;
  *bytes = attend_ws_bytes(kv->view, batch, q_len, n_groups);
  return PW_OK;
}

extern "C" pw_status pw_kv_attend(pw_kv_t kv, const pw_attend_desc* a, void* ws, size_t ws_bytes, void* stream) {
  if (!kv || !a) return PW_ERR_INVALID_ARG;
  const KvView& w = kv->view;
  size_t need = 0;
  const pw_status st = pw_kv_attend_workspace_size(kv, a->batch, a->q_len, a->n_groups, &need);
  if (st != PW_OK) return st;
  if (!std::isfinite(a->scale) || a->table_stride < 0 || a->prefix_stride < 0) return PW_ERR_INVALID_ARG;
  constexpr long long kMostKeys = 0x7ffff000ll;  // whole tiles of them still count in 32 bits
  if (((long long)a->table_stride << w.page_shift) > kMostKeys || ((long long)a->prefix_stride << w.page_shift) > kMostKeys)
    return PW_ERR_INVALID_ARG;
  if (a->batch > 0) {
    if (bad_rows(&a->q) || bad_rows(&a->out) || !aligned4(a->lse)) return PW_ERR_INVALID_ARG;
    if (!a->lens || !aligned4(a->lens) || !aligned4(a->table) || (a->table_stride > 0 && !a->table))
      return PW_ERR_INVALID_ARG;
    if (a->n_groups > 0) {
      if (!a->prefix_lens || !aligned4(a->prefix_lens) || !aligned4(a->prefix_table) ||
          (a->prefix_stride > 0 && !a->prefix_table))
        return PW_ERR_INVALID_ARG;
      if (!aligned4(a->group_offsets) || (a->n_groups > 1 && !a->group_offsets)) return PW_ERR_INVALID_ARG;
    }
    if (need > 0 && (!ws || (reinterpret_cast<uintptr_t>(ws) & 255))) return PW_ERR_INVALID_ARG;
    if (ws_bytes < need) return PW_ERR_OOM;
  }
  // the kernels count key tiles in 32 bits
  const double tiles = ((double)a->batch * ((double)((long long)a->table_stride << w.page_shift) / 64 + 3) *
                            ((double)a->q_len * (w.hq / w.hkv) / 16 + 1) +
                        ((double)a->n_groups + (double)a->batch * a->q_len * (w.hq / w.hkv) / 16) *
                            ((double)((long long)a->prefix_stride << w.page_shift) / 64 + 3)) *
                       w.hkv;
  if (tiles > 2e9) return PW_ERR_UNSUPPORTED;
  if (host_sim()) return PW_ERR_UNSUPPORTED;
  if (a->batch == 0) return PW_OK;
  Range range("pw_kv_attend");
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
  P.n_groups = a->n_groups;
  P.group_offsets = a->group_offsets;
  P.prefix_table = a->prefix_table;
  P.prefix_stride = a->prefix_stride;
  P.prefix_lens = a->prefix_lens;
  return launched(launch_attend(P, kv->maps, ws, as_stream(stream)));
}

extern "C" pw_status pw_verify_draft(const float* target_p, const float* draft_p, const int32_t* tokens,
                                     const int32_t* n_draft, const float* u, const float* noise, int B, int K, int V,
                                     int32_t* out, int32_t* accepted, int32_t* err, void* stream) {
  if (B < 0 || B > 65535 || K < 0 || K > kMaxDrafts || V < 1 || V > (1 << 24)) return PW_ERR_INVALID_ARG;
  if (!aligned4(err)) return PW_ERR_INVALID_ARG;
  if (B > 0) {
    for (const void* p : {(const void*)target_p, (const void*)noise, (const void*)out, (const void*)accepted})
      if (!p || !aligned4(p)) return PW_ERR_INVALID_ARG;
    if (K > 0)
      for (const void* p : {(const void*)draft_p, (const void*)tokens, (const void*)n_draft, (const void*)u})
        if (!p || !aligned4(p)) return PW_ERR_INVALID_ARG;
  }
  if (host_sim()) return PW_ERR_UNSUPPORTED;
  if (B == 0) return PW_OK;
  Range range("pw_verify_draft");
  const VerifyParams P = {target_p, draft_p, tokens, n_draft, u, noise, B, K, V, out, accepted, err};
  return launched(launch_verify(P, as_stream(stream)));
}
