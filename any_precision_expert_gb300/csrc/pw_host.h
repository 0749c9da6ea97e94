// Checks and handles shared by the host entry points around the layer
// (pw_serve.cpp, pw_context.cpp).
#pragma once

#include <cmath>
#include <new>

#include "pw_serve.h"

struct pw_kv_s {
  pw::KvView view;
  pw::KvMapSet maps;
};

namespace pw {

struct Range {
  explicit Range(const char* name) { range_push(name); }
  ~Range() { range_pop(); }
};

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }
inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }
inline pw_status launched(cudaError_t e) { return e == cudaSuccess ? PW_OK : record_cuda_error(e); }
inline bool bad_tokens(int T) { return T < 0 || T > (1 << 20); }
constexpr long long kMostKeys = 0x7ffff000ll;  // tokens of a table's row: whole tiles of them still count in 32 bits

inline pw_status check_heads(const pw_heads& h) {
  if (h.dtype != PW_F16 && h.dtype != PW_BF16) return PW_ERR_INVALID_ARG;
  if (h.n_heads < 1 || h.n_kv_heads < 1 || h.n_heads > 16384 || h.n_heads % h.n_kv_heads != 0)
    return PW_ERR_INVALID_ARG;
  if (h.n_heads / h.n_kv_heads > kMaxGroup) return PW_ERR_UNSUPPORTED;
  if (h.head_dim != 64 && h.head_dim != 128) return PW_ERR_UNSUPPORTED;
  return PW_OK;
}

// A set of head rows that a call reads or writes: 16-byte aligned rows.
inline bool bad_rows(const pw_rows* r) {
  return !r || !r->ptr || !aligned16(r->ptr) || (r->token_stride & 7) || (r->head_stride & 7);
}

// Reads and clears a handle's error word.
pw_status read_error(int* err, cudaStream_t s);

}  // namespace pw
