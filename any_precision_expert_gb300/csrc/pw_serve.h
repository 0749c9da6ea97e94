// Declarations shared by the host entry points around the layer (pw_serve.cpp)
// and their kernels: heads, the paged KV cache, attention, draft verification.
#pragma once

#include <cuda.h>

#include "pw_internal.h"

namespace pw {

constexpr int kMaxGroup = 128;       // query heads per key head
constexpr int kMaxBatch = 4096;      // sequences, and prefix groups, of one attention call
constexpr int kMaxQLen = 64;         // query tokens a sequence
constexpr int kMaxDrafts = 64;       // drafted tokens a sequence

// The paged cache as the kernels see it (strides in elements).
struct KvView {
  char* k;
  char* v;
  int* err;
  int dtype, hq, hkv, d;
  int page_shift;       // log2 of the tokens a page holds
  int n_pages;
  long long page_stride, head_stride, token_stride;
};

struct RopeParams {
  const float* cos_sin;
  const int* positions;
  const void* qw;
  const void* kw;
  float eps;
  int max_pos, rot, interleaved;
  int T, hq, hk, hv;             // rows a token: queries, then keys, then values (0 = that side is left out)
  pw_rows q, k, v, q_out, k_out;
  int* err;
  const int* slots;              // non-null: keys and values go to the cache
  KvView kv;
};

struct AttendParams {
  KvView kv;
  pw_rows q, out;
  float* lse;
  int B, ql, G;                  // G query heads per key head
  float scale;
  const int* table;
  int table_stride;
  const int* lens;
  int n_groups;
  const int* group_offsets;
  const int* prefix_table;
  int prefix_stride;
  const int* prefix_lens;
};

struct VerifyParams {
  const float* p;
  const float* q;
  const int* tokens;
  const int* n_draft;
  const float* u;
  const float* noise;
  int B, K, V;
  int* out;
  int* accepted;
  int* err;
};

// The cache held in 4 bits (contiguous: [page][key head][token][...]).
struct Kv4View {
  char *k, *v;          // codes, head_dim / 2 bytes a row
  char *ks, *vs;        // least value and step of every 32 values, head_dim / 8 bytes a row
  int* err;
  int dtype, hq, hkv, d;
  int page_shift, n_pages;
};

struct Row4Params {
  Kv4View kv;
  pw_rows k, v;         // read by an append, written by a load
  const int* slots;
  int T;
};

struct WeighParams {
  KvView kv;
  pw_rows q;
  const float* lse;
  int B, ql, G;
  float scale, decay;
  const int* table;
  int table_stride;
  const int* lens;
  const float* mass;
  float* out;
  int mass_stride;
};

struct EvictParams {
  KvView kv;
  int B, budget, recent;
  const int* table;
  int table_stride;
  const int* lens;
  const float* mass;
  int mass_stride;
  const int* new_table;
  int new_stride;
  int* new_lens;
  float* new_mass;
  int* kept;
  int2* ws_moves;       // [B][budget] slots of the tokens that stay, old and new (-1: none, or there already)
  int* ws_left;         // [B]
};

struct PromptParams {
  pw_rows q, k, v, out;
  float* lse;
  const int* offsets;
  int* err;
  int T, B, hq, hkv, G;
  float scale;
};

constexpr int kMaxTop = 32;          // alternatives a token

struct LogprobParams {
  const void* logits;
  long long row_stride;
  int T, V, n_top;
  const int* tokens;
  float* logprob;
  float* entropy;
  int* top_ids;
  float* top_logprobs;
  int* err;
};

// These kernels start while the one before them in the stream still ends (programmatic dependent launch), which takes the
// launch itself off a decode step's path (one token's norm and rotation 4.1 -> 2.3 us a call).  Each waits for the
// completion of what came before (behind_the_stream) before it reads or writes global memory, so the order of the stream
// holds as ever; a kernel that does not take part neither starts early nor lets the next one.
struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  Launch(dim3 grid, unsigned block, size_t smem, cudaStream_t s, int cluster = 0) {
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
  }
  Launch(const Launch&) = delete;  // cfg points into it
};
#ifdef __CUDACC__
__device__ __forceinline__ void behind_the_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
#endif

cudaError_t launch_rope(const RopeParams& P, int dtype, int d, cudaStream_t s);
size_t attend_ws_bytes(const KvView& kv, int B, int ql, int n_groups);
// Tensor maps of a cache's keys and values: (value, token of a page, head, page).
struct KvMaps {
  CUtensorMap k, v;
};
// Boxes of 64 values x up to 64 / heads tokens x 1, 2 or 4 heads (the latter where they divide the key heads).
struct KvMapSet {
  KvMaps heads1, heads2, heads4;
};
constexpr int kBoxTokens = 64;
cudaError_t encode_kv_maps(const KvView& kv, KvMapSet* maps);
cudaError_t launch_attend(const AttendParams& P, const KvMapSet& maps, void* ws, cudaStream_t s);
cudaError_t launch_verify(const VerifyParams& P, cudaStream_t s);
cudaError_t launch_weigh(const WeighParams& P, cudaStream_t s);
cudaError_t launch_evict(const EvictParams& P, cudaStream_t s);
cudaError_t launch_prompt(const PromptParams& P, int dtype, int d, cudaStream_t s);
cudaError_t prompt_error_word(int** word);  // the current device's, of calls that bring none
cudaError_t launch_logprobs(const LogprobParams& P, int dtype, cudaStream_t s);
cudaError_t launch_rows4(const Row4Params& P, bool load, cudaStream_t s);
size_t attend4_ws_bytes(const KvView& kv, int B, int ql);
cudaError_t launch_attend4(const AttendParams& P, const Kv4View& kv, void* ws, cudaStream_t s);

}  // namespace pw
