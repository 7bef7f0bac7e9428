// Declarations shared by the attention operators (k_rope, k_attn, k_decode,
// k_key_mass, k_evict) and their argument checks.
#pragma once

#include "mf_internal.h"

namespace mf {

// element (row n, head h, dim e) at p[n*ld + h*hs + e]
struct Strided {
  const void* p;
  int64_t ld, hs;
};

// one of the pools [n_pages][H_kv][page][d] of a cache and its page table
struct Cache {
  const void* K;
  const void* V;
  int64_t n_pages;
  int page;
  const int32_t* table;  // [S][max_pages] or null (page s*max_pages + i)
  int max_pages;
  const int32_t* lens;
  int max_len;
};

struct RopeArgs {
  int N, d, H_q, H_k;
  const void *q, *k, *v;
  int64_t ldq, ldk, ldv;
  const void *wq, *wk;
  float eps;
  const double* freq;
  int rot, layout;
  float attn_factor;
  const int32_t* positions;
  void *Q, *K, *V;
  int64_t ldQ, hsQ, ldK, hsK;
  const int64_t* slots;  // null: K by strides, no V
  int64_t n_pages;
  int page;
};
hipError_t launch_rope(int dt, const RopeArgs& a, hipStream_t st);

struct AttnArgs {
  Strided Q, K, V;
  void* O;
  int64_t ldO;
  float* lse;
  const float* scale;
  int H, H_kv, N_q, N_k, d, window, sinks;
  int S;                       // packed batch; 0: one sequence
  const int32_t *cu_q, *cu_k;
};
hipError_t launch_attention(int dt, const AttnArgs& a, void* workspace, size_t workspace_bytes,
                            hipStream_t st);
size_t attention_split_bytes(int dt, int H, int H_kv, int N_q, int N_k, int d, int window,
                             int sinks);

struct DecodeArgs {
  const void* Q;
  int64_t ldQ;
  Cache c;
  int S, H, H_kv, d, window, sinks;
  const float* scale;
  void* O;
  int64_t ldO;
  float* lse;
  const float* mass_in;
  float* mass_out;
  int64_t ldmass;
};
hipError_t launch_decode(int dt, const DecodeArgs& a, void* workspace, hipStream_t st);
size_t decode_workspace_bytes(int S, int max_len, int H, int H_kv, int d, int window, int sinks,
                              bool with_mass);

struct KeyMassArgs {
  Strided Q, K;
  const float *scale, *lse;
  int H, H_kv, N_q, N_k, d, window, sinks;
  const float* mass_in;
  float* mass_out;
};
hipError_t launch_key_mass(int dt, const KeyMassArgs& a, void* workspace, hipStream_t st);
size_t key_mass_workspace_bytes(int dt, int H, int H_kv, int N_q, int N_k, int d, int window,
                                int sinks);

struct EvictArgs {
  const float* mass;
  int64_t ldmass;
  Cache c;
  int S, H_kv, d, budget, sinks, recent;
  void *K_out, *V_out;
  int64_t cap_out;
  float* mass_out;
  int32_t *kept, *lens_out;
};
hipError_t launch_evict(int dt, const EvictArgs& a, hipStream_t st);

}  // namespace mf

namespace mfd {

// exp2 argument scale: scores are multiplied by scale * log2(e)
constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLn2f = 0.69314718055994531f;

// Row `j` of KV head g of sequence s in a paged cache, or -1 off the pool:
// the element offset of its first dim.
__device__ __forceinline__ int64_t cache_row(const mf::Cache& c, int s, int j, int g, int H_kv,
                                             int d) {
  const int pi = j / c.page, r = j - pi * c.page;
  const int64_t slot = (int64_t)s * c.max_pages + pi;
  const int64_t pg = c.table ? (int64_t)c.table[slot] : slot;
  if (pg < 0 || pg >= c.n_pages) return -1;
  return ((pg * H_kv + g) * c.page + r) * d;
}

__device__ __forceinline__ int cache_len(const mf::Cache& c, int s) {
  return min(max(c.lens[s], 0), c.max_len);
}

}  // namespace mfd
