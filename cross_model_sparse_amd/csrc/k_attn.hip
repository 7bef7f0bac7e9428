// Causal attention with a sliding window and visible first tokens.
//
//   s_ij = scale_h q_i . k_j;  O_i = sum_j exp(s_ij - lse_i) v_j,
//   lse_i = log sum_j exp(s_ij), over j <= p_i with j > p_i - window or j < sinks.
//
// k_attn_plain: one wavefront per (query, head), 64 keys at a time, one key a
// lane for the scores and two dims a lane for the output, with the running
// maximum and sum of the softmax.  It takes any alignment.
#include "mf_attn.h"

#include <algorithm>

namespace {

using namespace mfd;

// rows of the packed batch's sequence that holds query row `i`
struct SeqRows { int q0, q1, k0, k1; };

__device__ __forceinline__ SeqRows seq_rows(const mf::AttnArgs& a, int s) {
  SeqRows r;
  r.q0 = min(max(a.cu_q[s], 0), a.N_q);
  r.q1 = min(max(a.cu_q[s + 1], r.q0), a.N_q);
  r.k0 = min(max(a.cu_k[s], 0), a.N_k);
  r.k1 = min(max(a.cu_k[s + 1], r.k0), a.N_k);
  return r;
}

template <class TT, int D>
__global__ __launch_bounds__(256) void k_attn_plain(const mf::AttnArgs a) {
  using S = typename TT::S;
  constexpr int ND = D / 64;
  const int lane = threadIdx.x & 63;
  const int i = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int h = blockIdx.y, g = h / (a.H / a.H_kv);
  if (i >= a.N_q) return;
  SeqRows r{0, a.N_q, 0, a.N_k};
  if (a.cu_q) {
    // last sequence that starts at or before row i
    int lo = 0, hi = a.S;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (a.cu_q[mid + 1] <= i) lo = mid + 1; else hi = mid;
    }
    if (lo >= a.S) return;                      // behind the last sequence
    r = seq_rows(a, lo);
    if (i < r.q0 || i >= r.q1) return;
  }
  const int n_k = r.k1 - r.k0;
  const int p = n_k - (r.q1 - r.q0) + (i - r.q0);
  const S* q = (const S*)a.Q.p + (int64_t)i * a.Q.ld + (int64_t)h * a.Q.hs;
  const S* K = (const S*)a.K.p + (int64_t)r.k0 * a.K.ld + (int64_t)g * a.K.hs;
  const S* V = (const S*)a.V.p + (int64_t)r.k0 * a.V.ld + (int64_t)g * a.V.hs;
  const float sc = a.scale[h] * kLog2E;
  const int w0 = a.window > 0 ? max(0, p - a.window + 1) : 0;
  float m = -INFINITY, l = 0.f, acc[ND] = {};
  for (int j0 = 0; j0 <= p; j0 += 64) {
    if (j0 >= a.sinks && j0 + 63 < w0) { j0 = (w0 & ~63) - 64; continue; }
    const int j = j0 + lane;
    const bool vis = j <= p && (j >= w0 || j < a.sinks);
    float x = -INFINITY;
    if (vis) {
      const S* k = K + (int64_t)j * a.K.ld;
      float dot = 0.f;
      for (int e = 0; e < D; ++e) dot = fmaf(TT::tof(q[e]), TT::tof(k[e]), dot);
      x = dot * sc;
    }
    float mx = x;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
    mx = fmaxf(mx, m);
    const bool any_nan = __any(x != x);
    if (mx == -INFINITY && !any_nan) continue;
    const float f = exp2f(m - mx);
    const float e = vis ? exp2f(x - mx) : 0.f;
    float t = e;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) t += __shfl_xor(t, o);
    l = l * f + t;
    m = mx;
#pragma unroll
    for (int c = 0; c < ND; ++c) acc[c] *= f;
    uint64_t seen = __ballot(vis);
    while (seen) {
      const int kk = __ffsll((unsigned long long)seen) - 1;
      seen &= seen - 1;
      const float pk = __shfl(e, kk);
      const S* v = V + (int64_t)(j0 + kk) * a.V.ld;
#pragma unroll
      for (int c = 0; c < ND; ++c) acc[c] = fmaf(pk, TT::tof(v[lane + 64 * c]), acc[c]);
    }
  }
  const bool empty = l == 0.f;
  S* o = (S*)a.O + (int64_t)i * a.ldO + (int64_t)h * D;
#pragma unroll
  for (int c = 0; c < ND; ++c) o[lane + 64 * c] = TT::fromf(empty ? 0.f : acc[c] / l);
  if (a.lse && lane == 0)
    a.lse[(int64_t)h * a.N_q + i] = empty ? -INFINITY : (m + log2f(l)) * kLn2f;
}

template <class TT>
hipError_t run_plain(const mf::AttnArgs& a, hipStream_t st) {
  const dim3 grid((a.N_q + 3) / 4, a.H);
  if (a.d == 64) k_attn_plain<TT, 64><<<grid, 256, 0, st>>>(a);
  else k_attn_plain<TT, 128><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

namespace mf {

size_t attention_split_bytes(int, int, int, int, int, int, int, int) { return 0; }

hipError_t launch_attention(int dt, const AttnArgs& a, void*, size_t, hipStream_t st) {
  if (dt == MF_F32) return run_plain<TF32>(a, st);
  if (dt == MF_F16) return run_plain<TF16>(a, st);
  return run_plain<TBF16>(a, st);
}

}  // namespace mf
