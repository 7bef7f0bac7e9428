// Accumulated attention weight of every key of a prompt:
//   mass[g][j] = mass_in[g][j] + sum_{h of g} sum_i exp(s_h[i][j] - lse[h][i]).
#include "mf_attn.h"

#include <algorithm>

namespace {

using namespace mfd;

// one thread per (KV head, key)
template <class TT, int D>
__global__ __launch_bounds__(64) void k_key_mass_plain(const mf::KeyMassArgs a) {
  using S = typename TT::S;
  const int g = blockIdx.y, G = a.H / a.H_kv;
  const int j = blockIdx.x * 64 + threadIdx.x;
  if (j >= a.N_k) return;
  const int off = a.N_k - a.N_q;                // position of query 0
  const S* kp = (const S*)a.K.p + (int64_t)j * a.K.ld + (int64_t)g * a.K.hs;
  float k[D];
#pragma unroll
  for (int e = 0; e < D; ++e) k[e] = TT::tof(kp[e]);
  int i1 = a.N_q;
  if (a.window > 0 && j >= a.sinks)
    i1 = (int)min((int64_t)a.N_q, max((int64_t)0, (int64_t)j + a.window - off));
  double sum = a.mass_in ? a.mass_in[(int64_t)g * a.N_k + j] : 0.f;
  for (int h = g * G; h < (g + 1) * G; ++h) {
    const float sc = a.scale[h] * kLog2E;
    for (int i = max(0, j - off); i < i1; ++i) {
      const float L = a.lse[(int64_t)h * a.N_q + i];
      if (L == -INFINITY) continue;
      const S* q = (const S*)a.Q.p + (int64_t)i * a.Q.ld + (int64_t)h * a.Q.hs;
      float dot = 0.f;
#pragma unroll
      for (int e = 0; e < D; ++e) dot = fmaf(TT::tof(q[e]), k[e], dot);
      sum += exp2f(dot * sc - L * kLog2E);
    }
  }
  a.mass_out[(int64_t)g * a.N_k + j] = (float)sum;
}

template <class TT>
hipError_t run(const mf::KeyMassArgs& a, hipStream_t st) {
  const dim3 grid((a.N_k + 63) / 64, a.H_kv);
  if (a.d == 64) k_key_mass_plain<TT, 64><<<grid, 64, 0, st>>>(a);
  else k_key_mass_plain<TT, 128><<<grid, 64, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

namespace mf {

size_t key_mass_workspace_bytes(int, int, int, int, int, int, int, int) { return 0; }

hipError_t launch_key_mass(int dt, const KeyMassArgs& a, void*, hipStream_t st) {
  if (dt == MF_F32) return run<TF32>(a, st);
  if (dt == MF_F16) return run<TF16>(a, st);
  return run<TBF16>(a, st);
}

}  // namespace mf
