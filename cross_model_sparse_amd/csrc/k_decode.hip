// Attention of one query per sequence over a paged cache, optionally with the
// accumulated weight of every cached row.
#include "mf_attn.h"

#include <algorithm>

namespace {

using namespace mfd;

// one wavefront per (sequence, head)
template <class TT, int D>
__global__ __launch_bounds__(64) void k_decode_plain(const mf::DecodeArgs a, float* lse2) {
  using S = typename TT::S;
  constexpr int ND = D / 64;
  const int lane = threadIdx.x;
  const int s = blockIdx.x, h = blockIdx.y, g = h / (a.H / a.H_kv);
  const int n = cache_len(a.c, s);
  const S* q = (const S*)a.Q + (int64_t)s * a.ldQ + (int64_t)h * D;
  const float sc = a.scale[h] * kLog2E;
  const int w0 = a.window > 0 ? max(0, n - a.window) : 0;
  float m = -INFINITY, l = 0.f, acc[ND] = {};
  for (int j0 = 0; j0 < n; j0 += 64) {
    if (j0 >= a.sinks && j0 + 63 < w0) { j0 = (w0 & ~63) - 64; continue; }
    const int j = j0 + lane;
    int64_t row = -1;
    if (j < n && (j >= w0 || j < a.sinks)) row = cache_row(a.c, s, j, g, a.H_kv, D);
    float x = -INFINITY;
    if (row >= 0) {
      const S* k = (const S*)a.c.K + row;
      float dot = 0.f;
      for (int e = 0; e < D; ++e) dot = fmaf(TT::tof(q[e]), TT::tof(k[e]), dot);
      x = dot * sc;
    }
    float mx = x;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
    mx = fmaxf(mx, m);
    if (mx == -INFINITY && !__any(x != x)) continue;
    const float f = exp2f(m - mx);
    const float e = row >= 0 ? exp2f(x - mx) : 0.f;
    float t = e;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) t += __shfl_xor(t, o);
    l = l * f + t;
    m = mx;
#pragma unroll
    for (int c = 0; c < ND; ++c) acc[c] *= f;
    uint64_t seen = __ballot(row >= 0);
    while (seen) {
      const int kk = __ffsll((unsigned long long)seen) - 1;
      seen &= seen - 1;
      const float pk = __shfl(e, kk);
      const S* v = (const S*)a.c.V + __shfl(row, kk);
#pragma unroll
      for (int c = 0; c < ND; ++c) acc[c] = fmaf(pk, TT::tof(v[lane + 64 * c]), acc[c]);
    }
  }
  const bool empty = l == 0.f;
  S* o = (S*)a.O + (int64_t)s * a.ldO + (int64_t)h * D;
#pragma unroll
  for (int c = 0; c < ND; ++c) o[lane + 64 * c] = TT::fromf(empty ? 0.f : acc[c] / l);
  const float L = empty ? -INFINITY : m + log2f(l);
  if (lane == 0) {
    if (a.lse) a.lse[(int64_t)s * a.H + h] = L * kLn2f;
    if (lse2) lse2[(int64_t)s * a.H + h] = L;
  }
}

// one thread per (sequence, KV head, row)
template <class TT, int D>
__global__ __launch_bounds__(256) void k_decode_mass_plain(const mf::DecodeArgs a,
                                                           const float* lse2) {
  using S = typename TT::S;
  const int s = blockIdx.y, g = blockIdx.z, G = a.H / a.H_kv;
  const int n = cache_len(a.c, s);
  const int j = blockIdx.x * 256 + threadIdx.x;
  if (j >= n) return;
  const int64_t at = ((int64_t)s * a.H_kv + g) * a.ldmass + j;
  float w = a.mass_in ? a.mass_in[at] : 0.f;
  const bool vis = a.window == 0 || j >= n - a.window || j < a.sinks;
  const int64_t row = vis ? cache_row(a.c, s, j, g, a.H_kv, D) : -1;
  if (row >= 0) {
    const S* k = (const S*)a.c.K + row;
    float sum = 0.f;
    for (int h = g * G; h < (g + 1) * G; ++h) {
      const float L = lse2[(int64_t)s * a.H + h];
      if (L == -INFINITY) continue;
      const S* q = (const S*)a.Q + (int64_t)s * a.ldQ + (int64_t)h * D;
      float dot = 0.f;
      for (int e = 0; e < D; ++e) dot = fmaf(TT::tof(q[e]), TT::tof(k[e]), dot);
      sum += exp2f(dot * (a.scale[h] * kLog2E) - L);
    }
    w += sum;
  }
  a.mass_out[at] = w;
}

template <class TT, int D>
hipError_t run(const mf::DecodeArgs& a, void* ws, hipStream_t st) {
  k_decode_plain<TT, D><<<dim3(a.S, a.H), 64, 0, st>>>(a, (float*)ws);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.mass_out || a.c.max_len == 0) return e;
  k_decode_mass_plain<TT, D><<<dim3((a.c.max_len + 255) / 256, a.S, a.H_kv), 256, 0, st>>>(
      a, (const float*)ws);
  return hipGetLastError();
}

template <class TT>
hipError_t run_d(const mf::DecodeArgs& a, void* ws, hipStream_t st) {
  return a.d == 64 ? run<TT, 64>(a, ws, st) : run<TT, 128>(a, ws, st);
}

}  // namespace

namespace mf {

size_t decode_workspace_bytes(int S, int, int H, int, int, int, int, bool) {
  return (size_t)S * H * 4;
}

hipError_t launch_decode(int dt, const DecodeArgs& a, void* ws, hipStream_t st) {
  if (dt == MF_F32) return run_d<TF32>(a, ws, st);
  if (dt == MF_F16) return run_d<TF16>(a, ws, st);
  return run_d<TBF16>(a, ws, st);
}

}  // namespace mf
