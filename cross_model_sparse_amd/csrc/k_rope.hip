// Per-head RMS norm of q and k and rotary positions, in one pass.
//
//   y = x * w / sqrt(mean(x^2) + eps);  (a, b) -> (a cos t - b sin t, b cos t + a sin t) * f,
//   t = position * freq_i for the pairs of the first `rot` dims.
//
// Bound by memory: every row is read once and written once, and there is
// nothing to reuse but the angles, which all heads of a token share.  So a
// workgroup takes one token: its rows' loads are issued first (16 bytes a
// lane, d/8 lanes a row, up to four rows a lane), the token's cos and sin go
// to LDS meanwhile, and the norm's sum is a butterfly over the row's lanes.
// Angles: t / 2pi in fp64, its fraction in fp32 (error 2^-24 turns at any
// position; t itself in fp32 would be off by t * 2^-24), then sincospi.
#include "mf_attn.h"

namespace {

using namespace mfd;

constexpr int kRopeThreads = 256;
constexpr int kRopeRows = 4;   // rows per lane group

template <class TT, bool kVec>
__device__ __forceinline__ void load8(const typename TT::S* p, typename TT::S (&x)[8]) {
  if constexpr (kVec) {
    constexpr int NV = 8 * sizeof(typename TT::S) / 16;
    uint4 v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
    __builtin_memcpy(x, v, sizeof x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = p[i];
  }
}

template <class TT, bool kVec>
__device__ __forceinline__ void store8(typename TT::S* p, const typename TT::S (&x)[8]) {
  if constexpr (kVec) {
    constexpr int NV = 8 * sizeof(typename TT::S) / 16;
    uint4 v[NV];
    __builtin_memcpy(v, x, sizeof x);
#pragma unroll
    for (int i = 0; i < NV; ++i) reinterpret_cast<uint4*>(p)[i] = v[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = x[i];
  }
}

// grid (token, chunk of rows); rows 0..H_q-1 are q heads, then k heads, then
// (cache form) v heads, which are copied bit for bit
template <class TT, int D, bool kVec>
__global__ __launch_bounds__(kRopeThreads) void k_rope(const mf::RopeArgs a) {
  using S = typename TT::S;
  constexpr int LPR = D / 8;                    // lanes per row
  constexpr int RPS = kRopeThreads / LPR;       // rows per step
  __shared__ float cs[D / 2], sn[D / 2];
  __shared__ float rows[kRopeThreads * 8];      // a step's normed rows
  const int n = blockIdx.x;
  const int t = threadIdx.x;
  const int piece = t % LPR;
  const int r0 = blockIdx.y * (RPS * kRopeRows) + t / LPR;
  const int R = a.H_q + a.H_k * (a.slots ? 2 : 1);
  const int half = a.rot / 2;

  S x[kRopeRows][8];
#pragma unroll
  for (int i = 0; i < kRopeRows; ++i) {
    const int r = r0 + i * RPS;
    if (r < R) {
      const S* p = r < a.H_q ? (const S*)a.q + (int64_t)n * a.ldq + r * D
                 : r < a.H_q + a.H_k ? (const S*)a.k + (int64_t)n * a.ldk + (r - a.H_q) * D
                                     : (const S*)a.v + (int64_t)n * a.ldv + (r - a.H_q - a.H_k) * D;
      load8<TT, kVec>(p + 8 * piece, x[i]);
    }
  }
  int64_t slot = -1, pg = 0;
  if (a.slots) {
    slot = a.slots[n];
    if (slot >= 0 && slot < a.n_pages * a.page) pg = slot / a.page; else slot = -1;
  }
  if (t < half) {
    const double rev = (double)a.positions[n] * a.freq[t] * 0.15915494309189533577;   // 1 / 2pi
    const float fr = (float)(rev - rint(rev));
    float s, c;
    sincospif(2.f * fr, &s, &c);
    cs[t] = c * a.attn_factor;
    sn[t] = s * a.attn_factor;
  }
  __syncthreads();

#pragma unroll
  for (int i = 0; i < kRopeRows; ++i) {
    const int r = r0 + i * RPS;
    if (r - t / LPR >= R) break;                // uniform: no row of this step is left
    const bool live = r < R;
    const bool isq = r < a.H_q, isv = r >= a.H_q + a.H_k;
    float y[8];
    const S* w = (const S*)(isq ? a.wq : a.wk);
    if (live && !isv) {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = TT::tof(x[i][j]);
      if (w) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(y[j], y[j], ss);
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) ss += __shfl_xor(ss, o);
        const float inv = 1.f / sqrtf(ss * (1.f / D) + a.eps);
        S wv[8];
        load8<TT, kVec>(w + 8 * piece, wv);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = y[j] * inv * TT::tof(wv[j]);
      }
    }
    // the pairs' other elements: within the lane (interleaved), or from the
    // row's copy in LDS, which only this row's lanes (one wavefront) touch
    float o[8];
    if (a.layout == MF_ROPE_INTERLEAVED) {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = y[j ^ 1];
    } else {
      float* row = rows + (t / LPR) * D;
      if (live && !isv) {
#pragma unroll
        for (int j = 0; j < 8; ++j) row[8 * piece + j] = y[j];
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      if (live && !isv) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = 8 * piece + j;
          o[j] = e < half ? row[e + half] : e < a.rot ? row[e - half] : 0.f;
        }
      }
      __builtin_amdgcn_wave_barrier();          // read before the next step's rows
    }
    if (!live) continue;
    if (!isv) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = 8 * piece + j;
        if (e < a.rot) {
          const bool inter = a.layout == MF_ROPE_INTERLEAVED;
          const int f = inter ? e >> 1 : e < half ? e : e - half;
          const bool first = inter ? !(e & 1) : e < half;
          y[j] = y[j] * cs[f] + (first ? -o[j] : o[j]) * sn[f];
        }
        x[i][j] = TT::fromf(y[j]);
      }
    }
    S* dst;
    if (isq) {
      dst = (S*)a.Q + (int64_t)n * a.ldQ + (int64_t)r * a.hsQ;
    } else if (!a.slots) {
      dst = (S*)a.K + (int64_t)n * a.ldK + (int64_t)(r - a.H_q) * a.hsK;
    } else {
      if (slot < 0) continue;
      const int g = isv ? r - a.H_q - a.H_k : r - a.H_q;
      dst = (S*)(isv ? a.V : a.K) + ((pg * a.H_k + g) * a.page + (slot - pg * a.page)) * D;
    }
    store8<TT, kVec>(dst + 8 * piece, x[i]);
  }
}

bool vec_ok(const void* p, int64_t ld, int es) {
  return (reinterpret_cast<uintptr_t>(p) % 16) == 0 && (ld * es) % 16 == 0;
}

template <class TT, int D>
hipError_t run(const mf::RopeArgs& a, hipStream_t st) {
  constexpr int es = sizeof(typename TT::S);
  const int R = a.H_q + a.H_k * (a.slots ? 2 : 1);
  const int per = kRopeThreads / (D / 8) * kRopeRows;
  const dim3 grid(a.N, (R + per - 1) / per);
  const bool v = vec_ok(a.q, a.ldq, es) && vec_ok(a.k, a.ldk, es) && vec_ok(a.v, a.ldv, es) &&
                 vec_ok(a.wq, 0, es) && vec_ok(a.wk, 0, es) && vec_ok(a.Q, a.ldQ, es) &&
                 vec_ok(a.K, a.ldK, es) && vec_ok(a.V, 0, es) && (a.hsQ * es) % 16 == 0 &&
                 (a.hsK * es) % 16 == 0;
  if (v) k_rope<TT, D, true><<<grid, kRopeThreads, 0, st>>>(a);
  else k_rope<TT, D, false><<<grid, kRopeThreads, 0, st>>>(a);
  return hipGetLastError();
}

template <class TT>
hipError_t run_d(const mf::RopeArgs& a, hipStream_t st) {
  return a.d == 64 ? run<TT, 64>(a, st) : run<TT, 128>(a, st);
}

}  // namespace

namespace mf {

hipError_t launch_rope(int dt, const RopeArgs& a, hipStream_t st) {
  if (dt == MF_F32) return run_d<TF32>(a, st);
  if (dt == MF_F16) return run_d<TF16>(a, st);
  return run_d<TBF16>(a, st);
}

}  // namespace mf
