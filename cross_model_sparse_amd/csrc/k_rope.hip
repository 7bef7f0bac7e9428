// Per-head RMS norm of q and k and rotary positions, in one pass.
//
//   y = x * w / sqrt(mean(x^2) + eps);  (a, b) -> (a cos t - b sin t, b cos t + a sin t) * f,
//   t = position * freq_i for the pairs of the first `rot` dims.
//
// Bound by memory: every row is read once and written once, and there is
// nothing to reuse but the angles, which a token's heads share.  A workgroup
// takes four tokens and 16 rows (d = 128) of each: a lane group of d/8 lanes
// loads its row of all four tokens first (16 bytes a lane), each thread forms
// one of the four tokens' angles meanwhile, and the norm's sum is a butterfly
// over the row's lanes.  Four tokens, because Q and K are written head by head:
// a workgroup then writes runs of 1 KB.  Measured: 8192 tokens, 48 heads of 128,
// bf16, 40.5 us (5.0 TB/s; a copy of the same size takes 39 us); 4 tokens 5.5 us.
// Angles: t / 2pi in fp64, its fraction in fp32 (error 2^-24 turns at any
// position; t itself in fp32 would be off by t * 2^-24), then sincospi.
#include "mf_attn.h"

#include <type_traits>

namespace {

using namespace mfd;

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 4;   // tokens of a workgroup

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

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

// eight values rounded to nearest even by the conversion instructions
template <class TT>
__device__ __forceinline__ void round8(const float (&y)[8], typename TT::S (&x)[8]) {
  f32x8 v;
  __builtin_memcpy(&v, y, sizeof y);
  if constexpr (std::is_same<TT, TBF16>::value) {
    const bf16x8 w = __builtin_convertvector(v, bf16x8);
    __builtin_memcpy(x, &w, sizeof x);
  } else if constexpr (std::is_same<TT, TF16>::value) {
    const f16x8 w = __builtin_convertvector(v, f16x8);
    __builtin_memcpy(x, &w, sizeof x);
  } else {
    __builtin_memcpy(x, y, sizeof x);
  }
}

// Place of element e of n in LDS: a lane's eight consecutive elements lie as two
// groups of four, n / 2 apart, so that neighbouring lanes' 16-byte accesses are
// contiguous (eight in a row would be 32 bytes apart: conflicts took 60% of the time).
__device__ __forceinline__ constexpr int place(int e, int n) {
  return ((e >> 2) & 1) * (n / 2) + (e >> 3) * 4 + (e & 3);
}

// grid (token block, chunk of rows): a lane group takes one row of kRopeTokens
// tokens in turn.  Rows 0..H_q-1 are q heads, then k heads, then (cache form) v
// heads, which are copied bit for bit.
// kPieces: a lane's eight dims are rotated by one run of angles and against one
// run of dims (rot a multiple of 16, interleaved of 8), so that everything is
// read in 16-byte pieces; without it every dim looks its own up.
template <class TT, int D, bool kVec, bool kPieces>
__global__ __launch_bounds__(kRopeThreads) void k_rope(const mf::RopeArgs a) {
  using S = typename TT::S;
  constexpr int LPR = D / 8;                    // lanes per row
  constexpr int RPS = kRopeThreads / LPR;       // rows of a workgroup
  __shared__ __align__(16) float cs[kRopeTokens][D / 2], sn[2][kRopeTokens][D / 2];   // sin, -sin
  __shared__ __align__(16) float rows[kRopeThreads * 8];   // a token's normed rows
  const int n0 = blockIdx.x * kRopeTokens;
  const int t = threadIdx.x;
  const int piece = t % LPR;
  const int r = blockIdx.y * RPS + t / LPR;
  const int R = a.H_q + a.H_k * (a.slots ? 2 : 1);
  const int half = a.rot / 2;
  const bool inter = a.layout == MF_ROPE_INTERLEAVED;
  const bool live = r < R, isq = r < a.H_q, isv = r >= a.H_q + a.H_k;
  const int nt = min(kRopeTokens, a.N - n0);

  const int64_t ld = isq ? a.ldq : isv ? a.ldv : a.ldk;
  const int hr = isq ? r : isv ? r - a.H_q - a.H_k : r - a.H_q;   // head of its kind
  const S* src = (const S*)(isq ? a.q : isv ? a.v : a.k) + (int64_t)n0 * ld + hr * D + 8 * piece;
  S x[kRopeTokens][8], wv[8];
  const S* w = isv ? nullptr : (const S*)(isq ? a.wq : a.wk);
  if (live) {
#pragma unroll
    for (int i = 0; i < kRopeTokens; ++i)
      if (i < nt) load8<TT, kVec>(src + i * ld, x[i]);
    if (w) load8<TT, kVec>(w + 8 * piece, wv);
  }
  int64_t slot[kRopeTokens];
  if (a.slots) {
#pragma unroll
    for (int i = 0; i < kRopeTokens; ++i) slot[i] = i < nt ? a.slots[n0 + i] : -1;
  }
  {
    const int i = t / (D / 2), f = t % (D / 2);
    static_assert(kRopeTokens * (D / 2) <= kRopeThreads, "an angle a thread");
    if (i < nt && f < half) {
      const double rev = (double)a.positions[n0 + i] * a.freq[f] * 0.15915494309189533577;   // 1 / 2pi
      const float fr = (float)(rev - rint(rev));
      float s, c;
      if constexpr (sizeof(S) == 2) {           // hardware, in turns: off by at most 1.3e-7 (measured over a turn)
        s = __builtin_amdgcn_sinf(fr);
        c = __builtin_amdgcn_cosf(fr);
      } else {
        sincospif(2.f * fr, &s, &c);
      }
      cs[i][place(f, D / 2)] = c * a.attn_factor;
      sn[0][i][place(f, D / 2)] = s * a.attn_factor;
      sn[1][i][place(f, D / 2)] = -s * a.attn_factor;
    }
  }
  __syncthreads();

  float wf[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) wf[j] = live && w ? TT::tof(wv[j]) : 1.f;
  float* row = rows + (t / LPR) * D;
#pragma unroll
  for (int i = 0; i < kRopeTokens; ++i) {
    if (i >= nt) break;
    float y[8];
    if (live && !isv) {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = TT::tof(x[i][j]);
      if (w) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(y[j], y[j], ss);
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) ss += __shfl_xor(ss, o);
        const float inv = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = y[j] * inv * wf[j];
      }
    }
    // the pairs' other elements: within the lane (interleaved), or from the
    // row's copy in LDS, which only this row's lanes (one wavefront) touch
    if (!inter) {
      if (live && !isv) {
#pragma unroll
        for (int j = 0; j < 8; ++j) row[place(j, D) + 4 * piece] = y[j];
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
    if (live && !isv && 8 * piece < a.rot) {
      if constexpr (kPieces) {
        if (inter) {
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const int f = place(4 * piece, D / 2) + j / 2;
            const float c = cs[i][f], s = sn[0][i][f];
            const float y0 = y[j], y1 = y[j + 1];
            y[j] = y0 * c - y1 * s;
            y[j + 1] = y1 * c + y0 * s;
          }
        } else {
          const bool first = 8 * piece < half;
          const int f = (first ? 8 * piece : 8 * piece - half) / 2;
          const float* o = row + 4 * piece + (first ? half / 2 : -half / 2);
          const float* sg = &sn[first][i][f];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            y[j] = y[j] * cs[i][f + place(j, D / 2)] + o[place(j, D)] * sg[place(j, D / 2)];
        }
      } else {
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = y[j ^ 1];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = 8 * piece + j;
          if (e >= a.rot) continue;
          const int f = inter ? e >> 1 : e < half ? e : e - half;
          const bool first = inter ? !(e & 1) : e < half;
          const float other = inter ? o[j] : row[place(first ? e + half : e - half, D)];
          y[j] = y[j] * cs[i][place(f, D / 2)] + other * sn[first][i][place(f, D / 2)];
        }
      }
    }
    if (!inter) __builtin_amdgcn_wave_barrier();   // read before the next token's row
    if (!live) continue;
    if (!isv) round8<TT>(y, x[i]);
    S* dst;
    if (isq) {
      dst = (S*)a.Q + (int64_t)(n0 + i) * a.ldQ + (int64_t)hr * a.hsQ;
    } else if (!a.slots) {
      dst = (S*)a.K + (int64_t)(n0 + i) * a.ldK + (int64_t)hr * a.hsK;
    } else {
      if (slot[i] < 0 || slot[i] >= a.n_pages * a.page) continue;
      const int64_t pg = slot[i] <= 0xffffffffll ? (unsigned)slot[i] / (unsigned)a.page : slot[i] / a.page;
      dst = (S*)(isv ? a.V : a.K) + ((pg * a.H_k + hr) * a.page + (slot[i] - pg * a.page)) * D;
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
  const int per = kRopeThreads / (D / 8);
  const dim3 grid((a.N + kRopeTokens - 1) / kRopeTokens, (R + per - 1) / per);
  const bool v = vec_ok(a.q, a.ldq, es) && vec_ok(a.k, a.ldk, es) && vec_ok(a.v, a.ldv, es) &&
                 vec_ok(a.wq, 0, es) && vec_ok(a.wk, 0, es) && vec_ok(a.Q, a.ldQ, es) &&
                 vec_ok(a.K, a.ldK, es) && vec_ok(a.V, 0, es) && (a.hsQ * es) % 16 == 0 &&
                 (a.hsK * es) % 16 == 0;
  const bool pieces = a.rot % (a.layout == MF_ROPE_HALF ? 16 : 8) == 0;
  if (v && pieces) k_rope<TT, D, true, true><<<grid, kRopeThreads, 0, st>>>(a);
  else k_rope<TT, D, false, false><<<grid, kRopeThreads, 0, st>>>(a);
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
