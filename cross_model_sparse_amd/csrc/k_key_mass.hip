// Accumulated attention weight of every key of a prompt:
//   mass[g][j] = mass_in[g][j] + sum_{h of g} sum_i exp(s_h[i][j] - lse[h][i]).
//
// Bound by the matrix cores and the exponentials alike: one 2d-flop product and
// one exponential for every visible (query, key) pair, against few bytes.
// k_key_mass_tiles (16-byte aligned rows): a workgroup takes 256 keys of one
// query head (fp32: 128) and a run of queries.  S = Q K^T on 32x32 matrix
// instructions, A = 32 query rows from LDS, B = 32 key rows, which stay in
// registers for the whole run: 64 keys a wavefront (fp32: 32), so that a query
// piece read from LDS feeds two instructions.  A lane then owns one key: its 16
// scores of a block are 16 queries, whose negated log-sum-exps are added by the
// scaling fma, and the sum over queries never leaves the lane but for one
// exchange of halves at the end.  Query tiles pass through registers into two
// LDS buffers.  Runs leave fp32 sums in the workspace (a lane adds 16 terms to a
// tile's sum, at most 256 tiles' sums to a run's); k_key_mass_reduce adds runs
// and heads in a fixed order in fp64.
// Measured (d = 128, bf16, causal): N = 8192, 40 heads 376 to 390 us (880 to 915
// TFLOP/s); N = 1000, 32 heads, fp16 30 us.
//
// k_key_mass_plain: one thread per (KV head, key).  Any alignment.
#include "mf_attn.h"

#include <math.h>

#include <algorithm>
#include <type_traits>

namespace {

using namespace mfd;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

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

// ---- tiles on matrix cores -------------------------------------------------

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

struct Runs {
  int len;                                      // queries per run, a multiple of 64
  int count;                                    // runs of N_q
  int blocks;                                   // key blocks of a workgroup
  float* part;                                  // [H][count][N_k]
};

// queries that may see a key of [j0, j1): [first, last)
__device__ __forceinline__ void seers(const mf::KeyMassArgs& a, int j0, int j1, int& first, int& last) {
  const int off = a.N_k - a.N_q;
  first = max(0, j0 - off);
  last = a.N_q;
  if (a.window > 0 && j0 >= a.sinks)
    last = (int)max((int64_t)0, min((int64_t)a.N_q, (int64_t)j1 - 1 + a.window - off));
}

template <int RB>
__device__ __forceinline__ int q_piece(int r, int c) {
  if constexpr (RB == 128) return r * RB + 16 * (c ^ ((r >> 1) & 7));
  else return r * RB + 16 * (c ^ (r & 15));
}

template <class TT>
__device__ __forceinline__ f32x16 mfma(const u32x4& x, const u32x4& y, f32x16 c) {
  if constexpr (std::is_same<TT, TBF16>::value)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x),
                                                   __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
  else if constexpr (std::is_same<TT, TF16>::value)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, x),
                                                  __builtin_bit_cast(f16x8, y), c, 0, 0, 0);
  else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(x[i]), __uint_as_float(y[i]), c, 0, 0, 0);
    return c;
  }
}

template <class TT, int D>
__global__ __launch_bounds__(kThreads, 2) void k_key_mass_tiles(const mf::KeyMassArgs a, const Runs rn) {
  using S = typename TT::S;
  constexpr bool k16 = sizeof(S) == 2;
  constexpr int QT = k16 ? 64 : 32;             // queries per tile
  constexpr int NB = k16 ? 2 : 1;               // 32-key blocks per wavefront
  constexpr int RB = D * (int)sizeof(S);
  constexpr int CH = RB / 16;
  constexpr int NP = QT * CH / kThreads;        // pieces of a tile per thread
  constexpr int RSTEP = kThreads / CH;
  constexpr int NQ = RB / 32;                   // 16-byte pieces per lane and row
  constexpr int kTile = QT * RB;
  __shared__ __align__(16) unsigned char smem[2 * kTile];
  __shared__ __align__(16) float nlse[2][QT];   // -lse in log2 units; -infinity: adds nothing
  __shared__ int dead[2];                       // tile (number + 1) that holds such a query

  const int lane = threadIdx.x & 63, hf = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // heads that share K, and the key blocks that share Q, stay on one XCD
  int h, rest;
  if (a.H % 8 == 0) {
    const int hx = a.H / 8, i = blockIdx.x >> 3;
    h = (blockIdx.x & 7) * hx + i % hx;
    rest = i / hx;
  } else {
    h = blockIdx.x % a.H;
    rest = blockIdx.x / a.H;
  }
  const int run = rest / rn.blocks;
  const int J0 = (rest % rn.blocks) * (32 * NB * kWaves);
  const int J1 = min(J0 + 32 * NB * kWaves, a.N_k);
  const int g = h / (a.H / a.H_kv);
  const int off = a.N_k - a.N_q;
  const bool win = a.window > 0;
  int first, last;
  seers(a, J0, J1, first, last);
  const int i0 = max(first / QT * QT, run * rn.len), i1 = min(last, run * rn.len + rn.len);
  if (i0 >= i1) return;                         // the reduction leaves this run out too
  const int ntl = (i1 - i0 + QT - 1) / QT;

  // this wavefront's keys, one a lane and block, stay in registers
  const int j0 = J0 + 32 * NB * wave, j1 = j0 + 32 * NB - 1;
  const float sc = a.scale[h] * kLog2E;
  const float c = fabsf(sc);
  u32x4 k[NB][NQ];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int64_t j = min(j0 + 32 * nb + (lane & 31), a.N_k - 1);
    const char* kp = (const char*)a.K.p + (j * a.K.ld + (int64_t)g * a.K.hs) * (int64_t)sizeof(S) + 16 * hf;
    const unsigned flip = sc < 0.f ? (k16 ? 0x80008000u : 0x80000000u) : 0u;
#pragma unroll
    for (int s = 0; s < NQ; ++s) {
      k[nb][s] = *reinterpret_cast<const u32x4*>(kp + 32 * s);
      k[nb][s] ^= flip;
    }
  }

  const int tr = threadIdx.x / CH, tc = threadIdx.x % CH;
  const char* Qg = (const char*)a.Q.p + (int64_t)h * a.Q.hs * (int64_t)sizeof(S);
  const int64_t ldQ = a.Q.ld * (int64_t)sizeof(S);
  const float* lse = a.lse + (int64_t)h * a.N_q;
  u32x4 qs[NP];
  float ls = 0.f;
  auto load = [&](int it) {
    const int q0 = i0 + it * QT;
#pragma unroll
    for (int n = 0; n < NP; ++n)
      qs[n] = *reinterpret_cast<const u32x4*>(
          Qg + (int64_t)min(q0 + tr + n * RSTEP, a.N_q - 1) * ldQ + 16 * tc);
    const int i = q0 + (int)threadIdx.x;
    if (threadIdx.x < QT) ls = i < i1 ? -lse[i] * kLog2E : -INFINITY;
  };
  auto store = [&](int it) {
    const int b = it & 1;
#pragma unroll
    for (int n = 0; n < NP; ++n)
      *reinterpret_cast<u32x4*>(smem + b * kTile + q_piece<RB>(tr + n * RSTEP, tc)) = qs[n];
    if (threadIdx.x < QT) {
      // lse = -infinity: the query saw no key
      const bool none = ls == INFINITY || ls == -INFINITY;
      nlse[b][threadIdx.x] = none ? -INFINITY : ls;
      if (none) dead[b] = it + 1;
    }
  };

  float acc[NB] = {};
  if (threadIdx.x < 2) dead[threadIdx.x] = 0;
  __syncthreads();
  load(0);
  store(0);
  __syncthreads();
  for (int it = 0; it < ntl; ++it) {
    if (it + 1 < ntl) load(it + 1);
    const int b = it & 1, q0 = i0 + it * QT;
    const int p0 = off + q0, p1 = p0 + QT - 1;  // positions of the tile
    const bool none = j0 > p1 || j0 >= a.N_k || (win && j1 <= p0 - a.window && j0 >= a.sinks);
    if (!none) {
      const bool full = j1 <= p0 && (!win || j0 > p1 - a.window || j1 < a.sinks) && dead[b] != it + 1;
#pragma unroll
      for (int rb = 0; rb < QT / 32; ++rb) {
        f32x16 x[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) x[nb] = f32x16{};
#pragma unroll
        for (int s = 0; s < NQ; ++s) {
          const u32x4 qq = *reinterpret_cast<const u32x4*>(
              smem + b * kTile + q_piece<RB>(32 * rb + (lane & 31), 2 * s + hf));
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) x[nb] = mfma<TT>(qq, k[nb][s], x[nb]);
        }
        f32x4 nl[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          nl[e] = *reinterpret_cast<const f32x4*>(&nlse[b][32 * rb + 8 * e + 4 * hf]);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float t = 0.f;
          if (full) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              t += __builtin_amdgcn_exp2f(fmaf(x[nb][e], c, nl[e >> 2][e & 3]));
          } else {
            const int j = j0 + 32 * nb + (lane & 31);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int p = p0 + 32 * rb + 8 * (e >> 2) + 4 * hf + (e & 3);
              const bool vis = j <= p && (!win || j > p - a.window || j < a.sinks);
              const float y = nl[e >> 2][e & 3];
              t += vis && y != -INFINITY ? __builtin_amdgcn_exp2f(fmaf(x[nb][e], c, y)) : 0.f;
            }
          }
          acc[nb] += t;
        }
      }
    }
    if (it + 1 < ntl) store(it + 1);
    __syncthreads();
  }
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    acc[nb] += __shfl_xor(acc[nb], 32);
    const int j = j0 + 32 * nb + (lane & 31);
    if (hf == 0 && j < a.N_k) rn.part[((int64_t)h * rn.count + run) * a.N_k + j] = acc[nb];
  }
}

// one thread per (KV head, key): the runs that hold queries of its key block,
// head after head
__global__ __launch_bounds__(256) void k_key_mass_reduce(const mf::KeyMassArgs a, const Runs rn, int QT,
                                                         int block) {
  const int j = blockIdx.x * 256 + threadIdx.x, g = blockIdx.y, G = a.H / a.H_kv;
  if (j >= a.N_k) return;
  int first, last;
  const int J0 = j / block * block;
  seers(a, J0, min(J0 + block, a.N_k), first, last);
  first = first / QT * QT;
  double sum = a.mass_in ? a.mass_in[(int64_t)g * a.N_k + j] : 0.f;
  const int r0 = first / rn.len, r1 = last > first ? (last - 1) / rn.len + 1 : r0;
  for (int h = g * G; h < (g + 1) * G; ++h)
    for (int r = r0; r < r1; ++r) sum += rn.part[((int64_t)h * rn.count + r) * a.N_k + j];
  a.mass_out[(int64_t)g * a.N_k + j] = (float)sum;
}

bool rows16(const mf::Strided& x, int es) {
  return reinterpret_cast<uintptr_t>(x.p) % 16 == 0 && (x.ld * es) % 16 == 0 && (x.hs * es) % 16 == 0;
}

// Length of the runs of queries, at most 8192.  Every run costs a start (keys
// into registers, the first tile's latency) and the last ones leave CUs idle for
// half a run: with W queries in all, over heads and key blocks, the sum of both
// is least near sqrt(W).  Measured around it (d = 128, bf16): N = 2048, 32 heads
// 42 us with 512 queries, 50 with 256, 48 with 1024; window 1024 at N = 8192, 32
// heads 178 us with 1024, 216 with 2048, 340 with 4096; N = 8192, 40 heads,
// causal within 4% from 1280 to 5120.
Runs runs_of(int dt, int H, int N_q, int N_k, int window, int sinks) {
  Runs rn{};
  const int block = dt == MF_F32 ? 32 * kWaves : 64 * kWaves;
  rn.blocks = (N_k + block - 1) / block;
  // W from at most 64 of the key blocks
  const int n = std::min(rn.blocks, 64);
  double seen = 0;
  for (int i = 0; i < n; ++i) {
    const int64_t j0 = (int64_t)rn.blocks * i / n * block;
    int64_t q = std::min<int64_t>(N_q, N_k - j0);
    if (window > 0 && j0 >= sinks) q = std::min<int64_t>(q, (int64_t)window + block);
    seen += (double)q;
  }
  if (n > 0) seen *= (double)rn.blocks / n;
  const int64_t len = (int64_t)sqrt(0.65 * seen * H);
  rn.len = (int)std::min<int64_t>(8192, (len + 63) / 64 * 64);
  rn.len = std::max(rn.len, 64);
  rn.count = (N_q + rn.len - 1) / rn.len;
  return rn;
}

template <class TT, int D>
hipError_t run_tiles(const mf::KeyMassArgs& a, const Runs& rn, hipStream_t st) {
  constexpr bool k16 = sizeof(typename TT::S) == 2;
  const int64_t wgs = (int64_t)a.H * rn.blocks * rn.count;
  if (wgs > 0) k_key_mass_tiles<TT, D><<<(unsigned)wgs, kThreads, 0, st>>>(a, rn);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_key_mass_reduce<<<dim3((a.N_k + 255) / 256, a.H_kv), 256, 0, st>>>(a, rn, k16 ? 64 : 32,
                                                                     32 * kWaves * (k16 ? 2 : 1));
  return hipGetLastError();
}

template <class TT>
hipError_t run_plain(const mf::KeyMassArgs& a, hipStream_t st) {
  const dim3 grid((a.N_k + 63) / 64, a.H_kv);
  if (a.d == 64) k_key_mass_plain<TT, 64><<<grid, 64, 0, st>>>(a);
  else k_key_mass_plain<TT, 128><<<grid, 64, 0, st>>>(a);
  return hipGetLastError();
}

template <class TT>
hipError_t run(int dt, mf::KeyMassArgs a, void* ws, hipStream_t st) {
  constexpr int es = sizeof(typename TT::S);
  if (a.window >= a.N_k) a.window = 0;          // reaches every key
  a.sinks = std::min(a.sinks, a.N_k);
  if (!rows16(a.Q, es) || !rows16(a.K, es)) return run_plain<TT>(a, st);
  Runs rn = runs_of(dt, a.H, a.N_q, a.N_k, a.window, a.sinks);
  rn.part = (float*)ws;
  return a.d == 64 ? run_tiles<TT, 64>(a, rn, st) : run_tiles<TT, 128>(a, rn, st);
}

}  // namespace

namespace mf {

size_t key_mass_workspace_bytes(int dt, int H, int, int N_q, int N_k, int, int window, int sinks) {
  if (window >= N_k) window = 0;
  const Runs rn = runs_of(dt, H, N_q, N_k, window, std::min(sinks, N_k));
  return (size_t)H * rn.count * N_k * 4;
}

hipError_t launch_key_mass(int dt, const KeyMassArgs& a, void* ws, hipStream_t st) {
  if (dt == MF_F32) return run<TF32>(dt, a, ws, st);
  if (dt == MF_F16) return run<TF16>(dt, a, ws, st);
  return run<TBF16>(dt, a, ws, st);
}

}  // namespace mf
