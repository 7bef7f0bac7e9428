// Causal attention with a sliding window and visible first tokens.
//
//   s_ij = scale_h q_i . k_j;  O_i = sum_j exp(s_ij - lse_i) v_j,
//   lse_i = log sum_j exp(s_ij), over j <= p_i with j > p_i - window or j < sinks.
//
// k_attn_tiles (16-byte aligned rows): a workgroup of four wavefronts takes 128
// queries of one head and walks the key tiles that any of them sees (the
// sinks' tiles, then the window's), with the running maximum and sum of the
// softmax.  Both products run transposed on 32x32 matrix instructions:
//   S^T = K Q^T   (A = K rows from LDS, B = Q rows, kept in registers)
//   O^T = V^T P^T (A = V columns by the transposing LDS read, B = P)
// so that a lane owns one query throughout: its scores lie in its registers
// (lane l: query l % 32, keys 8(e/4) + 4(l/32) + e%4), the row statistics need
// one exchange with lane l ^ 32, rescaling is a multiplication by a lane's own
// factor, and exp(S)^T is already the next product's operand: with keys taken
// in the order in which the lane holds them, P never moves between lanes.
// K and V tiles (64 keys; 32 in fp32) pass through registers into two LDS
// buffers while the tile before is computed; 16-byte pieces are XOR-swizzled
// so that both LDS reads are free of bank conflicts without padding.
//
// k_attn_plain: one wavefront per (query, head), 64 keys at a time, one key a
// lane for the scores and two dims a lane for the output.  Any alignment.
#include "mf_attn.h"

#include <algorithm>

namespace {

using namespace mfd;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

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

// ---- tiles on matrix cores -------------------------------------------------

constexpr int kThreads = 256;
constexpr int kRows = 128;                      // queries per workgroup

// What the launch adds to the call's arguments.
struct TileGrid {
  int ntile;                                    // row tiles (packed batch: a bound)
  int nsplit;                                   // parts that the keys are cut into
  float* part;                                  // [nsplit][H][N_q][D], nsplit > 1
  float2* ml;                                   // [nsplit][H][N_q] (max, sum), log2 units
};

// Element type of the tiles: how 16-byte pieces multiply and how weights are
// rounded.
template <class TT> struct Elem;
template <> struct Elem<TBF16> {
  static constexpr unsigned kExp = 0x7f807f80u, kLow = 0x00800080u;
  static __device__ __forceinline__ f32x16 mfma(const u32x4& a, const u32x4& b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ unsigned pack(float x, float y) {
    return __builtin_bit_cast(unsigned, __builtin_convertvector((f32x2{x, y}), bf16x2));
  }
};
template <> struct Elem<TF16> {
  static constexpr unsigned kExp = 0x7c007c00u, kLow = 0x04000400u;
  static __device__ __forceinline__ f32x16 mfma(const u32x4& a, const u32x4& b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ unsigned pack(float x, float y) {
    return __builtin_bit_cast(unsigned, __builtin_convertvector((f32x2{x, y}), f16x2));
  }
};
template <> struct Elem<TF32> {
  static constexpr unsigned kExp = 0x7f800000u, kLow = 0x00800000u;
};

// one of the 16-bit or 32-bit elements packed in w is infinite or NaN
template <class TT>
__device__ __forceinline__ unsigned nonfinite_bits(unsigned w) {
  // an exponent of all ones carries into the (cleared) sign bit
  return ((w & Elem<TT>::kExp) + Elem<TT>::kLow) & (sizeof(typename TT::S) == 4 ? 0x80000000u : 0x80008000u);
}

// Byte offset of 16-byte piece c of row r in a K tile: the 16 lanes of a
// b128 read take one piece of 16 consecutive rows.
template <int RB>
__device__ __forceinline__ int k_piece(int r, int c) {
  if constexpr (RB == 128) return r * RB + 16 * (c ^ ((r >> 1) & 7));
  else return r * RB + 16 * (c ^ (r & 15));
}
// The same in a V tile: a transposing read takes 64 bytes of four consecutive
// rows, which the swizzle spreads over all 64 banks.
template <int RB>
__device__ __forceinline__ int v_piece(int r, int c) {
  if constexpr (RB == 128) return r * RB + 16 * (c ^ (4 * ((r >> 1) & 1)));
  else return r * RB + 16 * (c ^ (4 * (r & 3)));
}

__device__ __forceinline__ float other_half(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

template <class TT, int D>
__global__ __launch_bounds__(kThreads, 2) void k_attn_tiles(const mf::AttnArgs a, const TileGrid tg) {
  using S = typename TT::S;
  using E = Elem<TT>;
  constexpr bool k16 = sizeof(S) == 2;
  constexpr int KT = k16 ? 64 : 32;             // keys per tile
  constexpr int NB = KT / 32;                   // 32-key score blocks per tile
  constexpr int RB = D * (int)sizeof(S);        // bytes per row
  constexpr int CH = RB / 16;                   // 16-byte pieces per row
  constexpr int NP = KT * CH / kThreads;        // pieces of a tile per thread
  constexpr int RSTEP = kThreads / CH;          // rows between a thread's pieces
  constexpr int NQ = RB / 32;                   // 16-byte query pieces per lane
  constexpr int ND = D / 32;                    // 32-dim output blocks
  constexpr int kTile = KT * RB;
  __shared__ __align__(16) unsigned char smem[4 * kTile];   // K0 V0 K1 V1
  __shared__ int bad[2];                        // tile (number + 1) whose V holds a non-finite value

  const int lane = threadIdx.x & 63, hf = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Work item: heads that share K and V stay on one XCD (workgroups go to the
  // eight XCDs in turn), the row tiles with the most keys come first.
  int h, rest;
  if (a.H % 8 == 0) {
    const int hx = a.H / 8, i = blockIdx.x >> 3;
    h = (blockIdx.x & 7) * hx + i % hx;
    rest = i / hx;
  } else {
    h = blockIdx.x % a.H;
    rest = blockIdx.x / a.H;
  }
  int tile = tg.ntile - 1 - rest % tg.ntile;
  const int split = rest / tg.ntile;
  const int g = h / (a.H / a.H_kv);
  SeqRows sr{0, a.N_q, 0, a.N_k};
  if (a.cu_q) {
    // sequence s owns row tiles cu_q[s]/kRows + s and up: at least as many as
    // it needs, and the next sequence starts behind them
    int lo = 0, hi = a.S - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (min(max(a.cu_q[mid], 0), a.N_q) / kRows + mid <= tile) lo = mid; else hi = mid - 1;
    }
    sr = seq_rows(a, lo);
    tile -= sr.q0 / kRows + lo;
  }
  const int n_q = sr.q1 - sr.q0, n_k = sr.k1 - sr.k0;
  const int R0 = tile * kRows;
  if (tile < 0 || R0 >= n_q) return;            // whole workgroup
  const int off = n_k - n_q;                    // position of row 0
  const int Pa = off + R0, Pb = off + min(R0 + kRows, n_q) - 1;

  // key tiles that some row of the workgroup sees
  const int kend = max(Pb + 1, 0);
  const bool win = a.window > 0;
  const int nS = win ? (min(a.sinks, kend) + KT - 1) / KT : 0;
  const int tw0 = max(win ? max(0, Pa - a.window + 1) / KT : 0, nS);
  const int ntl = nS + max(0, (kend + KT - 1) / KT - tw0);
  const int it0 = (int)((int64_t)ntl * split / tg.nsplit);
  const int it1 = (int)((int64_t)ntl * (split + 1) / tg.nsplit);
  auto key0 = [&](int it) { return (it < nS ? it : tw0 + it - nS) * KT; };

  // this wavefront's rows
  const int r0 = R0 + 32 * wave;
  const int p_lo = off + r0, p_hi = off + min(r0 + 31, n_q - 1);
  const int row = r0 + (lane & 31);
  const int p = off + row;
  const float sc = a.scale[h] * kLog2E;
  const float c = fmaxf(fabsf(sc), 1e-45f);     // > 0: the maximum can be taken before scaling
  u32x4 q[NQ];
  {
    const int rr = sr.q0 + min(row, n_q - 1);
    const char* qp = (const char*)a.Q.p + ((int64_t)rr * a.Q.ld + (int64_t)h * a.Q.hs) * sizeof(S) + 16 * hf;
    const unsigned flip = sc < 0.f ? (k16 ? 0x80008000u : 0x80000000u) : 0u;
#pragma unroll
    for (int s = 0; s < NQ; ++s) {
      q[s] = *reinterpret_cast<const u32x4*>(qp + 32 * s);
      q[s] ^= flip;
    }
  }

  // thread's pieces of a tile: rows tr, tr + RSTEP, ..., piece tc
  const int tr = threadIdx.x / CH, tc = threadIdx.x % CH;
  const char* Kg = (const char*)a.K.p + ((int64_t)sr.k0 * a.K.ld + (int64_t)g * a.K.hs) * sizeof(S);
  const char* Vg = (const char*)a.V.p + ((int64_t)sr.k0 * a.V.ld + (int64_t)g * a.V.hs) * sizeof(S);
  const int64_t ldK = a.K.ld * (int64_t)sizeof(S), ldV = a.V.ld * (int64_t)sizeof(S);
  const unsigned ko = (unsigned)(tr * ldK) + 16 * tc, vo = (unsigned)(tr * ldV) + 16 * tc;
  u32x4 ks[NP], vs[NP];
  auto load = [&](int it) {
    const int j0 = key0(it);
    if (j0 + KT <= n_k) {
#pragma unroll
      for (int n = 0; n < NP; ++n) {
        ks[n] = *reinterpret_cast<const u32x4*>(Kg + (j0 + n * RSTEP) * ldK + ko);
        vs[n] = *reinterpret_cast<const u32x4*>(Vg + (j0 + n * RSTEP) * ldV + vo);
      }
    } else {                                    // rows behind the last key: a valid K row, V = 0
#pragma unroll
      for (int n = 0; n < NP; ++n) {
        const int j = j0 + tr + n * RSTEP;
        const int64_t jj = min(j, n_k - 1);
        ks[n] = *reinterpret_cast<const u32x4*>(Kg + jj * ldK + 16 * tc);
        vs[n] = *reinterpret_cast<const u32x4*>(Vg + jj * ldV + 16 * tc);
        if (j >= n_k) vs[n] = u32x4{0, 0, 0, 0};
      }
    }
  };
  auto store = [&](int it) {
    unsigned char* kb = smem + (it & 1) * 2 * kTile;
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      *reinterpret_cast<u32x4*>(kb + k_piece<RB>(tr + n * RSTEP, tc)) = ks[n];
      *reinterpret_cast<u32x4*>(kb + kTile + v_piece<RB>(tr + n * RSTEP, tc)) = vs[n];
    }
    // a masked key's weight is 0, but 0 * inf is not: note tiles that need care
    const int j0 = key0(it), j1 = j0 + KT - 1;
    if (!(j1 <= Pa && (!win || j0 > Pb - a.window || j1 < a.sinks))) {
      unsigned f = 0;
#pragma unroll
      for (int n = 0; n < NP; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) f |= nonfinite_bits<TT>(vs[n][i]);
      if (f) bad[it & 1] = it + 1;
    }
  };

  f32x16 o[ND];
#pragma unroll
  for (int b = 0; b < ND; ++b) o[b] = f32x16{};
  float m = -INFINITY, l = 0.f;                 // raw maximum; this half's sum

  if (threadIdx.x < 2) bad[threadIdx.x] = 0;
  __syncthreads();
  if (it0 < it1) {
    load(it0);
    store(it0);
  }
  __syncthreads();
  for (int it = it0; it < it1; ++it) {
    if (it + 1 < it1) load(it + 1);
    const int j0 = key0(it), j1 = j0 + KT - 1;
    const bool none = r0 >= n_q || j0 > p_hi || (win && j1 <= p_lo - a.window && j0 >= a.sinks);
    if (!none) {
      const unsigned char* kb = smem + (it & 1) * 2 * kTile;
      const unsigned char* vb = kb + kTile;
      f32x16 x[NB];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        x[nb] = f32x16{};
#pragma unroll
        for (int s = 0; s < NQ; ++s) {
          const u32x4 kk = *reinterpret_cast<const u32x4*>(kb + k_piece<RB>(32 * nb + (lane & 31), 2 * s + hf));
          if constexpr (k16) {
            x[nb] = E::mfma(kk, q[s], x[nb]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              x[nb] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(kk[i]), __uint_as_float(q[s][i]),
                                                           x[nb], 0, 0, 0);
          }
        }
      }
      const bool full = j1 <= p_lo && (!win || j0 > p_hi - a.window || j1 < a.sinks);
      auto seen = [&](int nb, int e) {
        const int j = j0 + 32 * nb + 8 * (e >> 2) + 4 * hf + (e & 3);
        return j <= p && (!win || j > p - a.window || j < a.sinks);
      };
      if (!full) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 16; ++e) x[nb][e] = seen(nb, e) ? x[nb][e] : -INFINITY;
      }
      float mx = x[0][0];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 16; ++e) mx = fmaxf(mx, x[nb][e]);
      mx = fmaxf(mx, other_half(mx));
      if (__any(mx > m)) {                      // some row's maximum grows: rescale
        const float mn = fmaxf(m, mx);
        const float f = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - mn) * c);
        l *= f;
#pragma unroll
        for (int b = 0; b < ND; ++b) o[b] *= f;
        m = mn;
      }
      const float mc = m == -INFINITY ? 0.f : m * c;
      float sum = 0.f;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          x[nb][e] = __builtin_amdgcn_exp2f(fmaf(x[nb][e], c, -mc));
          sum += x[nb][e];
        }
      l += sum;
      if (full || bad[it & 1] != it + 1) {
        if constexpr (k16) {
#pragma unroll
          for (int t = 0; t < 2 * NB; ++t) {
            u32x4 pp;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              pp[i] = E::pack(x[t >> 1][8 * (t & 1) + 2 * i], x[t >> 1][8 * (t & 1) + 2 * i + 1]);
#pragma unroll
            for (int b = 0; b < ND; ++b) {
              // four keys of this lane's dim, twice: lane (i of 16) addresses
              // row i / 4, dims 4 (i % 4).. and receives dim i of the four rows
              u32x4 vv;
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const int r = 16 * t + 8 * u + 4 * hf + ((lane & 15) >> 2);
                const int piece = 4 * b + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
                const unsigned char* ad = vb + v_piece<RB>(r, piece) + 8 * (lane & 1);
                const u32x2 w = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) s16x4*)(ad)));
                vv[2 * u] = w[0];
                vv[2 * u + 1] = w[1];
              }
              o[b] = E::mfma(vv, pp, o[b]);
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e)
#pragma unroll
            for (int b = 0; b < ND; ++b) {
              const int r = 8 * (e >> 2) + 4 * hf + (e & 3), dim = 32 * b + (lane & 31);
              const float vv = *reinterpret_cast<const float*>(vb + v_piece<RB>(r, dim >> 2) + 4 * (dim & 3));
              o[b] = __builtin_amdgcn_mfma_f32_32x32x2f32(vv, x[0][e], o[b], 0, 0, 0);
            }
        }
      } else {
        // Rare: V holds infinities or NaN and some of these keys are masked.
        // Key by key, masked keys left out; both halves need each weight.
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          for (int e = 0; e < 16; ++e) {
            const float w0 = x[nb][0];
#pragma unroll
            for (int i = 0; i < 15; ++i) x[nb][i] = x[nb][i + 1];
            float wr = w0;
            if constexpr (k16) wr = TT::tof(TT::fromf(w0));
            for (int hh = 0; hh < 2; ++hh) {
              const int r = 32 * nb + 8 * (e >> 2) + 4 * hh + (e & 3);
              const float w = __shfl(wr, (lane & 31) + 32 * hh);
              const int j = j0 + r;
              if (j <= p && (!win || j > p - a.window || j < a.sinks)) {
#pragma unroll
                for (int b = 0; b < ND; ++b)
#pragma unroll
                  for (int i = 0; i < 16; ++i) {
                    const int dim = 32 * b + 8 * (i >> 2) + 4 * hf + (i & 3);
                    constexpr int PE = 16 / (int)sizeof(S);
                    const S v = *reinterpret_cast<const S*>(vb + v_piece<RB>(r, dim / PE) + (dim % PE) * sizeof(S));
                    o[b][i] = fmaf(w, TT::tof(v), o[b][i]);
                  }
              }
            }
          }
        }
      }
    }
    if (it + 1 < it1) store(it + 1);
    __syncthreads();
  }

  l += other_half(l);
  if (row >= n_q) return;
  const int64_t i = sr.q0 + row;
  if (tg.nsplit > 1) {
    const int64_t at = ((int64_t)split * a.H + h) * a.N_q + i;
    if (hf == 0) tg.ml[at] = make_float2(m == -INFINITY ? -INFINITY : m * c, l);
    float* op = tg.part + at * D + 4 * hf;
#pragma unroll
    for (int b = 0; b < ND; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<f32x4*>(op + 32 * b + 8 * e) =
            f32x4{o[b][4 * e], o[b][4 * e + 1], o[b][4 * e + 2], o[b][4 * e + 3]};
    return;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (a.lse && hf == 0)
    a.lse[(int64_t)h * a.N_q + i] = l == 0.f ? -INFINITY : (m * c + log2f(l)) * kLn2f;
  S* op = (S*)a.O + i * a.ldO + (int64_t)h * D + 4 * hf;
#pragma unroll
  for (int b = 0; b < ND; ++b)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (k16) {
        *reinterpret_cast<u32x2*>(op + 32 * b + 8 * e) =
            u32x2{E::pack(o[b][4 * e] * inv, o[b][4 * e + 1] * inv),
                  E::pack(o[b][4 * e + 2] * inv, o[b][4 * e + 3] * inv)};
      } else {
        *reinterpret_cast<f32x4*>(op + 32 * b + 8 * e) =
            f32x4{o[b][4 * e] * inv, o[b][4 * e + 1] * inv, o[b][4 * e + 2] * inv, o[b][4 * e + 3] * inv};
      }
    }
}

// Joins the parts of split keys in part order; one wavefront per (query, head).
template <class TT, int D>
__global__ __launch_bounds__(256) void k_attn_join(const mf::AttnArgs a, const TileGrid tg) {
  using S = typename TT::S;
  constexpr int NE = D / 64;
  const int lane = threadIdx.x & 63;
  const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int h = blockIdx.y;
  if (i >= a.N_q) return;
  float m = -INFINITY, l = 0.f, acc[NE] = {};
  for (int s = 0; s < tg.nsplit; ++s) m = fmaxf(m, tg.ml[((int64_t)s * a.H + h) * a.N_q + i].x);
  const float mu = m == -INFINITY ? 0.f : m;
  for (int s = 0; s < tg.nsplit; ++s) {
    const int64_t at = ((int64_t)s * a.H + h) * a.N_q + i;
    const float2 ml = tg.ml[at];
    const float f = __builtin_amdgcn_exp2f(ml.x - mu);
    l += ml.y * f;
    if (ml.y == 0.f) continue;                  // no key of this part is visible
#pragma unroll
    for (int c = 0; c < NE; ++c) acc[c] = fmaf(tg.part[at * D + NE * lane + c], f, acc[c]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  S* o = (S*)a.O + i * a.ldO + (int64_t)h * D + NE * lane;
#pragma unroll
  for (int c = 0; c < NE; ++c) o[c] = TT::fromf(acc[c] * inv);
  if (a.lse && lane == 0)
    a.lse[(int64_t)h * a.N_q + i] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2f;
}

bool rows16(const void* p, int64_t ld, int64_t hs, int es) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * es) % 16 == 0 && (hs * es) % 16 == 0;
}

// Parts that the keys of a call are cut into: with fewer row tiles than half
// the CUs hold workgroups (two each), enough parts to fill them, each of at
// least kMinPart key tiles.
constexpr int kMinPart = 4;
int split_of(int H, int N_q, int N_k, int KT, int window, int sinks) {
  const int64_t wgs = (int64_t)H * ((N_q + kRows - 1) / kRows);
  if (wgs > 256) return 1;
  int64_t keys = N_k;
  if (window > 0) keys = std::min<int64_t>(keys, (int64_t)window + sinks + kRows);
  const int64_t tiles = (keys + KT - 1) / KT;
  return (int)std::max<int64_t>(1, std::min<int64_t>({(512 + wgs - 1) / wgs, tiles / kMinPart, 64}));
}

template <class TT, int D>
hipError_t run_tiles(const mf::AttnArgs& a, const TileGrid& tg, hipStream_t st) {
  const int64_t wgs = (int64_t)tg.ntile * a.H * tg.nsplit;
  k_attn_tiles<TT, D><<<(unsigned)wgs, kThreads, 0, st>>>(a, tg);
  if (tg.nsplit > 1)
    k_attn_join<TT, D><<<dim3((a.N_q + 3) / 4, a.H), 256, 0, st>>>(a, tg);
  return hipGetLastError();
}

template <class TT>
hipError_t run_plain(const mf::AttnArgs& a, hipStream_t st) {
  const dim3 grid((a.N_q + 3) / 4, a.H);
  if (a.d == 64) k_attn_plain<TT, 64><<<grid, 256, 0, st>>>(a);
  else k_attn_plain<TT, 128><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

template <class TT>
hipError_t run(mf::AttnArgs a, void* ws, size_t ws_bytes, size_t need, int KT, hipStream_t st) {
  constexpr int es = sizeof(typename TT::S);
  // a window that reaches every key is none; bounds the kernels' sums too
  if (a.window >= a.N_k) a.window = 0;
  a.sinks = std::min(a.sinks, a.N_k);
  const int64_t reach = (int64_t)(kThreads / 8) * es;     // largest row offset of a thread's first piece
  const bool tiles = rows16(a.Q.p, a.Q.ld, a.Q.hs, es) && rows16(a.K.p, a.K.ld, a.K.hs, es) &&
                     rows16(a.V.p, a.V.ld, a.V.hs, es) && rows16(a.O, a.ldO, 0, es) &&
                     a.K.ld < (int64_t(1) << 31) / reach && a.V.ld < (int64_t(1) << 31) / reach;
  if (!tiles) return run_plain<TT>(a, st);
  TileGrid tg{};
  tg.ntile = a.cu_q ? a.N_q / kRows + a.S : (a.N_q + kRows - 1) / kRows;
  tg.nsplit = 1;
  if (!a.cu_q && need > 0 && ws && ws_bytes >= need) {
    tg.nsplit = split_of(a.H, a.N_q, a.N_k, KT, a.window, a.sinks);
    tg.part = (float*)ws;
    tg.ml = (float2*)(tg.part + (int64_t)tg.nsplit * a.H * a.N_q * a.d);
  }
  return a.d == 64 ? run_tiles<TT, 64>(a, tg, st) : run_tiles<TT, 128>(a, tg, st);
}

}  // namespace

namespace mf {

size_t attention_split_bytes(int dt, int H, int, int N_q, int N_k, int d, int window, int sinks) {
  if (window >= N_k) window = 0;
  const int ns = split_of(H, N_q, N_k, dt == MF_F32 ? 32 : 64, window, std::min(sinks, N_k));
  return ns > 1 ? (size_t)ns * H * N_q * ((size_t)d * 4 + 8) : 0;
}

hipError_t launch_attention(int dt, const AttnArgs& a, void* ws, size_t ws_bytes, hipStream_t st) {
  const size_t need = a.cu_q || a.N_k == 0
      ? 0 : attention_split_bytes(dt, a.H, a.H_kv, a.N_q, a.N_k, a.d, a.window, a.sinks);
  if (dt == MF_F32) return run<TF32>(a, ws, ws_bytes, need, 32, st);
  if (dt == MF_F16) return run<TF16>(a, ws, ws_bytes, need, 64, st);
  return run<TBF16>(a, ws, ws_bytes, need, 64, st);
}

}  // namespace mf
