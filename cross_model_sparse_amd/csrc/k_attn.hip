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
// K and V tiles (64 keys; 32 in fp32) are copied straight into two LDS buffers
// each, a tile ahead (K two); 16-byte pieces are XOR-swizzled so that both LDS
// reads are free of bank conflicts without padding.
// A weight is rounded to the storage type before it multiplies V (the matrix
// instruction takes one type; a second product for the rest would cost half of
// the time again); sums, maxima and accumulators are fp32.
//
// Bound by the matrix cores together with the vector ALU: 32 products, 32
// exponentials and about 120 other vector instructions for a wavefront's 32 x 64
// tile at d = 128, which overlap within one wavefront and between the two of a
// SIMD (counters: matrix cores 48% busy, vector ALU 43%, LDS 24%, at 1.9 GHz
// under the load).  Measured, 32 heads, 8 KV heads, d = 128, bf16, causal:
// N = 32768 8.2 to 8.5 ms (1035 to 1077 TFLOP/s; an 8192^3 library product
// reaches 1188), N = 8192 560 us (980), window 1024 at N = 8192 177 us (728 of
// the visible pairs; the tiles' own pairs are 20% more).
//
// k_attn_plain: one wavefront per (query, head), 64 keys at a time, one key a
// lane for the scores and two dims a lane for the output.  Any alignment.
#include "mf_attn.h"

#include <algorithm>
#include <type_traits>

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

// One (query, head) by one wavefront over chunks of 64 keys: one key a lane for
// the scores, D / 64 dims a lane for the output, masked keys never multiplied.
template <class TT, int D>
struct PlainRow {
  static constexpr int ND = D / 64;
  using S = typename TT::S;
  float m = -INFINITY, l = 0.f, acc[ND] = {};

  __device__ __forceinline__ void chunk(const S* q, const S* K, int64_t ldK, const S* V, int64_t ldV,
                                        float sc, int j0, bool vis) {
    const int lane = threadIdx.x & 63;
    float x = -INFINITY;
    if (vis) {
      const S* k = K + (int64_t)(j0 + lane) * ldK;
      float dot = 0.f;
      for (int e = 0; e < D; ++e) dot = fmaf(TT::tof(q[e]), TT::tof(k[e]), dot);
      x = dot * sc;
    }
    float mx = x;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
    mx = fmaxf(mx, m);
    if (mx == -INFINITY && !__any(x != x)) return;
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
      const S* v = V + (int64_t)(j0 + kk) * ldV;
#pragma unroll
      for (int c = 0; c < ND; ++c) acc[c] = fmaf(pk, TT::tof(v[lane + 64 * c]), acc[c]);
    }
  }
  __device__ __forceinline__ void finish(const mf::AttnArgs& a, int64_t i, int h) const {
    const int lane = threadIdx.x & 63;
    const bool empty = l == 0.f;
    S* o = (S*)a.O + i * a.ldO + (int64_t)h * D;
#pragma unroll
    for (int c = 0; c < ND; ++c) o[lane + 64 * c] = TT::fromf(empty ? 0.f : acc[c] / l);
    if (a.lse && lane == 0)
      a.lse[(int64_t)h * a.N_q + i] = empty ? -INFINITY : (m + log2f(l)) * kLn2f;
  }
};

template <class TT, int D>
__global__ __launch_bounds__(256) void k_attn_plain(const mf::AttnArgs a) {
  using S = typename TT::S;
  const int lane = threadIdx.x & 63;
  const int i = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int h = blockIdx.y, g = h / (a.H / a.H_kv);
  if (i >= a.N_q) return;
  SeqRows r{0, a.N_q, 0, a.N_k};
  if (a.cu_q) {
    // first sequence that ends behind row i
    int lo = 0, hi = a.S;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (a.cu_q[mid + 1] <= i) lo = mid + 1; else hi = mid;
    }
    if (lo >= a.S) return;                      // behind the last sequence
    r = seq_rows(a, lo);
    if (i < r.q0 || i >= r.q1) return;
  }
  const int p = r.k1 - r.k0 - (r.q1 - r.q0) + (i - r.q0);
  const S* q = (const S*)a.Q.p + (int64_t)i * a.Q.ld + (int64_t)h * a.Q.hs;
  const S* K = (const S*)a.K.p + (int64_t)r.k0 * a.K.ld + (int64_t)g * a.K.hs;
  const S* V = (const S*)a.V.p + (int64_t)r.k0 * a.V.ld + (int64_t)g * a.V.hs;
  const float sc = a.scale[h] * kLog2E;
  const int w0 = a.window > 0 ? max(0, p - a.window + 1) : 0;
  PlainRow<TT, D> row;
  for (int j0 = 0; j0 <= p; j0 += 64) {
    if (j0 >= a.sinks && j0 + 63 < w0) { j0 = (w0 & ~63) - 64; continue; }
    const int j = j0 + lane;
    row.chunk(q, K, a.K.ld, V, a.V.ld, sc, j0, j <= p && (j >= w0 || j < a.sinks));
  }
  row.finish(a, i, h);
}

// ---- tiles on matrix cores -------------------------------------------------

constexpr int kThreads = 256;
constexpr int kRows = 128;                      // queries per workgroup

// What the launch adds to the call's arguments.
struct TileGrid {
  int ntile;                                    // row tiles (packed batch: a bound)
  int len;                                      // key tiles per part; 0: one part
  int nparts;                                   // parts of the longest row tile
  int total;                                    // workgroups per head
  float* part;                                  // [nparts][H][N_q][D], len > 0
  float2* ml;                                   // [nparts][H][N_q] (max, sum), log2 units
};

// The key tiles (KT keys) that rows at positions Pa..Pb see: the sinks' tiles
// 0..nS-1, then tiles tw0.. up to the last row's own.
struct KeyTiles {
  int nS, tw0, count;
  __host__ __device__ __forceinline__ KeyTiles(int window, int sinks, int Pa, int Pb, int KT) {
    const int kend = Pb + 1 > 0 ? Pb + 1 : 0;
    const int first = window > 0 && Pa - window + 1 > 0 ? (Pa - window + 1) / KT : 0;
    nS = window > 0 ? ((sinks < kend ? sinks : kend) + KT - 1) / KT : 0;
    tw0 = first > nS ? first : nS;
    const int rest = (kend + KT - 1) / KT - tw0;
    count = nS + (rest > 0 ? rest : 0);
  }
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

// 16-byte piece c of row r lies at place c ^ swizzle(r) of its row.  In a K
// tile the 16 lanes of a b128 read take one piece of 16 consecutive rows; in a
// V tile a transposing read takes 64 bytes of four consecutive rows: either way
// the swizzle spreads them over all 64 banks.
template <int RB>
__device__ __forceinline__ constexpr int k_swizzle(int r) { return RB == 128 ? (r >> 1) & 7 : r & 15; }
template <int RB>
__device__ __forceinline__ constexpr int v_swizzle(int r) { return RB == 128 ? 4 * ((r >> 1) & 1) : 4 * (r & 3); }
template <int RB>
__device__ __forceinline__ int k_piece(int r, int c) { return r * RB + 16 * (c ^ k_swizzle<RB>(r)); }
template <int RB>
__device__ __forceinline__ int v_piece(int r, int c) { return r * RB + 16 * (c ^ v_swizzle<RB>(r)); }

__device__ __forceinline__ float other_half(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

// 16 bytes a lane from memory (uniform base, 32-bit offset a lane) into LDS at
// lds + 16 * lane, in flight until wait_copies.  The wait states cover a base
// in registers that a vector instruction wrote, and the copy's read of M0.
__device__ __forceinline__ void copy16(unsigned voff, const void* base, unsigned lds) {
  asm volatile("s_nop 4\n\ts_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :: "s"(lds), "v"(voff), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void wait_copies() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ const char* uniform(const char* p) {
  const unsigned long long v = reinterpret_cast<unsigned long long>(p);
  const unsigned lo = __builtin_amdgcn_readfirstlane((unsigned)v);
  const unsigned hi = __builtin_amdgcn_readfirstlane((unsigned)(v >> 32));
  return reinterpret_cast<const char*>(((unsigned long long)hi << 32) | lo);
}
__device__ __forceinline__ unsigned lds_addr(const void* p) {
  return (unsigned)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

// The rare case of a workgroup whose partly masked tiles hold infinities or NaN
// in V: its rows again, key by key over the same tiles, one wavefront's 32 rows
// from r0 in turn.
template <class TT, int D>
__device__ void redo_rows(const mf::AttnArgs& a, const TileGrid& tg, const SeqRows& sr, int r0, int off,
                          int h, int part, int it0, int it1, int nS, int tw0, int KT) {
  using S = typename TT::S;
  const int lane = threadIdx.x & 63, g = h / (a.H / a.H_kv);
  const S* K = (const S*)a.K.p + (int64_t)sr.k0 * a.K.ld + (int64_t)g * a.K.hs;
  const S* V = (const S*)a.V.p + (int64_t)sr.k0 * a.V.ld + (int64_t)g * a.V.hs;
  const float sc = a.scale[h] * kLog2E;
  for (int r = r0; r < min(r0 + 32, sr.q1 - sr.q0); ++r) {
    const int64_t i = sr.q0 + r;
    const int p = off + r, w0 = a.window > 0 ? max(0, p - a.window + 1) : 0;
    const S* q = (const S*)a.Q.p + i * a.Q.ld + (int64_t)h * a.Q.hs;
    PlainRow<TT, D> row;
    for (int it = it0; it < it1; ++it) {
      const int j0 = (it < nS ? it : tw0 + it - nS) * KT, j = j0 + lane;
      row.chunk(q, K, a.K.ld, V, a.V.ld, sc, j0, lane < KT && j <= p && (j >= w0 || j < a.sinks));
    }
    if (tg.len) {
      const int64_t at = ((int64_t)part * a.H + h) * a.N_q + i;
      if (lane == 0) tg.ml[at] = make_float2(row.m, row.l);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) tg.part[at * D + lane + 64 * c] = row.acc[c];
    } else {
      row.finish(a, i, h);
    }
  }
}

#define PIN() __builtin_amdgcn_sched_barrier(0)

template <class TT, int D>
__global__ __launch_bounds__(kThreads, 2) void k_attn_tiles(const mf::AttnArgs a, const TileGrid tg) {
  using S = typename TT::S;
  using E = Elem<TT>;
  constexpr bool k16 = sizeof(S) == 2;
  constexpr int KT = k16 ? 64 : 32;             // keys per tile
  constexpr int NB = KT / 32;                   // 32-key score blocks per tile
  constexpr int RB = D * (int)sizeof(S);        // bytes per row
  constexpr int CH = RB / 16;                   // 16-byte pieces per row
  constexpr int NQ = RB / 32;                   // 16-byte query pieces per lane
  constexpr int ND = D / 32;                    // 32-dim output blocks
  constexpr int kTile = KT * RB;
  constexpr int NC = kTile / 4 / 1024;          // copies of a wavefront per tile
  constexpr int CR = 1024 / RB;                 // rows per copy
  __shared__ __align__(16) unsigned char smem[4 * kTile];   // K0 K1 V0 V1
  __shared__ int redo;                          // a partly masked tile's V is not finite

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
  int tile = tg.ntile - 1 - rest, part = 0;
  if (tg.len) {
    // Workgroup `rest` of the head among all row tiles' parts: counted by a
    // scan over the tiles, 64 at a time.  (A grid with room for the longest
    // tile's parts at every tile would leave gaps, and a CU that took an empty
    // workgroup does not take another's place in the dispatcher's round.)
    int before = 0;
    for (int t0 = 0;; t0 += 64) {
      const int t = tg.ntile - 1 - t0 - lane;
      int n = 0;
      if (t >= 0) {
        const int P0 = a.N_k - a.N_q + t * kRows, P1 = a.N_k - a.N_q + min((t + 1) * kRows, a.N_q) - 1;
        n = max(1, (KeyTiles(a.window, a.sinks, P0, P1, KT).count + tg.len - 1) / tg.len);
      }
      int incl = n;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int u = __shfl_up(incl, d);
        if (lane >= d) incl += u;
      }
      const int all = __builtin_amdgcn_readlane(incl, 63);
      if (rest < before + all || t0 + 64 >= tg.ntile) {
        const int at = __ffsll((unsigned long long)__ballot(rest < before + incl)) - 1;
        if (at < 0) return;                     // behind the last part
        tile = tg.ntile - 1 - t0 - at;
        part = rest - before - __shfl(incl - n, at);
        break;
      }
      before += all;
    }
    tile = __builtin_amdgcn_readfirstlane(tile);
    part = __builtin_amdgcn_readfirstlane(part);
  }
  const int g = h / (a.H / a.H_kv);
  SeqRows sr{0, a.N_q, 0, a.N_k};
  if (a.cu_q) {
    sr = SeqRows{0, 0, 0, 0};
    int first = 0;
    // sequence s owns row tiles cu_q[s]/kRows + s and up: at least as many as
    // it needs, and the next sequence starts behind them.  A sequence a lane, so
    // that all offsets are one load apart.
    for (int s0 = 0; s0 < a.S; s0 += 64) {
      const int s = s0 + lane;
      SeqRows mine{0, 0, 0, 0};
      if (s < a.S) mine = seq_rows(a, s);
      const uint64_t from = __ballot(s < a.S && mine.q0 / kRows + s <= tile);
      if (from == 0) break;                     // a later sequence's first
      const int at = 63 - __clzll((long long)from);
      sr.q0 = __shfl(mine.q0, at);
      sr.q1 = __shfl(mine.q1, at);
      sr.k0 = __shfl(mine.k0, at);
      sr.k1 = __shfl(mine.k1, at);
      first = sr.q0 / kRows + s0 + at;
    }
    sr.q0 = __builtin_amdgcn_readfirstlane(sr.q0);
    sr.q1 = __builtin_amdgcn_readfirstlane(sr.q1);
    sr.k0 = __builtin_amdgcn_readfirstlane(sr.k0);
    sr.k1 = __builtin_amdgcn_readfirstlane(sr.k1);
    tile -= __builtin_amdgcn_readfirstlane(first);
  }
  const int n_q = sr.q1 - sr.q0, n_k = sr.k1 - sr.k0;
  const int R0 = tile * kRows;
  if (tile < 0 || R0 >= n_q) return;            // whole workgroup
  const int off = n_k - n_q;                    // position of row 0
  const int Pa = off + R0, Pb = off + min(R0 + kRows, n_q) - 1;

  // key tiles that some row of the workgroup sees, and this part of them
  const bool win = a.window > 0;
  const KeyTiles kt(a.window, a.sinks, Pa, Pb, KT);
  const int nS = kt.nS, tw0 = kt.tw0;
  const int it0 = tg.len ? part * tg.len : 0;
  const int it1 = tg.len ? min(it0 + tg.len, kt.count) : kt.count;
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
    const char* qp = (const char*)a.Q.p + ((int64_t)rr * a.Q.ld + (int64_t)h * a.Q.hs) * (int64_t)sizeof(S) + 16 * hf;
    const unsigned flip = sc < 0.f ? (k16 ? 0x80008000u : 0x80000000u) : 0u;
#pragma unroll
    for (int s = 0; s < NQ; ++s) {
      q[s] = *reinterpret_cast<const u32x4*>(qp + 32 * s);
      q[s] ^= flip;
    }
  }

  // Copies: wavefront w fetches rows (KT/4) w .. of a tile, CR rows at a time;
  // lane l lands at byte 16 l, which holds the piece that the swizzle puts there.
  const int64_t ldK = a.K.ld * (int64_t)sizeof(S), ldV = a.V.ld * (int64_t)sizeof(S);
  const char* Kg = (const char*)a.K.p + ((int64_t)sr.k0 * a.K.ld + (int64_t)g * a.K.hs) * (int64_t)sizeof(S);
  const char* Vg = (const char*)a.V.p + ((int64_t)sr.k0 * a.V.ld + (int64_t)g * a.V.hs) * (int64_t)sizeof(S);
  const int cr = lane / CH, cp = lane % CH;     // row within a copy, place within the row
  // The swizzles are linear in the bits of the row, and a lane's row within a
  // copy and the copy's first row have no bit in common.
  const unsigned kx = 16 * (cp ^ k_swizzle<RB>(cr)), vx = 16 * (cp ^ v_swizzle<RB>(cr));
  const unsigned kr = (unsigned)(cr * ldK), vr = (unsigned)(cr * ldV);
  const unsigned lds0 = lds_addr(smem) + wave * (kTile / 4);
  auto copy = [&](int it, int buf, auto isv) {
    constexpr bool kV = decltype(isv)::value;
    const int j0 = key0(it) + wave * (KT / 4);
    const unsigned dst = lds0 + buf * kTile;
    const char* b = uniform(kV ? Vg : Kg);
    const int64_t ld = kV ? ldV : ldK;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const int r = wave * (KT / 4) + CR * n;   // the copy's first row within the tile
      const unsigned x = kV ? vx ^ (16 * v_swizzle<RB>(r)) : kx ^ (16 * k_swizzle<RB>(r));
      const int j = j0 + CR * n;
      if (j + CR <= n_k) {
        copy16(x + (kV ? vr : kr), b + j * ld, dst + 1024 * n);
      } else {                                  // rows behind the last key repeat it
        const int jf = min(j, n_k - 1);
        copy16(x + (unsigned)((min(j + cr, n_k - 1) - jf) * ld), b + jf * ld, dst + 1024 * n);
      }
    }
  };

  f32x16 o[ND];
#pragma unroll
  for (int b = 0; b < ND; ++b) o[b] = f32x16{};
  float m = -INFINITY, l = 0.f;                 // raw maximum; this half's sum

  // LDS places of this lane's operands, for tile buffer 0
  int ka[NQ], va[k16 ? ND : 1];
#pragma unroll
  for (int s = 0; s < NQ; ++s) ka[s] = k_piece<RB>(lane & 31, 2 * s + hf);
  if constexpr (k16) {
    // transposing read: lane (i of 16) addresses row i / 4, dims 4 (i % 4).. and
    // receives dim i of the four rows
#pragma unroll
    for (int b = 0; b < ND; ++b)
      va[b] = v_piece<RB>(4 * hf + ((lane & 15) >> 2), 4 * b + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) +
              8 * (lane & 1) + 2 * kTile;
  }
  auto read_k = [&](int buf, int nb, int s) {
    return *reinterpret_cast<const u32x4*>(smem + ka[s] + buf * kTile + nb * 32 * RB);
  };
  auto read_v = [&](int buf, int t, int b) {    // 16 keys 16 t.., dims 32 b..
    u32x4 vv;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const u32x2 w = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) s16x4*)(smem + va[b] + buf * kTile + (16 * t + 8 * u) * RB)));
      vv[2 * u] = w[0];
      vv[2 * u + 1] = w[1];
    }
    return vv;
  };
  auto qk = [&](const u32x4& kk, int s, f32x16 x) {
    if constexpr (k16) return E::mfma(kk, q[s], x);
    else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(kk[i]), __uint_as_float(q[s][i]), x, 0, 0, 0);
      return x;
    }
  };
  auto full_for = [&](int j0, int lo, int hi) {
    const int j1 = j0 + KT - 1;
    return j1 <= lo && (!win || j0 > hi - a.window || j1 < a.sinks);
  };
  auto row_max = [&](const f32x16 (&x)[NB]) {
    float mx = x[0][0];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 16; ++e) mx = fmaxf(mx, x[nb][e]);
    return mx;
  };
  // Takes a tile's maxima into m.  m follows only when some row's maximum has
  // grown by more than 2^8, so that o is rarely rescaled: weights are then at
  // most 2^8, which every type holds with its full relative precision.
  auto take_max = [&](float mx) {
    mx = fmaxf(mx, other_half(mx));
    if (__any((mx - m) * c > 8.f)) {
      const float mn = fmaxf(m, mx);
      const float f = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - mn) * c);
      l *= f;
#pragma unroll
      for (int b = 0; b < ND; ++b) o[b] *= f;
      m = mn;
    }
  };
  auto mask = [&](int j0, f32x16 (&x)[NB]) {
    // key of element e, less what the lane adds: 32 nb + 8 (e / 4) + e % 4
    const int top = p - j0 - 4 * hf, low = top - a.window, fst = a.sinks - j0 - 4 * hf;
    if (!(win && j0 <= p_hi - a.window)) {      // the diagonal only
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          x[nb][e] = 32 * nb + 8 * (e >> 2) + (e & 3) <= top ? x[nb][e] : -INFINITY;
    } else {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int j = 32 * nb + 8 * (e >> 2) + (e & 3);
          x[nb][e] = j <= top && (j > low || j < fst) ? x[nb][e] : -INFINITY;
        }
    }
  };

  auto look_at_v = [&](int it, const unsigned char* vb) {
    if (full_for(key0(it), Pa, Pb)) return;
    // a masked key's weight is 0, but 0 * inf is not: look for such values
    unsigned f = 0;
#pragma unroll
    for (int n = 0; n < kTile / (16 * kThreads); ++n) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(vb + 16 * (threadIdx.x + kThreads * n));
#pragma unroll
      for (int i = 0; i < 4; ++i) f |= nonfinite_bits<TT>(w[i]);
    }
    if (f) redo = 1;
  };

  if (threadIdx.x == 0) redo = 0;
  f32x16 x[NB];
  if (it0 < it1) {                              // tile it lies in buffer (it - it0) & 1
    copy(it0, 0, std::false_type{});
    copy(it0, 2, std::true_type{});
    if (it0 + 1 < it1) copy(it0 + 1, 1, std::false_type{});
    wait_copies();
  }
  __syncthreads();
  if (it0 < it1) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) x[nb] = f32x16{};
#pragma unroll
    for (int s = 0; s < NQ; ++s) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) x[nb] = qk(read_k(0, nb, s), s, x[nb]);
      PIN();
    }
    if (!full_for(key0(it0), p_lo, p_hi)) mask(key0(it0), x);
    take_max(row_max(x));
  }
  // One tile.  xc holds its scores, masked, and m covers them.  16-bit types:
  // the next tile's products (xn) run beside this one's exponentials, the next
  // maxima beside P V, so that matrix cores and vector ALU work at the same
  // time within one wavefront; the scheduling barriers keep that order.
  auto step = [&](auto P, int it, f32x16 (&xc)[NB], f32x16 (&xn)[NB]) {
    constexpr int b0 = decltype(P)::value, b1 = 1 - b0;
    wait_copies();
    __syncthreads();
    if (it + 2 < it1) copy(it + 2, b0, std::false_type{});
    if (it + 1 < it1) copy(it + 1, 2 + b1, std::true_type{});
    const unsigned char* vb = smem + (2 + b0) * kTile;
    look_at_v(it, vb);
    const float mc = m == -INFINITY ? 0.f : m * c;
    float sum = 0.f, mx = -INFINITY;
    if constexpr (k16) {
      unsigned pp[NB * 8];
      constexpr int AHEAD = 2;                  // steps that K pieces are read ahead
      u32x4 kp[AHEAD + 1][NB], vp[2][ND];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        xn[nb] = f32x16{};
#pragma unroll
        for (int s = 0; s < AHEAD; ++s) kp[s][nb] = read_k(b1, nb, s);
      }
#pragma unroll
      for (int s = 0; s < NQ; ++s) {
        if (s + AHEAD < NQ) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) kp[(s + AHEAD) % (AHEAD + 1)][nb] = read_k(b1, nb, s + AHEAD);
        }
        if (s + 1 == NQ) {
#pragma unroll
          for (int b = 0; b < ND; ++b) vp[0][b] = read_v(b0, 0, b);
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) xn[nb] = qk(kp[s % (AHEAD + 1)][nb], s, xn[nb]);
        constexpr int PER = 16 * NB / NQ;
#pragma unroll
        for (int u = 0; u < PER; u += 2) {
          const int e = s * PER + u;
          const float w0 = __builtin_amdgcn_exp2f(fmaf(xc[e >> 4][e & 15], c, -mc));
          const float w1 = __builtin_amdgcn_exp2f(fmaf(xc[e >> 4][(e & 15) + 1], c, -mc));
          pp[e >> 1] = E::pack(w0, w1);
          sum += w0 + w1;
        }
        PIN();
      }
#pragma unroll
      for (int t = 0; t < 2 * NB; ++t) {
        if (t + 1 < 2 * NB) {
#pragma unroll
          for (int b = 0; b < ND; ++b) vp[(t + 1) & 1][b] = read_v(b0, t + 1, b);
        }
        const u32x4 w = {pp[4 * t], pp[4 * t + 1], pp[4 * t + 2], pp[4 * t + 3]};
#pragma unroll
        for (int b = 0; b < ND; ++b) o[b] = E::mfma(vp[t & 1][b], w, o[b]);
#pragma unroll
        for (int e = 0; e < 8; ++e) mx = fmaxf(mx, xn[t >> 1][8 * (t & 1) + e]);
        PIN();
      }
    } else {
      // one V column element a lane and step, K pieces: both read ahead
      auto read_vf = [&](int e, int b) {
        const int r = 8 * (e >> 2) + 4 * hf + (e & 3), dim = 32 * b + (lane & 31);
        return *reinterpret_cast<const float*>(vb + v_piece<RB>(r, dim >> 2) + 4 * (dim & 3));
      };
      float vp[2][ND];
#pragma unroll
      for (int b = 0; b < ND; ++b) vp[0][b] = read_vf(0, b);
      u32x4 kp[2];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if (e + 1 < 16) {
#pragma unroll
          for (int b = 0; b < ND; ++b) vp[(e + 1) & 1][b] = read_vf(e + 1, b);
        } else {
          kp[0] = read_k(b1, 0, 0);
        }
        const float w = __builtin_amdgcn_exp2f(fmaf(xc[0][e], c, -mc));
        sum += w;
#pragma unroll
        for (int b = 0; b < ND; ++b)
          o[b] = __builtin_amdgcn_mfma_f32_32x32x2f32(vp[e & 1][b], w, o[b], 0, 0, 0);
        PIN();
      }
      if (it + 1 >= it1) {
        l += sum;
        return;
      }
      xn[0] = f32x16{};
#pragma unroll
      for (int s = 0; s < NQ; ++s) {
        if (s + 1 < NQ) kp[(s + 1) & 1] = read_k(b1, 0, s + 1);
        xn[0] = qk(kp[s & 1], s, xn[0]);
        PIN();
      }
      mx = row_max(xn);
    }
    l += sum;
    if (it + 1 < it1) {
      const int jn = key0(it + 1);
      if (!full_for(jn, p_lo, p_hi)) {
        mask(jn, xn);
        mx = row_max(xn);
      }
      take_max(mx);
    }
  };
  f32x16 y[NB];
  for (int it = it0; it < it1; it += 2) {
    step(std::integral_constant<int, 0>{}, it, x, y);
    if (it + 1 >= it1) break;
    step(std::integral_constant<int, 1>{}, it + 1, y, x);
  }

  __syncthreads();
  if (redo) {
    redo_rows<TT, D>(a, tg, sr, r0, off, h, part, it0, it1, nS, tw0, KT);
    return;
  }
  l += other_half(l);
  const int64_t i = sr.q0 + row;
  if (tg.len) {
    if (row >= n_q) return;
    const int64_t at = ((int64_t)part * a.H + h) * a.N_q + i;
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
  if (a.lse && hf == 0 && row < n_q)
    a.lse[(int64_t)h * a.N_q + i] = l == 0.f ? -INFINITY : (m * c + log2f(l)) * kLn2f;
  if constexpr (k16) {
    // A lane holds four dims at a time of its own row: through LDS (each
    // wavefront its own part of the tiles' buffers, which nobody reads any
    // more) to whole rows, 16 bytes a lane.
    unsigned char* ob = smem + wave * kTile;
    const int rl = lane & 31;
#pragma unroll
    for (int b = 0; b < ND; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<u32x2*>(ob + k_piece<RB>(rl, 4 * b + e) + 8 * hf) =
            u32x2{E::pack(o[b][4 * e] * inv, o[b][4 * e + 1] * inv),
                  E::pack(o[b][4 * e + 2] * inv, o[b][4 * e + 3] * inv)};
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int n = 0; n < 32 / (64 / CH); ++n) {
      const int r = lane / CH + 64 / CH * n, cc = lane % CH;
      const u32x4 w = *reinterpret_cast<const u32x4*>(ob + k_piece<RB>(r, cc));
      if (r0 + r < n_q)
        *reinterpret_cast<u32x4*>((S*)a.O + (int64_t)(sr.q0 + r0 + r) * a.ldO + (int64_t)h * D +
                                  cc * (16 / (int)sizeof(S))) = w;
    }
  } else {
    if (row >= n_q) return;
    S* op = (S*)a.O + i * a.ldO + (int64_t)h * D + 4 * hf;
#pragma unroll
    for (int b = 0; b < ND; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<f32x4*>(op + 32 * b + 8 * e) =
            f32x4{o[b][4 * e] * inv, o[b][4 * e + 1] * inv, o[b][4 * e + 2] * inv, o[b][4 * e + 3] * inv};
  }
}

// Joins a row's parts in part order; one wavefront per (query, head).
template <class TT, int D>
__global__ __launch_bounds__(256) void k_attn_join(const mf::AttnArgs a, const TileGrid tg, int KT) {
  using S = typename TT::S;
  constexpr int NE = D / 64;
  const int lane = threadIdx.x & 63;
  const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int h = blockIdx.y;
  if (i >= a.N_q) return;
  const int R0 = (int)i / kRows * kRows, off = a.N_k - a.N_q;
  const KeyTiles kt(a.window, a.sinks, off + R0, off + min(R0 + kRows, a.N_q) - 1, KT);
  const int np = max(1, (kt.count + tg.len - 1) / tg.len);
  const int64_t step = (int64_t)a.H * a.N_q, at = (int64_t)h * a.N_q + i;
  // a part a lane for the statistics
  float m = -INFINITY, l = 0.f, acc[NE] = {};
  for (int s = lane; s < np; s += 64) m = fmaxf(m, tg.ml[at + s * step].x);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
  const float mu = m == -INFINITY ? 0.f : m;
  for (int s0 = 0; s0 < np; s0 += 64) {
    const float2 ml = s0 + lane < np ? tg.ml[at + (s0 + lane) * step] : make_float2(-INFINITY, 0.f);
    const float fl = __builtin_amdgcn_exp2f(ml.x - mu);
    l = fmaf(ml.y, fl, l);
    const int n = min(64, np - s0);
#pragma unroll 8
    for (int s = 0; s < n; ++s) {
      const float f = __shfl(fl, s);
#pragma unroll
      for (int c = 0; c < NE; ++c) acc[c] = fmaf(tg.part[(at + (s0 + s) * step) * D + NE * lane + c], f, acc[c]);
    }
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) l += __shfl_xor(l, d);
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

// Few row tiles (at most one workgroup a CU): the keys may be cut into parts of
// one length, equally long whatever the mask makes of the rows.  The length is
// the one that an estimate of the time likes best: rounds of workgroups (one a
// CU, two where tiles leave the matrix cores gaps: 16-bit types) times a part's
// tiles and start, and the parts' way through memory to the join.  Measured on
// d = 128: 1.4 us a tile (two workgroups a CU), fp32 4.3 us; a start is about
// 5 us; 8 heads of 1000 fp32 queries 151 us whole, 44 us in parts.
void split_of(TileGrid& tg, int dt, int H, int N_q, int N_k, int d, int window, int sinks) {
  tg.len = 0;
  tg.nparts = 1;
  tg.total = (N_q + kRows - 1) / kRows;
  const int KT = dt == MF_F32 ? 32 : 64, ntile = tg.total;
  if ((int64_t)H * ntile > 256) return;
  int count[256];
  int longest = 0;
  for (int t = 0; t < ntile; ++t) {
    const int Pa = N_k - N_q + t * kRows, Pb = N_k - N_q + std::min((t + 1) * kRows, N_q) - 1;
    count[t] = KeyTiles(window, sinks, Pa, Pb, KT).count;
    longest = std::max(longest, count[t]);
  }
  const double us = (dt == MF_F32 ? 4.3 : 1.4) * d / 128, start = 5.0;
  const int slots = dt == MF_F32 ? 256 : 512;
  double best = start + us * longest;
  static const int cuts[] = {2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32, 48, 64, 96, 128, 192, 256};
  for (const int k : cuts) {
    const int len = (longest + k - 1) / k;
    if (len < 2) break;
    int64_t parts = 0;
    for (int t = 0; t < ntile; ++t) parts += std::max(1, (count[t] + len - 1) / len);
    const int64_t rounds = (parts * H + slots - 1) / slots;
    const double t = rounds * (start + us * len) + 6.0 + parts * H * (kRows * d * 8 / 4.5e6);
    if (t < best) {
      best = t;
      tg.len = len;
      tg.nparts = (longest + len - 1) / len;
      tg.total = (int)parts;
    }
  }
}

template <class TT, int D>
hipError_t run_tiles(const mf::AttnArgs& a, const TileGrid& tg, hipStream_t st) {
  const int64_t wgs = (int64_t)tg.total * a.H;
  k_attn_tiles<TT, D><<<(unsigned)wgs, kThreads, 0, st>>>(a, tg);
  if (tg.len)
    k_attn_join<TT, D><<<dim3((a.N_q + 3) / 4, a.H), 256, 0, st>>>(a, tg, sizeof(typename TT::S) == 2 ? 64 : 32);
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
hipError_t run(int dt, mf::AttnArgs a, void* ws, size_t ws_bytes, size_t need, hipStream_t st) {
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
  tg.nparts = 1;
  tg.total = tg.ntile;
  if (need > 0 && ws && ws_bytes >= need) {
    split_of(tg, dt, a.H, a.N_q, a.N_k, a.d, a.window, a.sinks);
    tg.part = (float*)ws;
    tg.ml = (float2*)(tg.part + (int64_t)tg.nparts * a.H * a.N_q * a.d);
  }
  return a.d == 64 ? run_tiles<TT, 64>(a, tg, st) : run_tiles<TT, 128>(a, tg, st);
}

}  // namespace

namespace mf {

size_t attention_split_bytes(int dt, int H, int, int N_q, int N_k, int d, int window, int sinks) {
  if (window >= N_k) window = 0;
  TileGrid tg{};
  split_of(tg, dt, H, N_q, N_k, d, window, std::min(sinks, N_k));
  return tg.len ? (size_t)tg.nparts * H * N_q * ((size_t)d * 4 + 8) : 0;
}

hipError_t launch_attention(int dt, const AttnArgs& a, void* ws, size_t ws_bytes, hipStream_t st) {
  const size_t need = a.cu_q || a.N_k == 0
      ? 0 : attention_split_bytes(dt, a.H, a.H_kv, a.N_q, a.N_k, a.d, a.window, a.sinks);
  if (dt == MF_F32) return run<TF32>(dt, a, ws, ws_bytes, need, st);
  if (dt == MF_F16) return run<TF16>(dt, a, ws, ws_bytes, need, st);
  return run<TBF16>(dt, a, ws, ws_bytes, need, st);
}

}  // namespace mf
