// Attention of one query per sequence over a paged cache, optionally with the
// accumulated weight of every cached row.
//
// Bound by memory: the visible K and V rows are read once and each element
// serves a group's G heads only.  k_decode_parts: a workgroup takes one part
// (P tiles of 32 keys) of one (sequence, KV head); its four wavefronts walk the
// part's tiles in turn, each on its own, and are joined once at the end.  The
// group's heads, padded to 16, are the columns of 16x16 matrix instructions:
//   S^T = K Q^T:   A = 16 K rows, straight from global memory in 16-byte pieces
//   O^T = V^T P^T: A = V columns by the transposing LDS read, B = P
// so a lane owns one head, and the keys of its scores are the keys of its
// operand of the second product.  The next tile's K and V (16 KB a wavefront)
// are in flight in registers while a tile is computed: with two workgroups a CU
// 128 KB, more than bandwidth times latency.  V goes to LDS in the wavefront's
// own 8 KB, masked rows as zeros.
// Parts have one length for all sequences of a call, so a batch of ragged
// lengths keeps every workgroup equally long.  k_decode_join adds the parts in
// part order, and, for the accumulated weights, turns the scores that the parts
// left in the workspace into exp2(score - lse).
// Measured (d = 128, 8 KV heads, 32 heads): 32 sequences of 8192 rows, fp16, 185 us
// (5.8 TB/s of K and V); one of 32768, bf16, 28 us (4.8 TB/s); 64 ragged ones up to
// 8192 under a window of 4096 with weights 192 us, 139 us without: storing the
// scores (25 MB) costs 30 us in every form tried (behind a branch or not, a step
// late, non-temporal, a tile's heads together or apart), their join 18 us.
#include "mf_attn.h"

#include <algorithm>

namespace {

using namespace mfd;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kUnit = 32;                       // keys that part lengths count in

template <class TT> struct Elem;
template <> struct Elem<TBF16> {
  static __device__ __forceinline__ f32x4 mfma(const u32x4& a, const u32x4& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ unsigned pack(float x, float y) {
    return __builtin_bit_cast(unsigned, __builtin_convertvector((f32x2{x, y}), bf16x2));
  }
};
template <> struct Elem<TF16> {
  static __device__ __forceinline__ f32x4 mfma(const u32x4& a, const u32x4& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ unsigned pack(float x, float y) {
    return __builtin_bit_cast(unsigned, __builtin_convertvector((f32x2{x, y}), f16x2));
  }
};
template <> struct Elem<TF32> {};

struct PartGrid {
  int nparts;                                   // parts of the longest sequence
  int units;                                    // units per part
  int slots;                                    // score entries per (sequence, head)
  float* part;                                  // [S][nparts][H][D]
  float2* ml;                                   // [S][nparts][H] (max, sum), log2 units
  // [S][16 heads of a group][tiles][heads][keys of a tile], log2 units, the last
  // unit spare; a tile's heads lie together, so that it leaves in one run
  float* score;
};

// The visible tiles of a sequence, tiles of KT keys: the sinks' tiles
// 0..nS-1, then tiles tw0.. up to its end.
struct Tiles {
  int n, w0, nS, tw0, count;
  __device__ __forceinline__ Tiles(const mf::DecodeArgs& a, int len, int KT) {
    n = len;
    w0 = a.window > 0 ? max(0, n - a.window) : 0;
    nS = a.window > 0 ? (min(a.sinks, n) + KT - 1) / KT : 0;
    tw0 = max(w0 / KT, nS);
    count = nS + max(0, (n + KT - 1) / KT - tw0);
  }
  __device__ __forceinline__ int key0(int it, int KT) const { return (it < nS ? it : tw0 + it - nS) * KT; }
};

// Byte offset of 16-byte piece c of row r in a wavefront's V tile: eight rows
// (fp32: every fourth of 16) of one piece column spread over all banks.
template <int ES, int RB>
__device__ __forceinline__ int v_piece(int r, int c) {
  if constexpr (ES == 4) return r * RB + 16 * (c ^ (4 * ((r >> 2) & 3)));
  else if constexpr (RB == 128) return r * RB + 16 * (c ^ (2 * ((r >> 1) & 3)));
  else return r * RB + 16 * (c ^ (2 * (r & 7)));
}

__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// kWhole: a tile never straddles pages (page is a multiple of the tile).
// kMass: the scores stay in the workspace for the weights.
template <class TT, int D, bool kWhole, bool kMass>
__global__ __launch_bounds__(kThreads, 2) void k_decode_parts(const mf::DecodeArgs a, const PartGrid pg) {
  using S = typename TT::S;
  constexpr bool k16 = sizeof(S) == 2;
  constexpr int ES = sizeof(S);
  constexpr int KT = k16 ? 32 : 16;             // keys per tile
  constexpr int NT = KT / 16;                   // 16-key score blocks
  constexpr int RB = D * ES;
  constexpr int CH = RB / 16;
  constexpr int NK = RB / 64;                   // pieces per lane and K row
  constexpr int NV = KT * CH / 64;              // V pieces per lane
  constexpr int VR = 64 / CH;                   // rows between them
  constexpr int NB = D / 16;                    // 16-dim output blocks
  constexpr int kTile = KT * RB;
  constexpr int kWaveLds = kTile;               // also holds the wavefront's O: 16 heads of fp32
  static_assert(kTile >= 16 * D * 4, "a tile's LDS must hold the joined output");
  __shared__ __align__(16) unsigned char smem[kWaves * kWaveLds];
  __shared__ float2 sml[kWaves][16];

  const int lane = threadIdx.x & 63, col = lane & 15, grp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = a.H / a.H_kv;
  const int gtiles = (G + 15) / 16;
  const int s = blockIdx.x, g = blockIdx.y / gtiles, h0 = g * G + 16 * (blockIdx.y % gtiles);
  const int nh = min(16, (g + 1) * G - h0);     // heads of this workgroup
  const int part = blockIdx.z;
  const Tiles tl(a, a.c.n_pages > 0 ? cache_len(a.c, s) : 0, KT);
  const int per = pg.units * (kUnit / KT);
  const int t0 = part * per, t1 = min(t0 + per, tl.count);
  // a sequence of no visible key still owns part 0
  if (part > 0 && t0 >= tl.count) return;

  const int h = h0 + min(col, nh - 1);
  const float sc = a.scale[h] * kLog2E;
  const float c = fmaxf(fabsf(sc), 1e-45f);
  u32x4 q[NK];
  {
    const S* qp = (const S*)a.Q + (int64_t)s * a.ldQ + (int64_t)h * D + grp * (16 / ES);
    const unsigned flip = sc < 0.f ? (k16 ? 0x80008000u : 0x80000000u) : 0u;
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      S e[16 / ES];
#pragma unroll
      for (int j = 0; j < 16 / ES; ++j) e[j] = qp[i * (64 / ES) + j];
      __builtin_memcpy(&q[i], e, 16);
      q[i] ^= flip;
    }
  }

  struct KTile { u32x4 k[NT][NK]; unsigned vm; };
  u32x4 v[NV];
  const char* Kp = (const char*)a.c.K;
  const char* Vp = (const char*)a.c.V;
  constexpr unsigned kAll = KT == 32 ? 0xffffffffu : 0xffffu;
  // Pool page of a tile (kWhole), fetched a step before the tile's rows.  The
  // table is constant during the call: a scalar load, which waits for no store.
  auto page_of = [&](int it) -> int64_t {
    if (!kWhole || it >= t1) return -1;
    const int64_t slot = (int64_t)s * a.c.max_pages + tl.key0(it, KT) / a.c.page;
    return a.c.table ? (int64_t)((__attribute__((address_space(4))) const int32_t*)(uintptr_t)a.c.table)[slot] : slot;
  };
  auto load = [&](int it, int64_t page, KTile& t) {
    const int j0 = tl.key0(it, KT);
    const int lj = j0 + (lane & (KT - 1));      // the key this lane answers for
    bool vis = lj < tl.n && (lj >= tl.w0 || lj < a.sinks);
    if constexpr (kWhole) {
      const bool there = page >= 0 && page < a.c.n_pages;
      vis = vis && there;
      t.vm = (unsigned)__ballot(vis) & kAll;
      const int64_t b = there ? ((page * a.H_kv + g) * a.c.page + j0 % a.c.page) * (int64_t)(D * ES) : 0;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < NK; ++i)
          t.k[nt][i] = *reinterpret_cast<const u32x4*>(Kp + b + (16 * nt + col) * RB + 64 * i + 16 * grp);
#pragma unroll
      for (int n = 0; n < NV; ++n)
        v[n] = *reinterpret_cast<const u32x4*>(Vp + b + 16 * lane + n * 1024);
    } else {
      int64_t r = vis ? cache_row(a.c, s, lj, g, a.H_kv, D) : -1;
      vis = r >= 0;
      t.vm = (unsigned)__ballot(vis) & kAll;
      r = vis ? r * ES : 0;                     // masked keys read the pool's first row
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int64_t b = __shfl(r, 16 * nt + col);
#pragma unroll
        for (int i = 0; i < NK; ++i)
          t.k[nt][i] = *reinterpret_cast<const u32x4*>(Kp + b + 64 * i + 16 * grp);
      }
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int64_t b = __shfl(r, lane / CH + VR * n);
        v[n] = *reinterpret_cast<const u32x4*>(Vp + b + 16 * (lane % CH));
      }
    }
  };

  unsigned char* vb = smem + wave * kWaveLds;
  f32x4 o[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) o[b] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;
  float* score = kMass ? pg.score + ((int64_t)s * a.H + h0) * pg.slots : nullptr;

  int64_t page = page_of(t0 + wave);
  auto step = [&](int it, KTile& cur, KTile& nxt) {
    const unsigned vm = __builtin_amdgcn_readfirstlane(cur.vm);
    wave_order();                               // the last tile's reads are done
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int r = lane / CH + VR * n;
      u32x4 w = v[n];
      if (vm != kAll && !((vm >> r) & 1)) w = u32x4{0, 0, 0, 0};
      *reinterpret_cast<u32x4*>(vb + v_piece<ES, RB>(r, lane % CH)) = w;
    }
    wave_order();
    if (it + kWaves < t1) load(it + kWaves, page, nxt);
    page = page_of(it + 2 * kWaves);
    f32x4 x[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      x[nt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        if constexpr (k16) {
          x[nt] = Elem<TT>::mfma(cur.k[nt][i], q[i], x[nt]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            x[nt] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(cur.k[nt][i][j]),
                                                         __uint_as_float(q[i][j]), x[nt], 0, 0, 0);
        }
      }
    }
    float mx = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (vm != kAll && !((vm >> (16 * nt + 4 * grp + i)) & 1)) x[nt][i] = -INFINITY;
        x[nt][i] *= c;
        mx = fmaxf(mx, x[nt][i]);
      }
    if constexpr (kMass) {
      // Every lane stores, those of the padding heads to a spare place: no
      // branch between the stores and the waits for older loads.
      float* to = score + (int64_t)(col < nh ? it * KT : pg.slots - kUnit) * nh +
                  (col < nh ? col : 0) * KT + 4 * grp;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) *reinterpret_cast<f32x4*>(to + 16 * nt) = x[nt];
    }
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    if (__any(mx > m)) {
      const float mn = fmaxf(m, mx);
      const float f = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - mn);
      l *= f;
#pragma unroll
      for (int b = 0; b < NB; ++b) o[b] *= f;
      m = mn;
    }
    const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[nt][i] = __builtin_amdgcn_exp2f(x[nt][i] - mu);
        l += x[nt][i];
      }
    if constexpr (k16) {
      u32x4 p;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        p[2 * nt] = Elem<TT>::pack(x[nt][0], x[nt][1]);
        p[2 * nt + 1] = Elem<TT>::pack(x[nt][2], x[nt][3]);
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        u32x4 vv;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          // lane (i of 16) addresses row i / 4, dims 4 (i % 4).. and receives
          // dim i of the four rows
          const int r = 16 * nt + 4 * grp + (col >> 2);
          const unsigned char* ad = vb + v_piece<ES, RB>(r, 2 * b + ((col & 3) >> 1)) + 8 * (col & 1);
          const u32x2 w = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (__attribute__((address_space(3))) s16x4*)(ad)));
          vv[2 * nt] = w[0];
          vv[2 * nt + 1] = w[1];
        }
        o[b] = Elem<TT>::mfma(vv, p, o[b]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const float w = *reinterpret_cast<const float*>(
              vb + v_piece<ES, RB>(4 * grp + i, 4 * b + (col >> 2)) + 4 * (col & 3));
          o[b] = __builtin_amdgcn_mfma_f32_16x16x4f32(w, x[0][i], o[b], 0, 0, 0);
        }
    }
  };

  KTile ka, kb;
  int it = t0 + wave;
  if (it < t1) load(it, page, ka);
  page = page_of(it + kWaves);
  while (it < t1) {
    step(it, ka, kb);
    it += kWaves;
    if (it >= t1) break;
    step(it, kb, ka);
    it += kWaves;
  }

  // join the wavefronts: O as [head][dim] in each one's LDS
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  wave_order();
  if (grp == 0) sml[wave][col] = make_float2(m, l);
#pragma unroll
  for (int b = 0; b < NB; ++b)
    *reinterpret_cast<f32x4*>(vb + (col * D + 16 * b + 4 * grp) * 4) = o[b];
  __syncthreads();
  for (int e = threadIdx.x; e < nh * D; e += kThreads) {
    const int hh = e / D, dim = e - hh * D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) M = fmaxf(M, sml[w][hh].x);
    const float mu = M == -INFINITY ? 0.f : M;
    float L = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float2 t = sml[w][hh];
      const float f = __builtin_amdgcn_exp2f(t.x - mu);
      L = fmaf(t.y, f, L);
      acc = fmaf(*reinterpret_cast<const float*>(smem + w * kWaveLds + e * 4), f, acc);
    }
    if (pg.part) {
      const int64_t at = ((int64_t)s * pg.nparts + part) * a.H + h0 + hh;
      pg.part[at * D + dim] = acc;
      if (dim == 0) pg.ml[at] = make_float2(M, L);
    } else {
      const float inv = L == 0.f ? 0.f : 1.f / L;
      ((S*)a.O)[(int64_t)s * a.ldO + (int64_t)(h0 + hh) * D + dim] = TT::fromf(acc * inv);
      if (a.lse && dim == 0)
        a.lse[(int64_t)s * a.H + h0 + hh] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2f;
    }
  }
}

constexpr int kMassKeys = 1024;                 // keys per workgroup of the weights
constexpr int kMaxParts = 1024;

// grid (S * (G + key chunks), H_kv): the first G workgroups of a (sequence, KV
// head) join the parts of one head each, the others add the weights of
// kMassKeys rows each.  A head's (max, sum) pairs are read one a thread and
// become factors in LDS; then each wavefront adds every fourth part, and the
// four sums are added in order.
template <class TT, int D>
__global__ __launch_bounds__(kThreads) void k_decode_join(const mf::DecodeArgs a, const PartGrid pg, int KT,
                                                          int chunks) {
  using S = typename TT::S;
  constexpr int NE = D / 64;
  __shared__ float fac[kMaxParts];
  __shared__ float acc4[kWaves][D];
  __shared__ float red[kWaves];
  __shared__ float lse2[64];
  const int G = a.H / a.H_kv, g = blockIdx.y;
  const int s = blockIdx.x / (G + chunks), chunk = blockIdx.x - s * (G + chunks);
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int len = cache_len(a.c, s);
  const Tiles tl(a, a.c.n_pages > 0 ? len : 0, KT);
  const int per = pg.units * (kUnit / KT);
  const int np = max(1, (tl.count + per - 1) / per);
  const int64_t at0 = (int64_t)s * pg.nparts * a.H + (int64_t)g * G;
  auto all_max = [&](float x) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor(x, o));
    return x;
  };
  auto all_sum = [&](float x) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
    return x;
  };
  if (chunk < G) {
    const int64_t at = at0 + chunk;
    float M = -INFINITY;
    for (int p = t; p < np; p += kThreads) {
      fac[p] = pg.ml[at + (int64_t)p * a.H].x;
      M = fmaxf(M, fac[p]);
    }
    M = all_max(M);
    if (lane == 0) red[wave] = M;
    __syncthreads();
    M = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float mu = M == -INFINITY ? 0.f : M;
    float L = 0.f;
    for (int p = t; p < np; p += kThreads) {
      const float f = __builtin_amdgcn_exp2f(fac[p] - mu);
      L = fmaf(pg.ml[at + (int64_t)p * a.H].y, f, L);
      fac[p] = f;
    }
    L = all_sum(L);
    __syncthreads();
    if (lane == 0) red[wave] = L;
    float acc[NE] = {};
#pragma unroll 4
    for (int p = wave; p < np; p += kWaves) {
      const float* src = pg.part + (at + (int64_t)p * a.H) * D + NE * lane;
      const float f = fac[p];
#pragma unroll
      for (int c = 0; c < NE; ++c) acc[c] = fmaf(src[c], f, acc[c]);
    }
#pragma unroll
    for (int c = 0; c < NE; ++c) acc4[wave][NE * lane + c] = acc[c];
    __syncthreads();
    L = ((red[0] + red[1]) + red[2]) + red[3];
    const int64_t h = (int64_t)g * G + chunk;
    if (t < D) {
      const float v = ((acc4[0][t] + acc4[1][t]) + acc4[2][t]) + acc4[3][t];
      ((S*)a.O)[(int64_t)s * a.ldO + h * D + t] = TT::fromf(L == 0.f ? 0.f : v / L);
    }
    if (t == 0 && a.lse) a.lse[(int64_t)s * a.H + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2f;
    return;
  }
  const int j0 = (chunk - G) * kMassKeys;
  if (j0 >= len) return;
  // four consecutive rows a thread: tiles hold a multiple of four.  The first
  // heads' scores are in flight while the log-sum-exps are formed.
  const int j = j0 + 4 * t;
  const int tile = j / KT;
  const int it = tile < tl.nS ? tile : tile - tl.tw0 + tl.nS;
  const bool listed = j < tl.n && (tile < tl.nS || tile >= tl.tw0);
  const float* score = pg.score + ((int64_t)s * a.H + (int64_t)g * G) * pg.slots + (listed ? j - tile * KT : 0);
  auto scores_of = [&](int hh) {
    const int h0 = hh & ~15, nh = min(16, G - h0);
    return *reinterpret_cast<const f32x4*>(score + (int64_t)h0 * pg.slots + (int64_t)(listed ? it * KT : 0) * nh +
                                           (hh - h0) * KT);
  };
  constexpr int NH = 4;
  f32x4 x[NH];
#pragma unroll
  for (int i = 0; i < NH; ++i) x[i] = scores_of(min(i, G - 1));
  const int64_t mrow = ((int64_t)s * a.H_kv + g) * a.ldmass + j;
  float w[4] = {};
  if (a.mass_in) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = j + i < len ? a.mass_in[mrow + i] : 0.f;
  }
  for (int hh = wave; hh < G; hh += kWaves) {
    float M = -INFINITY, L = 0.f;
    for (int p = lane; p < np; p += 64) M = fmaxf(M, pg.ml[at0 + (int64_t)p * a.H + hh].x);
    M = all_max(M);
    const float mu = M == -INFINITY ? 0.f : M;
    for (int p = lane; p < np; p += 64) {
      const float2 y = pg.ml[at0 + (int64_t)p * a.H + hh];
      L = fmaf(y.y, __builtin_amdgcn_exp2f(y.x - mu), L);
    }
    L = all_sum(L);
    // +infinity: no key of this head is visible, every weight is 0
    if (lane == 0) lse2[hh] = L == 0.f ? INFINITY : M + log2f(L);
  }
  __syncthreads();
  float sum[4] = {};
  for (int h0 = 0; h0 < G; h0 += NH) {
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      if (h0 + i >= G) break;
      const float L = lse2[h0 + i];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        sum[e] += x[i][e] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(x[i][e] - L);
    }
#pragma unroll
    for (int i = 0; i < NH; ++i)
      if (h0 + NH < G) x[i] = scores_of(min(h0 + NH + i, G - 1));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (j + i < len) {
      const int ji = j + i;
      const bool vis = listed && ji < tl.n && (ji >= tl.w0 || ji < a.sinks);
      a.mass_out[mrow + i] = w[i] + (vis ? sum[i] : 0.f);
    }
}

// 32-key units that the longest sequence can see
int64_t max_units(int max_len, int window, int sinks) {
  const int64_t all = ((int64_t)max_len + kUnit - 1) / kUnit;
  if (window == 0) return all;
  // a window's ends lie inside two tiles
  return std::min<int64_t>(all, ((int64_t)std::min(sinks, max_len) + kUnit - 1) / kUnit + window / kUnit + 2);
}

// Part length: enough parts for the two workgroups a CU that run at a time, each
// of at least two tiles a wavefront.  (Twice as many: 64 sequences of 512 rows 29
// instead of 23 us; four times: 64 ragged ones 158 instead of 141 us.)
PartGrid part_grid(int S, int max_len, int H, int H_kv, int window, int sinks) {
  PartGrid pg{};
  const int64_t u = std::max<int64_t>(1, max_units(max_len, window, sinks));
  const int64_t rows = (int64_t)S * H_kv * ((H / H_kv + 15) / 16);
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>((512 + rows - 1) / rows, u / (2 * kWaves)));
  pg.units = (int)((u + want - 1) / want);
  pg.nparts = (int)((u + pg.units - 1) / pg.units);
  pg.slots = (int)((u + 1) * kUnit);
  return pg;
}

template <class TT, int D>
hipError_t run(const mf::DecodeArgs& a, void* ws, hipStream_t st) {
  constexpr int KT = sizeof(typename TT::S) == 2 ? 32 : 16;
  PartGrid pg = part_grid(a.S, a.c.max_len, a.H, a.H_kv, a.window, a.sinks);
  const bool join = pg.nparts > 1 || a.mass_out;
  if (join) {
    pg.part = (float*)ws;
    pg.ml = (float2*)(pg.part + (int64_t)a.S * pg.nparts * a.H * D);
    if (a.mass_out) pg.score = (float*)(pg.ml + (((int64_t)a.S * pg.nparts * a.H + 1) & ~int64_t(1)));
  }
  const dim3 grid(a.S, a.H_kv * ((a.H / a.H_kv + 15) / 16), pg.nparts);
  if (a.c.page % KT == 0) {
    if (a.mass_out) k_decode_parts<TT, D, true, true><<<grid, kThreads, 0, st>>>(a, pg);
    else k_decode_parts<TT, D, true, false><<<grid, kThreads, 0, st>>>(a, pg);
  } else {
    if (a.mass_out) k_decode_parts<TT, D, false, true><<<grid, kThreads, 0, st>>>(a, pg);
    else k_decode_parts<TT, D, false, false><<<grid, kThreads, 0, st>>>(a, pg);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !join) return e;
  const int chunks = a.mass_out ? (a.c.max_len + kMassKeys - 1) / kMassKeys : 0;
  k_decode_join<TT, D><<<dim3(a.S * (a.H / a.H_kv + chunks), a.H_kv), kThreads, 0, st>>>(a, pg, KT, chunks);
  return hipGetLastError();
}

template <class TT>
hipError_t run_d(mf::DecodeArgs a, void* ws, hipStream_t st) {
  if (a.window >= a.c.max_len) a.window = 0;    // reaches every row
  a.sinks = std::min(a.sinks, a.c.max_len);
  return a.d == 64 ? run<TT, 64>(a, ws, st) : run<TT, 128>(a, ws, st);
}

}  // namespace

namespace mf {

size_t decode_workspace_bytes(int S, int max_len, int H, int H_kv, int d, int window, int sinks,
                              bool with_mass) {
  if (window >= max_len) window = 0;
  const PartGrid pg = part_grid(S, max_len, H, H_kv, window, std::min(sinks, max_len));
  if (pg.nparts == 1 && !with_mass) return 0;
  const size_t parts = (size_t)S * pg.nparts * H;
  return parts * d * 4 + ((parts + 1) & ~size_t(1)) * 8 + (with_mass ? (size_t)S * H * pg.slots * 4 : 0);
}

hipError_t launch_decode(int dt, const DecodeArgs& a, void* ws, hipStream_t st) {
  if (dt == MF_F32) return run_d<TF32>(a, ws, st);
  if (dt == MF_F16) return run_d<TF16>(a, ws, st);
  return run_d<TBF16>(a, ws, st);
}

}  // namespace mf
