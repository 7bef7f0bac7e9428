// Cache eviction by accumulated mass: selection and compaction.
//
// k_evict_select, one workgroup per (sequence, KV head): the budget-th largest
// mass is found digit by digit on order-preserving integer keys (four 8-bit
// histograms, one copy a wavefront), then the kept rows are written in
// ascending order: each wavefront owns a contiguous run of rows, counts its
// rows above the threshold and at it, and after one prefix over the wavefronts
// places its own by ballots.  Rows at the threshold are taken lowest first.
// k_evict_gather copies the kept rows, 16 bytes a lane: every kept row is read
// once and written once.
// The selection is bound by latency (four passes of one workgroup, barriers): 13 us
// for rows of 8192, 33 us for 256 rows of up to 16384; the copy by memory: 32
// sequences cut to 4096 rows of 8 heads, 0.9 GB in 187 us (4.8 TB/s).
#include "mf_attn.h"

#include <algorithm>

namespace {

using namespace mfd;

constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / 64;

// larger mass -> larger key; NaN counts as -infinity, -0 as 0
__device__ __forceinline__ unsigned mass_key(float f) {
  if (f != f) f = -INFINITY;
  f += 0.f;                                     // -0 -> +0
  const unsigned u = __float_as_uint(f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// NR > 0: a thread holds its NR candidates' keys in registers, so that the row
// is read once (rows of up to 1024 NR); NR = 0: every pass reads it again.
template <int NR>
__global__ __launch_bounds__(kSelThreads) void k_evict_select(const mf::EvictArgs a) {
  __shared__ __align__(16) unsigned hist[kSelWaves][256];
  __shared__ __align__(16) unsigned total[256];
  __shared__ unsigned above_w[kSelWaves], tie_w[kSelWaves];
  __shared__ unsigned s_digit, s_left;
  const int sg = blockIdx.x;
  const int s = sg / a.H_kv;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int len = cache_len(a.c, s);
  const int n = min(len, a.budget);
  const float* mass = a.mass + (int64_t)sg * a.ldmass;
  int32_t* kept = a.kept + (int64_t)sg * a.budget;
  float* mo = a.mass_out ? a.mass_out + (int64_t)sg * a.cap_out : nullptr;
  const int c0 = a.sinks, c1 = len - a.recent;  // candidates
  // a wavefront's candidates are one run of rows
  const int seg = NR > 0 ? 64 * NR : (max(c1 - c0, 0) / kSelWaves / 64 + 1) * 64;
  const int w0 = (int)min((int64_t)c0 + (int64_t)wave * seg, (int64_t)max(c1, c0));
  const int w1 = (int)min((int64_t)w0 + seg, (int64_t)max(c1, c0));
  float mass_r[NR > 0 ? NR : 1];
  const bool cut = len > a.budget;
  if constexpr (NR > 0) {
    if (cut) {
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const int j = w0 + 64 * i + lane;
        mass_r[i] = j < w1 ? mass[j] : 0.f;
      }
    }
  }
  if (t == 0 && a.lens_out && sg % a.H_kv == 0) a.lens_out[s] = n;
  for (int64_t r = n + t; r < a.budget; r += kSelThreads) kept[r] = -1;
  if (mo)
    for (int64_t r = n + t; r < a.cap_out; r += kSelThreads) mo[r] = 0.f;
  if (!cut) {
    for (int r = t; r < n; r += kSelThreads) {
      kept[r] = r;
      if (mo) mo[r] = mass[r];
    }
    return;
  }
  // first tokens and last tokens, whatever their mass
  for (int r = t; r < a.sinks; r += kSelThreads) {
    kept[r] = r;
    if (mo) mo[r] = mass[r];
  }
  for (int r = t; r < a.recent; r += kSelThreads) {
    kept[n - a.recent + r] = len - a.recent + r;
    if (mo) mo[n - a.recent + r] = mass[len - a.recent + r];
  }
  unsigned want = n - a.sinks - a.recent;       // < c1 - c0, since len > budget
  if (want == 0) return;
  // f(key, mass, present) for the wavefront's rows, 64 at a time
  auto each = [&](auto&& f) {
    if constexpr (NR > 0) {
#pragma unroll
      for (int i = 0; i < NR; ++i)
        if (w0 + 64 * i < w1) f(w0 + 64 * i + lane, mass_r[i], w0 + 64 * i + lane < w1);
    } else {
      for (int j = w0; j < w1; j += 64) {
        const bool in = j + lane < w1;
        f(j + lane, in ? mass[j + lane] : 0.f, in);
      }
    }
  };

  unsigned prefix = 0;                          // digits found so far
  for (int shift = 24; shift >= 0; shift -= 8) {
    *reinterpret_cast<uint4*>(&hist[0][0] + 4 * t) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    const unsigned hi = shift == 24 ? 0u : ~0u << (shift + 8);
    each([&](int, float m, bool in) {
      const unsigned k = mass_key(m);
      if (in && (k & hi) == prefix) atomicAdd(&hist[wave][(k >> shift) & 255], 1u);
    });
    __syncthreads();
    if (t < 256) {
      unsigned v = 0;
#pragma unroll
      for (int w = 0; w < kSelWaves; ++w) v += hist[w][t];
      total[t] = v;
    }
    __syncthreads();
    if (wave == 0) {
      // lane l holds digits 4l..4l+3; `over` counts the keys of higher lanes
      const uint4 v = *reinterpret_cast<const uint4*>(total + 4 * lane);
      const unsigned mine = v.x + v.y + v.z + v.w;
      unsigned incl = mine;                     // keys of this lane and higher ones
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const unsigned u = __shfl_down(incl, o);
        incl += lane + o < 64 ? u : 0u;
      }
      const unsigned over = incl - mine;
      if (over < want && want <= incl) {        // exactly one lane
        unsigned left = want - over;
        int dgt = 3;
        const unsigned c[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 3; i > 0; --i)
          if (dgt == i && c[i] < left) { left -= c[i]; dgt = i - 1; }
        s_digit = 4 * lane + dgt;
        s_left = left;
      }
    }
    __syncthreads();
    prefix |= s_digit << shift;
    want = s_left;                              // still to take among this prefix
  }
  // keys above `prefix` are kept, and the first `want` rows equal to it
  unsigned na = 0, nt = 0;
  each([&](int, float m, bool in) {
    const unsigned k = mass_key(m);
    na += __popcll(__ballot(in && k > prefix));
    nt += __popcll(__ballot(in && k == prefix));
  });
  if (lane == 0) { above_w[wave] = na; tie_w[wave] = nt; }
  __syncthreads();
  unsigned ties = 0, out = a.sinks;
  for (int w = 0; w < wave; ++w) {
    out += above_w[w] + (min(ties + tie_w[w], want) - min(ties, want));
    ties += tie_w[w];
  }
  const uint64_t below = (1ull << lane) - 1;
  each([&](int j, float m, bool in) {
    const unsigned k = mass_key(m);
    const uint64_t bt = __ballot(in && k == prefix);
    const bool keep = in && (k > prefix || (k == prefix && ties + __popcll(bt & below) < want));
    const uint64_t bk = __ballot(keep);
    if (keep) {
      const unsigned o = out + __popcll(bk & below);
      kept[o] = j;
      if (mo) mo[o] = m;
    }
    out += __popcll(bk);
    ties += __popcll(bt);
  });
}

// one workgroup per (sequence, KV head, row chunk); a lane moves 16 bytes of K and of V
template <int kRowBytes>
__global__ __launch_bounds__(256) void k_evict_gather(const mf::EvictArgs a, int es, int chunks) {
  constexpr int LPR = kRowBytes / 16;
  constexpr int RPB = 256 / LPR;
  const int sg = blockIdx.x / chunks;
  const int s = sg / a.H_kv, g = sg - s * a.H_kv;
  const int n = min(cache_len(a.c, s), a.budget);
  const int r = (blockIdx.x - sg * chunks) * RPB + threadIdx.x / LPR;
  const int b = 16 * (threadIdx.x % LPR);
  if (r >= n) return;
  const int j = a.kept[(int64_t)sg * a.budget + r];
  const int64_t src = cache_row(a.c, s, j, g, a.H_kv, a.d);
  const int64_t dst = ((int64_t)sg * a.cap_out + r) * kRowBytes + b;
  uint4 k = make_uint4(0, 0, 0, 0), v = k;
  if (src >= 0) {
    k = *reinterpret_cast<const uint4*>((const char*)a.c.K + src * es + b);
    v = *reinterpret_cast<const uint4*>((const char*)a.c.V + src * es + b);
  }
  *reinterpret_cast<uint4*>((char*)a.K_out + dst) = k;
  *reinterpret_cast<uint4*>((char*)a.V_out + dst) = v;
}

template <int RB>
void gather(const mf::EvictArgs& a, int es, int rows, hipStream_t st) {
  constexpr int RPB = 256 / (RB / 16);
  const int chunks = (rows + RPB - 1) / RPB;
  k_evict_gather<RB><<<(unsigned)a.S * a.H_kv * chunks, 256, 0, st>>>(a, es, chunks);
}

}  // namespace

namespace mf {

hipError_t launch_evict(int dt, const EvictArgs& a, hipStream_t st) {
  const int rows_sg = a.S * a.H_kv;
  if (a.c.max_len <= 8 * kSelThreads) k_evict_select<8><<<rows_sg, kSelThreads, 0, st>>>(a);
  else if (a.c.max_len <= 32 * kSelThreads) k_evict_select<32><<<rows_sg, kSelThreads, 0, st>>>(a);
  else k_evict_select<0><<<rows_sg, kSelThreads, 0, st>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int es = dtype_bytes(dt), rows = std::min(a.budget, a.c.max_len);
  if (rows == 0) return hipSuccess;
  switch (a.d * es) {
    case 128: gather<128>(a, es, rows, st); break;
    case 256: gather<256>(a, es, rows, st); break;
    default: gather<512>(a, es, rows, st); break;
  }
  return hipGetLastError();
}

}  // namespace mf
