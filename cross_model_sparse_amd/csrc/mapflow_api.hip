// C boundary of libmapflow: argument validation, status codes and error text.
// Every entry point checks its arguments on the host before touching the GPU.
#include <math.h>
#include <stdio.h>
#include <string.h>

#include <mutex>
#include <string>

#include "mf_attn.h"

// Fixed scratch of mf_topp_select_bsr_noalloc: the selection's kept[T][T] and
// count[T] int32 arrays for up to kNoAllocMaxT block rows.  Each GPU the
// library runs on holds its own copy for the life of the process.  Host code
// never uses this name as an address: the per-device address comes from
// hipGetSymbolAddress (noalloc_scratch below).
namespace {
constexpr int kNoAllocMaxT = 1024;
constexpr size_t kNoAllocScratchBytes = ((size_t)kNoAllocMaxT * kNoAllocMaxT + kNoAllocMaxT) * 4;
}  // namespace
static __device__ __align__(256) unsigned char scratch[kNoAllocScratchBytes];

namespace mf {

namespace {
thread_local std::string g_last_error;
}

int fail(int st, const std::string& msg) {
  g_last_error = msg;
  return st;
}

int hip_check(hipError_t e, const char* what) {
  if (e == hipSuccess) return MF_OK;
  return fail(MF_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
}

int row_vec_bytes(const void* base, int N, int B, int esize) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(base);
  for (int v = 16; v > esize; v >>= 1) {
    if ((a % v) == 0 && ((int64_t)N * esize) % v == 0 && ((int64_t)B * esize) % v == 0)
      return v;
  }
  return esize;
}

bool ragged_rows_ok(const void* base, int N, int esize) {
  return (reinterpret_cast<uintptr_t>(base) % esize) == 0 && (int64_t)N * esize >= 16;
}

}  // namespace mf

namespace {

bool valid_dtype(int dt) { return dt == MF_F32 || dt == MF_F16 || dt == MF_BF16; }
bool valid_block(int B) { return B == 16 || B == 32 || B == 64 || B == 128; }

std::string fmt(const char* f, long long a, long long b = 0) {
  char buf[256];
  snprintf(buf, sizeof buf, f, a, b);
  return buf;
}

// Shared checks of the map geometry; returns MF_OK or records the error.
int check_geom(const char* fn, int dtype, int H_s, int N, int B) {
  using mf::fail;
  std::string f = std::string(fn) + ": ";
  if (!valid_dtype(dtype)) return fail(MF_ERR_INVALID, f + fmt("unknown dtype code %lld", dtype));
  if (N < 1) return fail(MF_ERR_INVALID, f + fmt("N must be >= 1 (got %lld)", N));
  if (!valid_block(B)) return fail(MF_ERR_INVALID, f + fmt("B must be 16, 32, 64 or 128 (got %lld)", B));
  if (H_s < 1 || H_s > 64) return fail(MF_ERR_INVALID, f + fmt("H_s must be in [1, 64] (got %lld)", H_s));
  return MF_OK;
}

}  // namespace

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_dev[kMaxDevices] = {};

// Device address of `scratch` on the calling thread's current device, looked
// up once per device and cached.
int noalloc_scratch(const char* fn, void** out) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return mf::hip_check(e, fn);
  if (dev < 0 || dev >= kMaxDevices)
    return mf::fail(MF_ERR_UNSUPPORTED, std::string(fn) + fmt(": device index %lld >= 64", dev));
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (g_scratch_dev[dev] == nullptr) {
    void* ptr = nullptr;
    e = hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch));
    if (e != hipSuccess || ptr == nullptr)
      return mf::hip_check(e != hipSuccess ? e : hipErrorInvalidSymbol,
                           (std::string(fn) + " scratch address").c_str());
    g_scratch_dev[dev] = ptr;
  }
  *out = g_scratch_dev[dev];
  return MF_OK;
}

}  // namespace

extern "C" {

int mf_abi_version(void) { return MF_ABI_VERSION; }

const char* mf_status_string(int status) {
  switch (status) {
    case MF_OK: return "MF_OK";
    case MF_ERR_INVALID: return "MF_ERR_INVALID: invalid argument";
    case MF_ERR_UNSUPPORTED: return "MF_ERR_UNSUPPORTED: valid arguments, combination not built";
    case MF_ERR_CAPACITY: return "MF_ERR_CAPACITY: BSR larger than the given capacity";
    case MF_ERR_HIP: return "MF_ERR_HIP: HIP runtime error";
    default: return "unknown mapflow status";
  }
}

const char* mf_last_error(void) { return mf::g_last_error.c_str(); }

size_t mf_block_mass_ws_bytes(int H_s, int N, int B) {
  if (H_s < 1 || N < 1 || B < 1) return 0;
  return mf::block_mass_rows_workspace_bytes(H_s, N, B);
}

int mf_block_mass_ws(const void* A, int dtype, int H_s, int N, int B, float* mass,
                     void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "mf_block_mass_ws";
  int st = check_geom(fn, dtype, H_s, N, B);
  if (st != MF_OK) return st;
  if (!A || !mass || !workspace) return mf::fail(MF_ERR_INVALID, std::string(fn) + ": null pointer");
  const size_t need = mf::block_mass_rows_workspace_bytes(H_s, N, B);
  if (workspace_bytes < need)
    return mf::fail(MF_ERR_INVALID, std::string(fn) + fmt(": workspace of %lld bytes < %lld required",
                                                          (long long)workspace_bytes, (long long)need));
  return mf::hip_check(mf::launch_block_mass_rows(A, dtype, H_s, N, B, mass, workspace,
                                                  (hipStream_t)stream),
                       "mf_block_mass_ws launch");
}

int mf_block_mass(const void* A, int dtype, int H_s, int N, int B, float* mass,
                  void* stream) {
  int st = check_geom("mf_block_mass", dtype, H_s, N, B);
  if (st != MF_OK) return st;
  if (!A || !mass) return mf::fail(MF_ERR_INVALID, "mf_block_mass: null pointer");
  return mf::hip_check(
      mf::launch_block_mass(A, dtype, H_s, N, B, mass, (hipStream_t)stream),
      "mf_block_mass launch");
}

size_t mf_topp_workspace_bytes(int N, int B) {
  if (N < 1 || B < 1) return 0;
  const size_t T = (size_t)mf::blocks_of(N, B);
  const size_t bytes = (T * T + T) * sizeof(int32_t);
  return (bytes + 255) & ~(size_t)255;
}

int mf_topp_select_bsr(const float* mass, const void* A, int dtype, int H_s,
                       int N, int B, float p, int32_t* row_ptr,
                       int32_t* col_idx, void* vals, int64_t cap_nnzb,
                       int64_t* nnzb_out, void* workspace,
                       size_t workspace_bytes, void* stream) {
  const char* fn = "mf_topp_select_bsr";
  int st = check_geom(fn, dtype, H_s, N, B);
  if (st != MF_OK) return st;
  if (!mass || !A || !row_ptr || !workspace)
    return mf::fail(MF_ERR_INVALID, std::string(fn) + ": null pointer");
  if (cap_nnzb < 0) return mf::fail(MF_ERR_INVALID, std::string(fn) + ": cap_nnzb < 0");
  if (cap_nnzb > 0 && (!col_idx || !vals))
    return mf::fail(MF_ERR_INVALID, std::string(fn) + ": null col_idx/vals with cap_nnzb > 0");
  if (!(p > 0.0f && p <= 1.0f))  // also rejects NaN
    return mf::fail(MF_ERR_INVALID, std::string(fn) + ": p must be in (0, 1]");
  const int T = mf::blocks_of(N, B);
  if (T > 4096)
    return mf::fail(MF_ERR_UNSUPPORTED, std::string(fn) + fmt(": T = %lld block rows > 4096", T));
  if (workspace_bytes < mf_topp_workspace_bytes(N, B))
    return mf::fail(MF_ERR_INVALID, std::string(fn) + fmt(": workspace of %lld bytes < %lld required",
                                                          (long long)workspace_bytes,
                                                          (long long)mf_topp_workspace_bytes(N, B)));
  hipStream_t s = (hipStream_t)stream;
  st = mf::hip_check(mf::launch_topp_bsr(mass, A, dtype, H_s, N, B, p, row_ptr,
                                         col_idx, vals, cap_nnzb, workspace, s),
                     "mf_topp_select_bsr launch");
  if (st != MF_OK || !nnzb_out) return st;
  int32_t nnzb = 0;
  st = mf::hip_check(hipMemcpyAsync(&nnzb, row_ptr + T, sizeof nnzb,
                                    hipMemcpyDeviceToHost, s),
                     "mf_topp_select_bsr nnzb read-back");
  if (st != MF_OK) return st;
  st = mf::hip_check(hipStreamSynchronize(s), "mf_topp_select_bsr synchronise");
  if (st != MF_OK) return st;
  *nnzb_out = nnzb;
  if (nnzb > cap_nnzb)
    return mf::fail(MF_ERR_CAPACITY, std::string(fn) + fmt(": nnzb = %lld exceeds cap_nnzb = %lld",
                                                           nnzb, cap_nnzb));
  return MF_OK;
}

int mf_topp_select_bsr_noalloc(const float* mass, const void* A, int dtype, int H_s, int N, int B,
                               float p, int32_t* row_ptr, int32_t* col_idx, void* vals,
                               int64_t cap_nnzb, void* stream) {
  const char* fn = "mf_topp_select_bsr_noalloc";
  int st = check_geom(fn, dtype, H_s, N, B);
  if (st != MF_OK) return st;
  if (!mass || !A || !row_ptr) return mf::fail(MF_ERR_INVALID, std::string(fn) + ": null pointer");
  if (cap_nnzb < 0) return mf::fail(MF_ERR_INVALID, std::string(fn) + ": cap_nnzb < 0");
  if (cap_nnzb > 0 && (!col_idx || !vals))
    return mf::fail(MF_ERR_INVALID, std::string(fn) + ": null col_idx/vals with cap_nnzb > 0");
  if (!(p > 0.0f && p <= 1.0f))  // also rejects NaN
    return mf::fail(MF_ERR_INVALID, std::string(fn) + ": p must be in (0, 1]");
  const int T = mf::blocks_of(N, B);
  if (T > kNoAllocMaxT)
    return mf::fail(MF_ERR_UNSUPPORTED,
                    std::string(fn) + fmt(": T = %lld block rows exceeds the %lld that the fixed scratch "
                                          "holds (use mf_topp_select_bsr with a workspace)",
                                          T, kNoAllocMaxT));
  void* ws = nullptr;
  st = noalloc_scratch(fn, &ws);
  if (st != MF_OK) return st;
  return mf::hip_check(mf::launch_topp_bsr(mass, A, dtype, H_s, N, B, p, row_ptr, col_idx, vals,
                                           cap_nnzb, ws, (hipStream_t)stream),
                       "mf_topp_select_bsr_noalloc launch");
}

// Shape checks shared by the calls that read Q and K.
static int check_qk(const char* fn, int dtype, int H_s, int H_ks, int N, int d, int B) {
  int st = check_geom(fn, dtype, H_s, N, B);
  if (st != MF_OK) return st;
  if (H_ks < 1 || H_s % H_ks != 0)
    return mf::fail(MF_ERR_INVALID, std::string(fn) + fmt(": H_ks = %lld does not divide H_s", H_ks));
  if (d != 64 && d != 128) return mf::fail(MF_ERR_INVALID, std::string(fn) + fmt(": d must be 64 or 128 (got %lld)", d));
  return MF_OK;
}

int mf_row_lse(const void* Q, const void* K, int dtype, int H_s, int H_ks, int N, int d,
               const float* scale, float* lse, void* stream) {
  const char* fn = "mf_row_lse";
  // any valid block size passes the shared geometry check
  int st = check_qk(fn, dtype, H_s, H_ks, N, d, 16);
  if (st != MF_OK) return st;
  if (!Q || !K || !scale || !lse) return mf::fail(MF_ERR_INVALID, std::string(fn) + ": null pointer");
  return mf::hip_check(mf::launch_row_lse(Q, K, dtype, H_s, H_ks, N, d, scale, lse,
                                          (hipStream_t)stream), "mf_row_lse launch");
}

size_t mf_block_mass_qk_workspace_bytes(int H_s, int N, int B) {
  if (H_s < 1 || H_s > 64 || N < 1 || !valid_block(B)) return 0;
  return mf::block_mass_qk_workspace_bytes(H_s, N, B);
}

size_t mf_lse_block_mass_qk_workspace_bytes(int H_s, int N, int B) {
  if (H_s < 1 || H_s > 64 || N < 1 || !valid_block(B)) return 0;
  return mf::lse_block_mass_qk_workspace_bytes(H_s, N, B);
}

int mf_lse_block_mass_qk(const void* Q, const void* K, const float* scale, int dtype, int H_s,
                         int H_ks, int N, int d, int B, float* lse, float* mass,
                         void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "mf_lse_block_mass_qk";
  int st = check_qk(fn, dtype, H_s, H_ks, N, d, B);
  if (st != MF_OK) return st;
  if (!Q || !K || !scale || !lse || !mass || !workspace)
    return mf::fail(MF_ERR_INVALID, std::string(fn) + ": null pointer");
  const size_t need = mf::lse_block_mass_qk_workspace_bytes(H_s, N, B);
  if (workspace_bytes < need)
    return mf::fail(MF_ERR_INVALID, std::string(fn) + fmt(": workspace of %lld bytes < %lld required",
                                                          (long long)workspace_bytes, (long long)need));
  return mf::hip_check(mf::launch_lse_block_mass_qk(Q, K, scale, dtype, H_s, H_ks, N, d, B, lse, mass,
                                                    workspace, (hipStream_t)stream),
                       "mf_lse_block_mass_qk launch");
}

int mf_block_mass_qk(const void* Q, const void* K, const float* scale, const float* lse,
                     int dtype, int H_s, int H_ks, int N, int d, int B, float* mass,
                     void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "mf_block_mass_qk";
  int st = check_qk(fn, dtype, H_s, H_ks, N, d, B);
  if (st != MF_OK) return st;
  if (!Q || !K || !scale || !lse || !mass || !workspace)
    return mf::fail(MF_ERR_INVALID, std::string(fn) + ": null pointer");
  const size_t need = mf::block_mass_qk_workspace_bytes(H_s, N, B);
  if (workspace_bytes < need)
    return mf::fail(MF_ERR_INVALID, std::string(fn) + fmt(": workspace of %lld bytes < %lld required",
                                                          (long long)workspace_bytes, (long long)need));
  return mf::hip_check(mf::launch_block_mass_qk(Q, K, scale, lse, dtype, H_s, H_ks, N, d, B, mass,
                                                workspace, (hipStream_t)stream),
                       "mf_block_mass_qk launch");
}

int mf_topp_select_bsr_qk(const float* mass, const void* Q, const void* K,
                          const float* scale, const float* lse, int dtype, int H_s,
                          int H_ks, int N, int d, int B, float p, int32_t* row_ptr,
                          int32_t* col_idx, void* vals, int64_t cap_nnzb,
                          int64_t* nnzb_out, void* workspace, size_t workspace_bytes,
                          void* stream) {
  const char* fn = "mf_topp_select_bsr_qk";
  int st = check_qk(fn, dtype, H_s, H_ks, N, d, B);
  if (st != MF_OK) return st;
  if (!mass || !Q || !K || !scale || !lse || !row_ptr || !workspace)
    return mf::fail(MF_ERR_INVALID, std::string(fn) + ": null pointer");
  if (cap_nnzb < 0) return mf::fail(MF_ERR_INVALID, std::string(fn) + ": cap_nnzb < 0");
  if (cap_nnzb > 0 && (!col_idx || !vals))
    return mf::fail(MF_ERR_INVALID, std::string(fn) + ": null col_idx/vals with cap_nnzb > 0");
  if (!(p > 0.0f && p <= 1.0f))  // also rejects NaN
    return mf::fail(MF_ERR_INVALID, std::string(fn) + ": p must be in (0, 1]");
  const int T = mf::blocks_of(N, B);
  if (T > 4096)
    return mf::fail(MF_ERR_UNSUPPORTED, std::string(fn) + fmt(": T = %lld block rows > 4096", T));
  if (workspace_bytes < mf_topp_workspace_bytes(N, B))
    return mf::fail(MF_ERR_INVALID, std::string(fn) + fmt(": workspace of %lld bytes < %lld required",
                                                          (long long)workspace_bytes,
                                                          (long long)mf_topp_workspace_bytes(N, B)));
  hipStream_t s = (hipStream_t)stream;
  st = mf::hip_check(mf::launch_select_scan(mass, N, B, p, row_ptr, workspace, s),
                     "mf_topp_select_bsr_qk selection launch");
  if (st != MF_OK) return st;
  st = mf::hip_check(mf::launch_gather_qk(Q, K, scale, lse, dtype, H_s, H_ks, N, d, B, row_ptr,
                                          reinterpret_cast<const int32_t*>(workspace), cap_nnzb,
                                          col_idx, vals, s),
                     "mf_topp_select_bsr_qk gather launch");
  if (st != MF_OK || !nnzb_out) return st;
  int32_t nnzb = 0;
  st = mf::hip_check(hipMemcpyAsync(&nnzb, row_ptr + T, sizeof nnzb, hipMemcpyDeviceToHost, s),
                     "mf_topp_select_bsr_qk nnzb read-back");
  if (st != MF_OK) return st;
  st = mf::hip_check(hipStreamSynchronize(s), "mf_topp_select_bsr_qk synchronise");
  if (st != MF_OK) return st;
  *nnzb_out = nnzb;
  if (nnzb > cap_nnzb)
    return mf::fail(MF_ERR_CAPACITY, std::string(fn) + fmt(": nnzb = %lld exceeds cap_nnzb = %lld",
                                                           nnzb, cap_nnzb));
  return MF_OK;
}

size_t mf_retrieve_workspace_bytes(int N, int B, int H_kv, int d, int dtype) {
  if (N < 1 || !valid_block(B) || H_kv < 1 || !valid_dtype(dtype)) return 0;
  return mf::retrieve_workspace_bytes(N, B, H_kv, d, dtype);
}

size_t mf_retrieve_split_workspace_bytes(int64_t nnzb, int dtype, int H_s, int N, int B, int H_r,
                                         int H_kv, int d) {
  if (nnzb <= 0 || N < 1 || !valid_block(B) || !valid_dtype(dtype) || H_s < 1 || H_s > 64 ||
      H_r < 1 || H_r > 64 || H_kv < 1 || H_r % H_kv != 0)
    return 0;
  return mf::split_workspace_bytes(dtype, H_s, N, B, H_r, H_kv, d, nnzb);
}

// Shape and stride checks shared by mf_retrieve_fused and mf_retrieve_kernel.
static int check_retrieve_shape(const char* fn, int dtype, int H_s, int N, int B, int H_r,
                                int H_kv, int d, int64_t ldV, int64_t ldO) {
  int st = check_geom(fn, dtype, H_s, N, B);
  if (st != MF_OK) return st;
  if (H_r < 1 || H_r > 64) return mf::fail(MF_ERR_INVALID, std::string(fn) + fmt(": H_r must be in [1, 64] (got %lld)", H_r));
  if (H_kv < 1 || H_r % H_kv != 0)
    return mf::fail(MF_ERR_INVALID, std::string(fn) + fmt(": H_r = %lld is not a multiple of H_kv = %lld", H_r, H_kv));
  if (d != 64 && d != 128) return mf::fail(MF_ERR_INVALID, std::string(fn) + fmt(": d must be 64 or 128 (got %lld)", d));
  if (ldV < (int64_t)H_kv * d) return mf::fail(MF_ERR_INVALID, std::string(fn) + ": ldV < H_kv*d");
  if (ldO < (int64_t)H_r * d) return mf::fail(MF_ERR_INVALID, std::string(fn) + ": ldO < H_r*d");
  return MF_OK;
}

int mf_retrieve_kernel(int dtype, int H_s, int N, int B, int H_r, int H_kv, int d,
                       const void* vals, const void* V, int64_t ldV, const void* O,
                       int64_t ldO) {
  const int st = check_retrieve_shape("mf_retrieve_kernel", dtype, H_s, N, B, H_r, H_kv, d, ldV, ldO);
  if (st != MF_OK) return -st;
  return mf::retrieve_uses_mfma(dtype, H_s, B, H_r, H_kv, d, vals, V, ldV, O, ldO) ? 1 : 0;
}

int mf_retrieve_fused(const int32_t* row_ptr, const int32_t* col_idx,
                      const void* vals, int64_t nnzb, int dtype, int H_s,
                      int N, int B, const float* W, int H_r, const void* V,
                      int H_kv, int d, int64_t ldV, void* O, int64_t ldO,
                      void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "mf_retrieve_fused";
  int st = check_geom(fn, dtype, H_s, N, B);
  if (st != MF_OK) return st;
  if (!row_ptr || !W || !V || !O) return mf::fail(MF_ERR_INVALID, std::string(fn) + ": null pointer");
  if (nnzb < 0) return mf::fail(MF_ERR_INVALID, std::string(fn) + ": nnzb < 0");
  if (nnzb > 0 && (!col_idx || !vals))
    return mf::fail(MF_ERR_INVALID, std::string(fn) + ": null col_idx/vals with nnzb > 0");
  if (H_r < 1 || H_r > 64) return mf::fail(MF_ERR_INVALID, std::string(fn) + fmt(": H_r must be in [1, 64] (got %lld)", H_r));
  if (H_kv < 1 || H_r % H_kv != 0)
    return mf::fail(MF_ERR_INVALID, std::string(fn) + fmt(": H_r = %lld is not a multiple of H_kv = %lld", H_r, H_kv));
  if (d != 64 && d != 128) return mf::fail(MF_ERR_INVALID, std::string(fn) + fmt(": d must be 64 or 128 (got %lld)", d));
  if (ldV < (int64_t)H_kv * d) return mf::fail(MF_ERR_INVALID, std::string(fn) + ": ldV < H_kv*d");
  if (ldO < (int64_t)H_r * d) return mf::fail(MF_ERR_INVALID, std::string(fn) + ": ldO < H_r*d");
  const size_t need = mf::retrieve_workspace_bytes(N, B, H_kv, d, dtype);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return mf::fail(MF_ERR_INVALID, std::string(fn) + fmt(": workspace of %lld bytes < %lld required",
                                                          workspace ? (long long)workspace_bytes : 0LL,
                                                          (long long)need));
  return mf::launch_retrieve(row_ptr, col_idx, vals, nnzb, dtype, H_s, N, B, W,
                             H_r, V, H_kv, d, ldV, O, ldO, workspace, workspace_bytes,
                             (hipStream_t)stream);
}

int mf_retrieve_fused_multi(const int32_t* row_ptr, const int32_t* col_idx, const void* vals,
                            int64_t nnzb, int dtype, int H_s, int N, int B, int n_recv,
                            const float* const* W, const int* H_r, const void* const* V,
                            const int* H_kv, int d, const int64_t* ldV, void* const* O,
                            const int64_t* ldO, void* stream) {
  const char* fn = "mf_retrieve_fused_multi";
  if (n_recv < 1 || n_recv > 4)
    return mf::fail(MF_ERR_INVALID, std::string(fn) + fmt(": n_recv must be in [1, 4] (got %lld)", n_recv));
  if (!W || !H_r || !V || !H_kv || !ldV || !O || !ldO)
    return mf::fail(MF_ERR_INVALID, std::string(fn) + ": null receiver array");
  if (!row_ptr) return mf::fail(MF_ERR_INVALID, std::string(fn) + ": null pointer");
  if (nnzb < 0) return mf::fail(MF_ERR_INVALID, std::string(fn) + ": nnzb < 0");
  if (nnzb > 0 && (!col_idx || !vals))
    return mf::fail(MF_ERR_INVALID, std::string(fn) + ": null col_idx/vals with nnzb > 0");
  for (int i = 0; i < n_recv; ++i) {
    const std::string fi = std::string(fn) + fmt(" (receiver %lld)", i);
    const int st = check_retrieve_shape(fi.c_str(), dtype, H_s, N, B, H_r[i], H_kv[i], d, ldV[i], ldO[i]);
    if (st != MF_OK) return st;
    if (!W[i] || !V[i] || !O[i]) return mf::fail(MF_ERR_INVALID, fi + ": null pointer");
    for (int j = 0; j < i; ++j)
      if (O[j] == O[i]) return mf::fail(MF_ERR_INVALID, fi + ": output shared with another receiver");
  }
  return mf::launch_retrieve_multi(row_ptr, col_idx, vals, nnzb, dtype, H_s, N, B, n_recv, W, H_r, V,
                                   H_kv, d, ldV, O, ldO, (hipStream_t)stream);
}

int mf_retrieve_fused_varlen(int S, int R, const int32_t* cu_seqlens, const int32_t* cu_rows,
                             const int32_t* row_ptr, const int32_t* col_idx,
                             const int32_t* block_table, const void* vals, int64_t n_pages,
                             int64_t nnzb, int dtype, int H_s, int B, const float* W, int H_r,
                             const void* V, int H_kv, int d, int64_t ldV, void* O, int64_t ldO,
                             void* stream) {
  const char* fn = "mf_retrieve_fused_varlen";
  if (S < 1) return mf::fail(MF_ERR_INVALID, std::string(fn) + fmt(": S must be >= 1 (got %lld)", S));
  if (R < 0) return mf::fail(MF_ERR_INVALID, std::string(fn) + ": R < 0");
  // N = 1 stands in for the per-sequence lengths, which live on the device
  const int st = check_retrieve_shape(fn, dtype, H_s, 1, B, H_r, H_kv, d, ldV, ldO);
  if (st != MF_OK) return st;
  if (!cu_seqlens || !cu_rows || !row_ptr || !W || !V || !O)
    return mf::fail(MF_ERR_INVALID, std::string(fn) + ": null pointer");
  if (nnzb < 0) return mf::fail(MF_ERR_INVALID, std::string(fn) + ": nnzb < 0");
  if (nnzb > 0 && (!col_idx || !vals))
    return mf::fail(MF_ERR_INVALID, std::string(fn) + ": null col_idx/vals with nnzb > 0");
  if (block_table && n_pages < 0) return mf::fail(MF_ERR_INVALID, std::string(fn) + ": n_pages < 0");
  return mf::launch_retrieve_varlen(S, R, cu_seqlens, cu_rows, row_ptr, col_idx, block_table, vals,
                                    n_pages, nnzb, dtype, H_s, B, W, H_r, V, H_kv, d, ldV, O, ldO,
                                    (hipStream_t)stream);
}

// ---- attention operators --------------------------------------------------

#define MF_REQUIRE(cond, msg) \
  do {                        \
    if (!(cond)) return mf::fail(MF_ERR_INVALID, std::string(fn) + ": " + (msg)); \
  } while (0)

static int check_heads(const char* fn, int dtype, int H, int H_kv, int d) {
  MF_REQUIRE(valid_dtype(dtype), fmt("unknown dtype code %lld", dtype));
  MF_REQUIRE(H >= 1 && H <= 64, fmt("head counts must be in [1, 64] (got %lld)", H));
  MF_REQUIRE(H_kv >= 1 && H % H_kv == 0, fmt("H = %lld is not a multiple of H_kv = %lld", H, H_kv));
  MF_REQUIRE(d == 64 || d == 128, fmt("d must be 64 or 128 (got %lld)", d));
  return MF_OK;
}

static int check_workspace(const char* fn, const void* ws, size_t have, size_t need) {
  MF_REQUIRE(need == 0 || (ws && have >= need),
             fmt("workspace of %lld bytes < %lld required", ws ? (long long)have : 0LL,
                 (long long)need));
  MF_REQUIRE(!ws || reinterpret_cast<uintptr_t>(ws) % 16 == 0, "workspace off 16 bytes");
  return MF_OK;
}

// strides of an output that keep its N x H rows of d elements apart
static bool rows_apart(int64_t N, int64_t H, int64_t d, int64_t ld, int64_t hs) {
  const bool by_row = hs >= d && ld >= (H - 1) * hs + d;
  const bool by_head = ld >= d && hs >= (N - 1) * ld + d;
  return by_row || by_head || (N <= 1 && hs >= d) || (H <= 1 && ld >= d);
}

static int check_mask(const char* fn, int window, int sinks) {
  MF_REQUIRE(window >= 0, fmt("window must be >= 0 (got %lld)", window));
  MF_REQUIRE(sinks >= 0, fmt("sinks must be >= 0 (got %lld)", sinks));
  return MF_OK;
}

static int check_cache(const char* fn, const mf::Cache& c, int S, bool empty) {
  MF_REQUIRE(S >= 0, "S < 0");
  MF_REQUIRE(c.n_pages >= 0, "n_pages < 0");
  MF_REQUIRE(c.page >= 1, fmt("page must be >= 1 (got %lld)", c.page));
  MF_REQUIRE(c.max_pages >= 0, "max_pages < 0");
  MF_REQUIRE(c.max_len >= 0 && c.max_len <= (int64_t)c.max_pages * c.page,
             fmt("max_len = %lld outside [0, max_pages*page = %lld]", c.max_len,
                 (long long)c.max_pages * c.page));
  if (empty) return MF_OK;
  MF_REQUIRE(c.lens, "null lens");
  MF_REQUIRE((c.K && c.V) || c.n_pages == 0 || c.max_len == 0, "null pool");
  MF_REQUIRE(reinterpret_cast<uintptr_t>(c.K) % 16 == 0 && reinterpret_cast<uintptr_t>(c.V) % 16 == 0,
             "pools must be 16-byte aligned");
  return MF_OK;
}

int mf_rope_frequencies(int rot, double base, int scaling, double factor, double orig_len,
                        double beta_fast, double beta_slow, double* freq, double* attn_factor) {
  const char* fn = "mf_rope_frequencies";
  MF_REQUIRE(freq && attn_factor, "null pointer");
  MF_REQUIRE(rot >= 2 && rot <= 256 && rot % 2 == 0, fmt("rot must be even and in [2, 256] (got %lld)", rot));
  MF_REQUIRE(base > 1.0 && isfinite(base), "base must be > 1");
  MF_REQUIRE(factor >= 1.0 && isfinite(factor), "factor must be >= 1");
  MF_REQUIRE(scaling >= MF_ROPE_PLAIN && scaling <= MF_ROPE_YARN, fmt("unknown scaling %lld", scaling));
  MF_REQUIRE(scaling != MF_ROPE_NTK || rot > 2, "rot must be > 2 for this scaling");
  double lo = 0, hi = 0;
  if (scaling == MF_ROPE_YARN) {
    MF_REQUIRE(orig_len > 0 && isfinite(orig_len), "orig_len must be > 0");
    MF_REQUIRE(beta_slow > 0 && beta_fast > beta_slow && isfinite(beta_fast), "need 0 < beta_slow < beta_fast");
    const double two_pi = 6.283185307179586476925;
    lo = floor(rot * log(orig_len / (beta_fast * two_pi)) / (2 * log(base)));
    hi = ceil(rot * log(orig_len / (beta_slow * two_pi)) / (2 * log(base)));
    lo = lo < 0 ? 0 : lo;
    hi = hi > rot - 1 ? rot - 1 : hi;
  }
  if (scaling == MF_ROPE_NTK) base *= pow(factor, rot / (rot - 2.0));
  for (int i = 0; i < rot / 2; ++i) {
    double f = pow(base, -2.0 * i / rot);
    if (scaling == MF_ROPE_LINEAR) f /= factor;
    if (scaling == MF_ROPE_YARN) {
      const double span = hi - lo > 0.001 ? hi - lo : 0.001;
      double r = (i - lo) / span;
      r = r < 0 ? 0 : r > 1 ? 1 : r;
      f = f / factor * r + f * (1 - r);
    }
    freq[i] = f;
  }
  *attn_factor = scaling == MF_ROPE_YARN ? 0.1 * log(factor) + 1.0 : 1.0;
  return MF_OK;
}

static int check_rope(const char* fn, int dtype, const mf::RopeArgs& a) {
  MF_REQUIRE(valid_dtype(dtype), fmt("unknown dtype code %lld", dtype));
  MF_REQUIRE(a.N >= 0, "N < 0");
  MF_REQUIRE(a.d == 64 || a.d == 128, fmt("d must be 64 or 128 (got %lld)", a.d));
  MF_REQUIRE(a.H_q >= 1 && a.H_q <= 64 && a.H_k >= 1 && a.H_k <= 64, "head counts must be in [1, 64]");
  MF_REQUIRE(a.rot >= 0 && a.rot <= a.d && a.rot % 2 == 0, fmt("rot must be even and in [0, d] (got %lld)", a.rot));
  MF_REQUIRE(a.layout == MF_ROPE_HALF || a.layout == MF_ROPE_INTERLEAVED, fmt("unknown layout %lld", a.layout));
  MF_REQUIRE(a.eps >= 0.f, "eps must be >= 0");
  MF_REQUIRE(a.ldq >= (int64_t)a.H_q * a.d && a.ldk >= (int64_t)a.H_k * a.d, "ldq or ldk smaller than a row");
  MF_REQUIRE(rows_apart(a.N, a.H_q, a.d, a.ldQ, a.hsQ), "rows of Q overlap");
  if (a.N == 0) return MF_OK;
  MF_REQUIRE(a.q && a.k && a.Q, "null pointer");
  MF_REQUIRE(a.rot == 0 || (a.freq && a.positions), "null freq or positions");
  return MF_OK;
}

int mf_qk_norm_rope(int dtype, int N, int d, const void* q, int H_q, int64_t ldq, const void* k,
                    int H_k, int64_t ldk, const void* wq, const void* wk, float eps,
                    const double* freq, int rot, int layout, float attn_factor,
                    const int32_t* positions, void* Q, int64_t ldQ, int64_t hsQ, void* K,
                    int64_t ldK, int64_t hsK, void* stream) {
  const char* fn = "mf_qk_norm_rope";
  mf::RopeArgs a = {};
  a.N = N; a.d = d; a.H_q = H_q; a.H_k = H_k;
  a.q = q; a.k = k; a.ldq = ldq; a.ldk = ldk;
  a.wq = wq; a.wk = wk; a.eps = eps;
  a.freq = freq; a.rot = rot; a.layout = layout; a.attn_factor = attn_factor;
  a.positions = positions;
  a.Q = Q; a.K = K; a.ldQ = ldQ; a.hsQ = hsQ; a.ldK = ldK; a.hsK = hsK;
  const int st = check_rope(fn, dtype, a);
  if (st != MF_OK) return st;
  MF_REQUIRE(rows_apart(N, H_k, d, ldK, hsK), "rows of K overlap");
  if (N == 0) return MF_OK;
  MF_REQUIRE(K && K != Q, "null K, or K equal to Q");
  MF_REQUIRE((Q != q || (ldQ == ldq && hsQ == d)) && (K != k || (ldK == ldk && hsK == d)) && Q != k && K != q,
             "an output overlaps an input with another layout");
  return mf::hip_check(mf::launch_rope(dtype, a, (hipStream_t)stream), "mf_qk_norm_rope launch");
}

int mf_qk_norm_rope_cache(int dtype, int N, int d, const void* q, int H_q, int64_t ldq,
                          const void* k, int H_k, int64_t ldk, const void* v, int64_t ldv,
                          const void* wq, const void* wk, float eps, const double* freq, int rot,
                          int layout, float attn_factor, const int32_t* positions, void* Q,
                          int64_t ldQ, int64_t hsQ, const int64_t* slots, void* K, void* V,
                          int64_t n_pages, int page, void* stream) {
  const char* fn = "mf_qk_norm_rope_cache";
  mf::RopeArgs a = {};
  a.N = N; a.d = d; a.H_q = H_q; a.H_k = H_k;
  a.q = q; a.k = k; a.v = v; a.ldq = ldq; a.ldk = ldk; a.ldv = ldv;
  a.wq = wq; a.wk = wk; a.eps = eps;
  a.freq = freq; a.rot = rot; a.layout = layout; a.attn_factor = attn_factor;
  a.positions = positions;
  a.Q = Q; a.K = K; a.V = V; a.ldQ = ldQ; a.hsQ = hsQ;
  a.slots = slots; a.n_pages = n_pages; a.page = page;
  const int st = check_rope(fn, dtype, a);
  if (st != MF_OK) return st;
  MF_REQUIRE(ldv >= (int64_t)H_k * d, "ldv smaller than a row");
  MF_REQUIRE(n_pages >= 0 && page >= 1, "n_pages < 0 or page < 1");
  if (N == 0) return MF_OK;
  MF_REQUIRE(v && slots, "null v or slots");
  MF_REQUIRE((K && V) || n_pages == 0, "null pool");
  MF_REQUIRE(reinterpret_cast<uintptr_t>(K) % 16 == 0 && reinterpret_cast<uintptr_t>(V) % 16 == 0,
             "pools must be 16-byte aligned");
  MF_REQUIRE(n_pages == 0 || K != V, "K and V are one pool");
  MF_REQUIRE((Q != q || (ldQ == ldq && hsQ == d)) && Q != k && Q != v,
             "an output overlaps an input with another layout");
  return mf::hip_check(mf::launch_rope(dtype, a, (hipStream_t)stream), "mf_qk_norm_rope_cache launch");
}

static int check_attention(const char* fn, int dtype, const mf::AttnArgs& a) {
  int st = check_heads(fn, dtype, a.H, a.H_kv, a.d);
  if (st != MF_OK) return st;
  MF_REQUIRE(a.N_q >= 0 && a.N_k >= 0, "N_q or N_k < 0");
  st = check_mask(fn, a.window, a.sinks);
  if (st != MF_OK) return st;
  MF_REQUIRE(a.Q.ld >= 0 && a.Q.hs >= 0 && a.K.ld >= 0 && a.K.hs >= 0 && a.V.ld >= 0 && a.V.hs >= 0,
             "a stride is negative");
  MF_REQUIRE(a.ldO >= (int64_t)a.H * a.d, "ldO < H*d");
  if (a.N_q == 0) return MF_OK;
  MF_REQUIRE(a.Q.p && a.O && a.scale && ((a.K.p && a.V.p) || a.N_k == 0), "null pointer");
  MF_REQUIRE(a.O != a.Q.p && a.O != a.K.p && a.O != a.V.p, "O is one of the inputs");
  return MF_OK;
}

size_t mf_attention_split_workspace_bytes(int dtype, int H, int H_kv, int N_q, int N_k, int d,
                                          int window, int sinks) {
  if (!valid_dtype(dtype) || H < 1 || H > 64 || H_kv < 1 || H % H_kv != 0 || (d != 64 && d != 128) ||
      N_q < 1 || N_k < 1 || window < 0 || sinks < 0)
    return 0;
  return mf::attention_split_bytes(dtype, H, H_kv, N_q, N_k, d, window, sinks);
}

int mf_attention_window(const void* Q, int64_t ldQ, int64_t hsQ, const void* K, int64_t ldK,
                        int64_t hsK, const void* V, int64_t ldV, int64_t hsV, int dtype, int H,
                        int H_kv, int N_q, int N_k, int d, const float* scale, int window,
                        int sinks, void* O, int64_t ldO, float* lse, void* workspace,
                        size_t workspace_bytes, void* stream) {
  const char* fn = "mf_attention_window";
  mf::AttnArgs a = {};
  a.Q = {Q, ldQ, hsQ}; a.K = {K, ldK, hsK}; a.V = {V, ldV, hsV};
  a.O = O; a.ldO = ldO; a.lse = lse; a.scale = scale;
  a.H = H; a.H_kv = H_kv; a.N_q = N_q; a.N_k = N_k; a.d = d; a.window = window; a.sinks = sinks;
  int st = check_attention(fn, dtype, a);
  if (st != MF_OK || N_q == 0) return st;
  st = check_workspace(fn, workspace, workspace_bytes, 0);
  if (st != MF_OK) return st;
  return mf::hip_check(mf::launch_attention(dtype, a, workspace, workspace ? workspace_bytes : 0,
                                            (hipStream_t)stream), "mf_attention_window launch");
}

int mf_attention_window_varlen(int S, const int32_t* cu_q, const int32_t* cu_k, const void* Q,
                               int64_t ldQ, int64_t hsQ, const void* K, int64_t ldK, int64_t hsK,
                               const void* V, int64_t ldV, int64_t hsV, int dtype, int H, int H_kv,
                               int N_q, int N_k, int d, const float* scale, int window, int sinks,
                               void* O, int64_t ldO, float* lse, void* stream) {
  const char* fn = "mf_attention_window_varlen";
  mf::AttnArgs a = {};
  a.Q = {Q, ldQ, hsQ}; a.K = {K, ldK, hsK}; a.V = {V, ldV, hsV};
  a.O = O; a.ldO = ldO; a.lse = lse; a.scale = scale;
  a.H = H; a.H_kv = H_kv; a.N_q = N_q; a.N_k = N_k; a.d = d; a.window = window; a.sinks = sinks;
  a.S = S; a.cu_q = cu_q; a.cu_k = cu_k;
  MF_REQUIRE(S >= 0, fmt("S must be >= 0 (got %lld)", S));
  const int st = check_attention(fn, dtype, a);
  if (st != MF_OK || N_q == 0 || S == 0) return st;
  MF_REQUIRE(cu_q && cu_k, "null cu_q or cu_k");
  return mf::hip_check(mf::launch_attention(dtype, a, nullptr, 0, (hipStream_t)stream),
                       "mf_attention_window_varlen launch");
}

size_t mf_attention_decode_workspace_bytes(int S, int max_len, int H, int H_kv, int d, int window,
                                           int sinks, int with_mass) {
  if (S < 1 || max_len < 0 || H < 1 || H > 64 || H_kv < 1 || H % H_kv != 0 || (d != 64 && d != 128) ||
      window < 0 || sinks < 0)
    return 0;
  return mf::decode_workspace_bytes(S, max_len, H, H_kv, d, window, sinks, with_mass != 0);
}

int mf_attention_decode(const void* Q, int64_t ldQ, const void* K, const void* V, int64_t n_pages,
                        int page, const int32_t* block_table, int max_pages, const int32_t* lens,
                        int dtype, int S, int max_len, int H, int H_kv, int d, const float* scale,
                        int window, int sinks, void* O, int64_t ldO, float* lse,
                        const float* mass_in, float* mass_out, int64_t ldmass, void* workspace,
                        size_t workspace_bytes, void* stream) {
  const char* fn = "mf_attention_decode";
  mf::DecodeArgs a = {};
  a.Q = Q; a.ldQ = ldQ;
  a.c = {K, V, n_pages, page, block_table, max_pages, lens, max_len};
  a.S = S; a.H = H; a.H_kv = H_kv; a.d = d; a.window = window; a.sinks = sinks;
  a.scale = scale; a.O = O; a.ldO = ldO; a.lse = lse;
  a.mass_in = mass_in; a.mass_out = mass_out; a.ldmass = ldmass;
  int st = check_heads(fn, dtype, H, H_kv, d);
  if (st != MF_OK) return st;
  st = check_mask(fn, window, sinks);
  if (st != MF_OK) return st;
  st = check_cache(fn, a.c, S, S == 0);
  if (st != MF_OK) return st;
  MF_REQUIRE(ldQ >= (int64_t)H * d && ldO >= (int64_t)H * d, "ldQ or ldO < H*d");
  MF_REQUIRE(!mass_in || mass_out, "mass_in without mass_out");
  MF_REQUIRE(!mass_out || ldmass >= max_len, "ldmass < max_len");
  if (S == 0) return MF_OK;
  MF_REQUIRE(Q && O && scale, "null pointer");
  MF_REQUIRE(O != Q && O != K && O != V, "O is one of the inputs");
  st = check_workspace(fn, workspace, workspace_bytes,
                       mf::decode_workspace_bytes(S, max_len, H, H_kv, d, window, sinks, mass_out != nullptr));
  if (st != MF_OK) return st;
  return mf::hip_check(mf::launch_decode(dtype, a, workspace, (hipStream_t)stream),
                       "mf_attention_decode launch");
}

size_t mf_key_mass_qk_workspace_bytes(int dtype, int H, int H_kv, int N_q, int N_k, int d,
                                      int window, int sinks) {
  if (!valid_dtype(dtype) || H < 1 || H > 64 || H_kv < 1 || H % H_kv != 0 || (d != 64 && d != 128) ||
      N_q < 0 || N_k < 0 || window < 0 || sinks < 0)
    return 0;
  return mf::key_mass_workspace_bytes(dtype, H, H_kv, N_q, N_k, d, window, sinks);
}

int mf_key_mass_qk(const void* Q, int64_t ldQ, int64_t hsQ, const void* K, int64_t ldK, int64_t hsK,
                   const float* scale, const float* lse, int dtype, int H, int H_kv, int N_q,
                   int N_k, int d, int window, int sinks, const float* mass_in, float* mass_out,
                   void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "mf_key_mass_qk";
  mf::KeyMassArgs a = {};
  a.Q = {Q, ldQ, hsQ}; a.K = {K, ldK, hsK}; a.scale = scale; a.lse = lse;
  a.H = H; a.H_kv = H_kv; a.N_q = N_q; a.N_k = N_k; a.d = d; a.window = window; a.sinks = sinks;
  a.mass_in = mass_in; a.mass_out = mass_out;
  int st = check_heads(fn, dtype, H, H_kv, d);
  if (st != MF_OK) return st;
  MF_REQUIRE(N_q >= 0 && N_k >= 0, "N_q or N_k < 0");
  st = check_mask(fn, window, sinks);
  if (st != MF_OK) return st;
  MF_REQUIRE(ldQ >= 0 && hsQ >= 0 && ldK >= 0 && hsK >= 0, "a stride is negative");
  if (N_k == 0) return MF_OK;
  MF_REQUIRE(K && scale && mass_out && ((Q && lse) || N_q == 0), "null pointer");
  st = check_workspace(fn, workspace, workspace_bytes,
                       mf::key_mass_workspace_bytes(dtype, H, H_kv, N_q, N_k, d, window, sinks));
  if (st != MF_OK) return st;
  return mf::hip_check(mf::launch_key_mass(dtype, a, workspace, (hipStream_t)stream),
                       "mf_key_mass_qk launch");
}

int mf_cache_evict(const float* mass, int64_t ldmass, const void* K, const void* V, int64_t n_pages,
                   int page, const int32_t* block_table, int max_pages, const int32_t* lens,
                   int dtype, int S, int max_len, int H_kv, int d, int budget, int sinks,
                   int recent, void* K_out, void* V_out, int64_t cap_out, float* mass_out,
                   int32_t* kept, int32_t* lens_out, void* stream) {
  const char* fn = "mf_cache_evict";
  mf::EvictArgs a = {};
  a.mass = mass; a.ldmass = ldmass;
  a.c = {K, V, n_pages, page, block_table, max_pages, lens, max_len};
  a.S = S; a.H_kv = H_kv; a.d = d; a.budget = budget; a.sinks = sinks; a.recent = recent;
  a.K_out = K_out; a.V_out = V_out; a.cap_out = cap_out; a.mass_out = mass_out;
  a.kept = kept; a.lens_out = lens_out;
  int st = check_heads(fn, dtype, H_kv, H_kv, d);
  if (st != MF_OK) return st;
  st = check_cache(fn, a.c, S, S == 0);
  if (st != MF_OK) return st;
  MF_REQUIRE(budget >= 1, fmt("budget must be >= 1 (got %lld)", budget));
  MF_REQUIRE(sinks >= 0 && recent >= 0 && (int64_t)sinks + recent <= budget,
             "sinks and recent must be >= 0 and together at most budget");
  MF_REQUIRE(cap_out >= budget, "cap_out < budget");
  MF_REQUIRE(ldmass >= max_len, "ldmass < max_len");
  if (S == 0) return MF_OK;
  MF_REQUIRE((mass || max_len == 0) && kept && K_out && V_out, "null pointer");
  MF_REQUIRE(reinterpret_cast<uintptr_t>(K_out) % 16 == 0 && reinterpret_cast<uintptr_t>(V_out) % 16 == 0,
             "pools must be 16-byte aligned");
  MF_REQUIRE(K_out != K && K_out != V && V_out != K && V_out != V && K_out != V_out,
             "an output pool is a source pool or the other output");
  MF_REQUIRE(mass_out != mass || !mass, "mass_out is mass");
  // every head of a sequence reads its length while one of them writes the new one
  MF_REQUIRE(lens_out != lens, "lens_out is lens");
  return mf::hip_check(mf::launch_evict(dtype, a, (hipStream_t)stream), "mf_cache_evict launch");
}

}  // extern "C"
