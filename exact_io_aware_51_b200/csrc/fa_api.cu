// Host side of the C ABI: argument validation, TMA descriptors, per-device
// state and kernel launches.  See include/fa.h for the contract.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <mutex>

#include "fa.h"
#include "fa_internal.h"
#include "fa_testing.h"

namespace fa {

// Device status word and the epoch of the last launch that hit a wait limit.
__device__ int g_status;
__device__ unsigned int g_abort_epoch;

namespace {

constexpr int kMaxDevices = 64;
constexpr long long kMaxN = 1LL << 22;

thread_local int t_last_cuda_error = 0;
thread_local int t_bound_device = -1;  // device whose primary context this thread has made current
thread_local cudaEvent_t t_ev_start = nullptr;
thread_local cudaEvent_t t_ev_stop = nullptr;
std::atomic<unsigned int> g_epoch{1};
std::atomic<unsigned long long> g_limit_ns{0};
std::atomic<int> g_inject{0};

struct DeviceState {
  std::once_flag once;
  int arch_ok = 0;
  int init_err = 0;
  int* status = nullptr;
  unsigned int* abort_epoch = nullptr;
};
DeviceState g_dev[kMaxDevices];

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

unsigned long long wait_limit_ns() {
  unsigned long long v = g_limit_ns.load();
  if (v == 0) {
    const char* e = std::getenv("FA_TIMEOUT_MS");
    long long ms = e ? std::atoll(e) : 2000;
    if (ms <= 0) ms = 2000;
    v = static_cast<unsigned long long>(ms) * 1000000ull;
    g_limit_ns.store(v);
  }
  return v;
}

int fail_cuda(cudaError_t e) {
  t_last_cuda_error = static_cast<int>(e);
  return FA_ERR_LAUNCH;
}

// A failed TMA descriptor encode is reported as 100000 + the CUresult.
int fail_encode(CUresult r) {
  t_last_cuda_error = 100000 + static_cast<int>(r);
  return FA_ERR_LAUNCH;
}

// Per-device one-time set-up: architecture check and the device addresses of
// the status word and abort epoch (done with that device current).
int device_state(DeviceState** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail_cuda(e);
  if (dev < 0 || dev >= kMaxDevices) return FA_ERR_ARCH;
  // A thread that has not yet made a CUDA runtime call that needs a context
  // (for example an autograd worker thread) has none current; the driver's TMA
  // descriptor encoder needs one, so bind the device's primary context once.
  if (t_bound_device != dev) {
    e = cudaSetDevice(dev);
    if (e != cudaSuccess) return fail_cuda(e);
    t_bound_device = dev;
  }
  DeviceState& st = g_dev[dev];
  std::call_once(st.once, [&] {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
      st.init_err = FA_ERR_ARCH;
      return;
    }
    st.arch_ok = (major == 10 && minor == 0);
    void* p = nullptr;
    cudaError_t e1 = cudaGetSymbolAddress(&p, g_status);
    if (e1 != cudaSuccess) {
      st.init_err = fail_cuda(e1);
      return;
    }
    st.status = static_cast<int*>(p);
    cudaError_t e2 = cudaGetSymbolAddress(&p, g_abort_epoch);
    if (e2 != cudaSuccess) {
      st.init_err = fail_cuda(e2);
      return;
    }
    st.abort_epoch = static_cast<unsigned int*>(p);
  });
  if (st.init_err) return st.init_err;
  if (!st.arch_ok) return FA_ERR_ARCH;
  *out = &st;
  return FA_OK;
}

DevCtl make_ctl(const DeviceState& st) {
  DevCtl c;
  c.status = st.status;
  c.abort_epoch = st.abort_epoch;
  unsigned int ep = g_epoch.fetch_add(1);
  if (ep == 0) ep = g_epoch.fetch_add(1);  // 0 never names a launch
  c.epoch = ep;
  c.limit_ns = wait_limit_ns();
  c.inject = g_inject.load();
  return c;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

int check_shape(int B, int H, int N, int d, int dtype) {
  if (B < 0 || H < 0 || N < 0) return FA_ERR_INVALID_ARG;
  if (dtype != FA_BF16 && dtype != FA_FP32) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (N > kMaxN || H > 65535 || B > 65535) return FA_ERR_TOO_LARGE;
  const double elems = static_cast<double>(B) * N * H * d;
  if (elems >= 1099511627776.0) return FA_ERR_TOO_LARGE;  // 2^40
  return FA_OK;
}

// K/V heads: each of the Hkv heads serves H / Hkv query heads.
int check_kv_heads(int H, int Hkv) {
  if (Hkv < 0 || Hkv > H) return FA_ERR_INVALID_ARG;
  if (H > 0 && (Hkv == 0 || H % Hkv != 0)) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// Window bounds: -1 leaves a side unbounded, otherwise 0 <= bound.
int check_window(int left, int right) {
  if (left < -1 || right < -1) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// Kernel form of a window: a side with no bound gets kUnbounded, which is
// above any sequence length the library accepts, so q - wl and q + wr never
// clip a visible key and never overflow an int.
constexpr int kUnbounded = 1 << 30;
static_assert(kMaxN < kUnbounded / 2, "window sentinel must exceed every sequence length");

void set_window(int left, int right, int* wl, int* wr, int* causal) {
  // a bound at or above the longest sequence hides nothing: same as no bound
  *wl = (left < 0 || left >= kMaxN) ? kUnbounded : left;
  *wr = (right < 0 || right >= kMaxN) ? kUnbounded : right;
  *causal = (*wl == kUnbounded && *wr == 0) ? 1 : 0;
}

// Parts each key tile's (query head, query tile) walk is split into (1, 2, 4 or
// 8; each part keeps at least 8 query tiles, non-causal count).  One CTA runs
// per SM (148 SMs).
//   * Unmasked walks are equally long: the launch takes ceil(CTAs / 148) waves
//     of whole walks, so parts = p costs ceil(p CTAs / 148) / p waves, plus the
//     partial sums (zeroing, reduce-adds, convert), taken as the time of 4 query
//     tiles per part: a factor 1 + 4 p / (query tiles per walk).  The cheapest p
//     wins (ties: fewer parts).  Measured on B200: +16% at B1 H64 Hkv8 N8192
//     d128 (2 parts), and the factor keeps d = 64 walks of 32 tiles unsplit.
//   * Causal and windowed walks differ in length from one key tile to the next,
//     so a grid of fewer than three waves is split until it has three.
int bwd_splits(int B, int H, int Hkv, int N, bool masked) {
  const long long nkt = (static_cast<long long>(N) + 127) / 128;
  const long long ctas = nkt * Hkv * B;
  const long long per_cta = (H / (Hkv > 0 ? Hkv : 1)) * nkt;
  int parts = 1;
  if (masked) {
    while (parts < 8 && ctas * parts < 3 * 148 && per_cta / (2 * parts) >= 8) parts *= 2;
    return parts;
  }
  double best = static_cast<double>((ctas + 147) / 148);
  for (int p = 2; p <= 8 && per_cta / p >= 8; p *= 2) {
    const double cost = static_cast<double>((ctas * p + 147) / 148) / p * (1.0 + 4.0 * p / per_cta);
    if (cost < best - 1e-9) {
      best = cost;
      parts = p;
    }
  }
  return parts;
}

int check_scale(float scale) {
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

}  // namespace

namespace {
// The driver's TMA descriptor encoder, looked up once through the runtime.
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_encode;
}
}  // namespace

CUresult make_tile_map(CUtensorMap* map, const void* base, int B, int N, int H, int d, int rows) {
  if (!encoder()) return CUDA_ERROR_NOT_FOUND;
  // dims innermost first: feature, sequence, head, batch
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(H),
                              static_cast<cuuint64_t>(B)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(H) * d * 2, static_cast<cuuint64_t>(d) * 2,
                                 static_cast<cuuint64_t>(N) * H * d * 2};
  const cuuint32_t box[4] = {64u, static_cast<cuuint32_t>(rows), 1u, 1u};
  const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

CUresult make_paged_map(CUtensorMap* map, const void* base, int num_pages, int page_size, int Hkv, int d) {
  if (!encoder()) return CUDA_ERROR_NOT_FOUND;
  // dims innermost first: (K/V head, feature), pool row = page * page_size + slot
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(Hkv) * d,
                              static_cast<cuuint64_t>(num_pages) * static_cast<cuuint64_t>(page_size)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(Hkv) * d * 2};
  const cuuint32_t box[2] = {64u, static_cast<cuuint32_t>(page_size < 64 ? page_size : 64)};
  const cuuint32_t estr[2] = {1u, 1u};
  return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

CUresult make_paged_map_u8(CUtensorMap* map, const void* base, int num_pages, int page_size, int Hkv, int d) {
  if (!encoder()) return CUDA_ERROR_NOT_FOUND;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(Hkv) * d,
                              static_cast<cuuint64_t>(num_pages) * static_cast<cuuint64_t>(page_size)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(Hkv) * d};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(d), static_cast<cuuint32_t>(page_size < 128 ? page_size : 128)};
  const cuuint32_t estr[2] = {1u, 1u};
  return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

CUresult make_tile_map_e4m3(CUtensorMap* map, const void* base, int B, int N, int H, int d, int rows) {
  if (!encoder()) return CUDA_ERROR_NOT_FOUND;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(H),
                              static_cast<cuuint64_t>(B)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(H) * d, static_cast<cuuint64_t>(d),
                                 static_cast<cuuint64_t>(N) * H * d};
  const cuuint32_t box[4] = {128u, static_cast<cuuint32_t>(rows), 1u, 1u};
  const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

size_t bwd_workspace_base(int B, int H, int N, int d, int dtype) {
  if (check_shape(B, H, N, d, dtype) != FA_OK) return 0;
  if (static_cast<long long>(B) * H * N == 0) return 0;
  const size_t npad = (static_cast<size_t>(N) + 127) / 128 * 128;
  const size_t dq = align256(static_cast<size_t>(B) * N * H * d * sizeof(float));
  const size_t rows = align256(static_cast<size_t>(B) * H * npad * sizeof(float));
  return dq + 2 * rows;
}

CUresult make_kv_accum_map(CUtensorMap* map, float* base, int B, int N, int Hkv, int d) {
  if (!encoder()) return CUDA_ERROR_NOT_FOUND;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(Hkv),
                              static_cast<cuuint64_t>(B)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(Hkv) * d * 4, static_cast<cuuint64_t>(d) * 4,
                                 static_cast<cuuint64_t>(N) * Hkv * d * 4};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(d), d == 128 ? 64u : 128u, 1u, 1u};
  const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

CUresult make_dq_accum_map_sw128(CUtensorMap* map, float* base, int B, int N, int H, int d) {
  if (!encoder()) return CUDA_ERROR_NOT_FOUND;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(H),
                              static_cast<cuuint64_t>(B)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(H) * d * 4, static_cast<cuuint64_t>(d) * 4,
                                 static_cast<cuuint64_t>(N) * H * d * 4};
  const cuuint32_t box[4] = {32u, 128u, 1u, 1u};
  const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

CUresult make_dq_accum_map(CUtensorMap* map, float* base, int B, int N, int H, int d) {
  if (!encoder()) return CUDA_ERROR_NOT_FOUND;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(H),
                              static_cast<cuuint64_t>(B)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(H) * d * 4, static_cast<cuuint64_t>(d) * 4,
                                 static_cast<cuuint64_t>(N) * H * d * 4};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(d), 64u, 1u, 1u};
  const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

}  // namespace fa

using namespace fa;

extern "C" {

int fa_version(void) { return 100; }

const char* fa_status_string(int status) {
  switch (status) {
    case FA_OK: return "ok";
    case FA_ERR_INVALID_ARG: return "invalid argument (null pointer, negative size, bad scale or dtype)";
    case FA_ERR_UNSUPPORTED: return "unsupported configuration (head dim, dtype or pass)";
    case FA_ERR_MISALIGNED: return "tensor pointer not 16-byte aligned";
    case FA_ERR_WORKSPACE: return "backward workspace missing, too small or misaligned";
    case FA_ERR_ARCH: return "current CUDA device is not an sm_100 (B200-class) GPU";
    case FA_ERR_LAUNCH: return "CUDA call failed (see fa_last_cuda_error)";
    case FA_ERR_DEVICE_TIMEOUT: return "a kernel wait exceeded its limit; outputs of that launch are undefined";
    case FA_ERR_TOO_LARGE: return "problem exceeds a size limit";
    case FA_ERR_DEVICE_INPUT: return "device-side input out of range (sequence length or page index)";
    case FA_ERR_DEVICE_CHECK: return "a device-side bounds check of the checking build failed";
    default: return "unknown status";
  }
}

int fa_last_cuda_error(void) { return t_last_cuda_error; }

void fa_set_wait_limit_ms(int ms) {
  g_limit_ns.store(ms > 0 ? static_cast<unsigned long long>(ms) * 1000000ull : 0ull);
}

void fa_debug_inject(int mode) { g_inject.store(mode); }

void fa_set_kernel_events(void* start, void* stop) {
  t_ev_start = static_cast<cudaEvent_t>(start);
  t_ev_stop = static_cast<cudaEvent_t>(stop);
}

int fa_last_device_status(void* stream, int* detail) {
  DeviceState* st = nullptr;
  int rc = device_state(&st);
  if (rc) return rc;
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail_cuda(e);
  int v = 0;
  e = cudaMemcpy(&v, st->status, sizeof(int), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return fail_cuda(e);
  const int zero = 0;
  e = cudaMemcpy(st->status, &zero, sizeof(int), cudaMemcpyHostToDevice);
  if (e != cudaSuccess) return fail_cuda(e);
  if (detail) *detail = v;
  if (v & kDevCheck) return FA_ERR_DEVICE_CHECK;
  if (v & kDevBadInput) return FA_ERR_DEVICE_INPUT;
  return v ? FA_ERR_DEVICE_TIMEOUT : FA_OK;
}

}  // extern "C"

namespace {
// Block-sparse mask checks: mask_heads is 1 or H and the key-tile count fits the
// kernels' per-CTA list.  A null mask means no mask.  (Both dtypes take a mask in
// the forward; the backward refuses fp32 on its own.)
int check_mask(const uint8_t* mask, int mask_heads, int H, int N, int dtype) {
  (void)dtype;
  if (!mask) return FA_OK;
  if (mask_heads != 1 && mask_heads != H) return FA_ERR_INVALID_ARG;
  if ((N + 127) / 128 > kMaxSparseTiles) return FA_ERR_TOO_LARGE;
  return FA_OK;
}

int fwd_common(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H, int Hkv, int N, int d,
               float scale, int window_left, int window_right, const uint8_t* mask, int mask_heads, int dtype,
               void* stream) {
  int rc = check_shape(B, H, N, d, dtype);
  if (rc) return rc;
  if ((rc = check_kv_heads(H, Hkv))) return rc;
  if ((rc = check_window(window_left, window_right))) return rc;
  if ((rc = check_mask(mask, mask_heads, H, N, dtype))) return rc;
  if ((rc = check_scale(scale))) return rc;
  if (static_cast<long long>(B) * H * N == 0) return FA_OK;
  if (!Q || !K || !V || !O || !LSE) return FA_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O) || !aligned16(LSE)) return FA_ERR_MISALIGNED;
  DeviceState* st = nullptr;
  if ((rc = device_state(&st))) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  FwdArgs a;
  a.B = B;
  a.H = H;
  a.Hkv = Hkv;
  a.N = N;
  a.d = d;
  a.scale_log2 = scale * 1.4426950408889634f;
  set_window(window_left, window_right, &a.wl, &a.wr, &a.causal);
  a.O = O;
  a.LSE = LSE;
  a.block_mask = mask;
  a.mask_heads = mask_heads;
  a.nb = (N + 127) / 128;
  cudaError_t e;
  if (dtype == FA_FP32) {
    e = launch_fwd_f32(static_cast<const float*>(Q), static_cast<const float*>(K), static_cast<const float*>(V), a, s);
  } else {
    CUtensorMap tq, tk, tv, to;
    CUresult r;
    if ((r = make_tile_map(&tq, Q, B, N, H, d, 128)) != CUDA_SUCCESS ||
        (r = make_tile_map(&tk, K, B, N, Hkv, d, 128)) != CUDA_SUCCESS ||
        (r = make_tile_map(&tv, V, B, N, Hkv, d, 128)) != CUDA_SUCCESS ||
        (r = make_tile_map(&to, O, B, N, H, d, 128)) != CUDA_SUCCESS)
      return fail_encode(r);
    if (t_ev_start) cudaEventRecord(t_ev_start, s);
    e = launch_fwd_bf16(tq, tk, tv, to, a, make_ctl(*st), s);
    if (t_ev_stop && e == cudaSuccess) cudaEventRecord(t_ev_stop, s);
  }
  if (e != cudaSuccess) return fail_cuda(e);
  return FA_OK;
}

}  // namespace

extern "C" {

int fa_fwd_window(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H, int Hkv, int N,
                  int d, float scale, int window_left, int window_right, int dtype, void* stream) {
  return fwd_common(Q, K, V, O, LSE, B, H, Hkv, N, d, scale, window_left, window_right, nullptr, 0, dtype, stream);
}

int fa_fwd_blocksparse(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H, int Hkv, int N,
                       int d, float scale, int window_left, int window_right, const void* block_mask,
                       int mask_heads, int dtype, void* stream) {
  if (!block_mask && static_cast<long long>(B) * H * N > 0) return FA_ERR_INVALID_ARG;
  return fwd_common(Q, K, V, O, LSE, B, H, Hkv, N, d, scale, window_left, window_right,
                    static_cast<const uint8_t*>(block_mask), mask_heads, dtype, stream);
}

int fa_fwd_gqa(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H, int Hkv, int N, int d,
               float scale, int causal, int dtype, void* stream) {
  return fa_fwd_window(Q, K, V, O, LSE, B, H, Hkv, N, d, scale, -1, causal ? 0 : -1, dtype, stream);
}

int fa_fwd(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H, int N, int d, float scale,
           int causal, int dtype, void* stream) {
  return fa_fwd_window(Q, K, V, O, LSE, B, H, H, N, d, scale, -1, causal ? 0 : -1, dtype, stream);
}

int fa_fwd_fp8_blocksparse(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H, int Hkv,
                           int N, int d, float scale, float scale_q, float scale_k, float scale_v, int window_left,
                           int window_right, const void* block_mask, int mask_heads, void* stream) {
  int rc = check_shape(B, H, N, d, FA_BF16);
  if (rc) return rc;
  if (d != 128) return FA_ERR_UNSUPPORTED;
  if ((rc = check_kv_heads(H, Hkv))) return rc;
  if ((rc = check_window(window_left, window_right))) return rc;
  const uint8_t* mask = static_cast<const uint8_t*>(block_mask);
  if ((rc = check_mask(mask, mask_heads, H, N, FA_BF16))) return rc;
  if ((rc = check_scale(scale)) || (rc = check_scale(scale_q)) || (rc = check_scale(scale_k)) ||
      (rc = check_scale(scale_v)))
    return rc;
  if (static_cast<long long>(B) * H * N == 0) return FA_OK;
  if (!Q || !K || !V || !O || !LSE) return FA_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O) || !aligned16(LSE)) return FA_ERR_MISALIGNED;
  DeviceState* st = nullptr;
  if ((rc = device_state(&st))) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  FwdArgs a;
  a.B = B;
  a.H = H;
  a.Hkv = Hkv;
  a.N = N;
  a.d = d;
  // the per-tensor scales of Q and K fold into the softmax's exponent scale
  a.scale_log2 = static_cast<float>(static_cast<double>(scale) * scale_q * scale_k * 1.4426950408889634);
  set_window(window_left, window_right, &a.wl, &a.wr, &a.causal);
  a.O = O;
  a.LSE = LSE;
  a.block_mask = mask;
  a.mask_heads = mask ? mask_heads : 0;
  a.nb = (N + 127) / 128;
  CUtensorMap tq, tk, tv;
  CUresult r;
  if ((r = make_tile_map_e4m3(&tq, Q, B, N, H, d, 128)) != CUDA_SUCCESS ||
      (r = make_tile_map_e4m3(&tk, K, B, N, Hkv, d, 128)) != CUDA_SUCCESS ||
      (r = make_tile_map_e4m3(&tv, V, B, N, Hkv, d, 128)) != CUDA_SUCCESS)
    return fail_encode(r);
  if (t_ev_start) cudaEventRecord(t_ev_start, s);
  cudaError_t e = launch_fwd_fp8(tq, tk, tv, a, scale_v, make_ctl(*st), s);
  if (e != cudaSuccess) return fail_cuda(e);
  if (t_ev_stop) cudaEventRecord(t_ev_stop, s);
  return FA_OK;
}

int fa_fwd_fp8(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H, int Hkv, int N, int d,
               float scale, float scale_q, float scale_k, float scale_v, int window_left, int window_right,
               void* stream) {
  return fa_fwd_fp8_blocksparse(Q, K, V, O, LSE, B, H, Hkv, N, d, scale, scale_q, scale_k, scale_v, window_left,
                                window_right, nullptr, 0, stream);
}

size_t fa_bwd_workspace_size_gqa(int B, int H, int Hkv, int N, int d, int dtype) {
  if (check_kv_heads(H, Hkv) != FA_OK) return 0;
  const size_t base = fa::bwd_workspace_base(B, H, N, d, dtype);
  if (base == 0) return 0;
  // the accumulators whenever masked or unmasked walks of this shape would split
  const bool split = bwd_splits(B, H, Hkv, N, true) > 1 || bwd_splits(B, H, Hkv, N, false) > 1;
  const size_t kv = split ? 2 * align256(static_cast<size_t>(B) * N * Hkv * d * sizeof(float)) : 0;
  return base + kv;
}

size_t fa_bwd_workspace_size(int B, int H, int N, int d, int dtype) {
  return fa_bwd_workspace_size_gqa(B, H, H, N, d, dtype);
}

}  // extern "C"

namespace {
int bwd_common(const void* Q, const void* K, const void* V, const void* O, const void* dO, const float* LSE,
               void* dQ, void* dK, void* dV, int B, int H, int Hkv, int N, int d, float scale, int window_left,
               int window_right, const uint8_t* mask, int mask_heads, int dtype, void* workspace,
               size_t workspace_bytes, void* stream) {
  int rc = check_shape(B, H, N, d, dtype);
  if (rc) return rc;
  if ((rc = check_kv_heads(H, Hkv))) return rc;
  if ((rc = check_window(window_left, window_right))) return rc;
  if ((rc = check_mask(mask, mask_heads, H, N, dtype))) return rc;
  if ((rc = check_scale(scale))) return rc;
  if (dtype != FA_BF16) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * H * N == 0) return FA_OK;
  if (!Q || !K || !V || !O || !dO || !LSE || !dQ || !dK || !dV) return FA_ERR_INVALID_ARG;
  const void* ptrs[] = {Q, K, V, O, dO, LSE, dQ, dK, dV};
  for (const void* p : ptrs)
    if (!aligned16(p)) return FA_ERR_MISALIGNED;
  const size_t need = bwd_workspace_base(B, H, N, d, dtype);
  if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return FA_ERR_WORKSPACE;
  // split the walks when the grid is small and the workspace holds the fp32 dK / dV sums
  const bool masked = window_left >= 0 || window_right >= 0 || mask != nullptr;
  const int parts = (workspace_bytes >= fa_bwd_workspace_size_gqa(B, H, Hkv, N, d, dtype))
                        ? bwd_splits(B, H, Hkv, N, masked)
                        : 1;
  DeviceState* st = nullptr;
  if ((rc = device_state(&st))) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  const int npad = (N + 127) / 128 * 128;
  BwdArgs a;
  a.B = B;
  a.H = H;
  a.Hkv = Hkv;
  a.N = N;
  a.d = d;
  a.Npad = npad;
  a.scale = scale;
  a.scale_log2 = scale * 1.4426950408889634f;
  set_window(window_left, window_right, &a.wl, &a.wr, &a.causal);
  a.block_mask = mask;
  a.mask_heads = mask_heads;
  a.nb = (N + 127) / 128;
  a.O = O;
  a.dO = dO;
  a.LSE = LSE;
  a.dQ = dQ;
  a.dK = dK;
  a.dV = dV;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.dQacc = reinterpret_cast<float*>(ws);
  ws += align256(static_cast<size_t>(B) * N * H * d * sizeof(float));
  a.Dvec = reinterpret_cast<float*>(ws);
  ws += align256(static_cast<size_t>(B) * H * npad * sizeof(float));
  a.LSE2 = reinterpret_cast<float*>(ws);
  ws += align256(static_cast<size_t>(B) * H * npad * sizeof(float));
  a.splits = parts;
  a.dKacc = parts > 1 ? reinterpret_cast<float*>(ws) : nullptr;
  a.dVacc = parts > 1 ? reinterpret_cast<float*>(ws + align256(static_cast<size_t>(B) * N * Hkv * d * sizeof(float)))
                      : nullptr;

  CUtensorMap tq, tk, tv, tdo, tdq, tdk, tdv;
  CUresult r;
  if ((r = make_tile_map(&tq, Q, B, N, H, d, 128)) != CUDA_SUCCESS ||
      (r = make_tile_map(&tdo, dO, B, N, H, d, 128)) != CUDA_SUCCESS ||
      (r = make_tile_map(&tk, K, B, N, Hkv, d, 128)) != CUDA_SUCCESS ||
      (r = make_tile_map(&tv, V, B, N, Hkv, d, 128)) != CUDA_SUCCESS ||
      (r = (d == 128 ? make_dq_accum_map(&tdq, a.dQacc, B, N, H, d)
                     : make_dq_accum_map_sw128(&tdq, a.dQacc, B, N, H, d))) != CUDA_SUCCESS)
    return fail_encode(r);
  if (parts > 1) {
    if ((r = make_kv_accum_map(&tdk, a.dKacc, B, N, Hkv, d)) != CUDA_SUCCESS ||
        (r = make_kv_accum_map(&tdv, a.dVacc, B, N, Hkv, d)) != CUDA_SUCCESS)
      return fail_encode(r);
  } else {
    tdk = tdq;  // not read by the kernels without a split
    tdv = tdq;
  }
  cudaError_t e = launch_bwd_pre(a, s);
  if (e == cudaSuccess && parts > 1) e = launch_bwd_kv_zero(a, s);
  if (e != cudaSuccess) return fail_cuda(e);
  if (t_ev_start) cudaEventRecord(t_ev_start, s);
  e = (d == 128) ? launch_bwd_main(tq, tk, tv, tdo, tdq, tdk, tdv, a, make_ctl(*st), s)
                 : launch_bwd_main64(tq, tk, tv, tdo, tdq, tdk, tdv, a, make_ctl(*st), s);
  if (e != cudaSuccess) return fail_cuda(e);
  if (t_ev_stop) cudaEventRecord(t_ev_stop, s);
  e = launch_bwd_dq(a, s);
  if (e == cudaSuccess && parts > 1) e = launch_bwd_kv_convert(a, s);
  if (e != cudaSuccess) return fail_cuda(e);
  return FA_OK;
}

}  // namespace

extern "C" {

int fa_bwd_window(const void* Q, const void* K, const void* V, const void* O, const void* dO, const float* LSE,
                  void* dQ, void* dK, void* dV, int B, int H, int Hkv, int N, int d, float scale, int window_left,
                  int window_right, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
  return bwd_common(Q, K, V, O, dO, LSE, dQ, dK, dV, B, H, Hkv, N, d, scale, window_left, window_right, nullptr, 0,
                    dtype, workspace, workspace_bytes, stream);
}

int fa_bwd_blocksparse(const void* Q, const void* K, const void* V, const void* O, const void* dO, const float* LSE,
                       void* dQ, void* dK, void* dV, int B, int H, int Hkv, int N, int d, float scale,
                       int window_left, int window_right, const void* block_mask, int mask_heads, int dtype,
                       void* workspace, size_t workspace_bytes, void* stream) {
  if (!block_mask && static_cast<long long>(B) * H * N > 0) return FA_ERR_INVALID_ARG;
  return bwd_common(Q, K, V, O, dO, LSE, dQ, dK, dV, B, H, Hkv, N, d, scale, window_left, window_right,
                    static_cast<const uint8_t*>(block_mask), mask_heads, dtype, workspace, workspace_bytes, stream);
}

int fa_bwd_gqa(const void* Q, const void* K, const void* V, const void* O, const void* dO, const float* LSE,
               void* dQ, void* dK, void* dV, int B, int H, int Hkv, int N, int d, float scale, int causal, int dtype,
               void* workspace, size_t workspace_bytes, void* stream) {
  return fa_bwd_window(Q, K, V, O, dO, LSE, dQ, dK, dV, B, H, Hkv, N, d, scale, -1, causal ? 0 : -1, dtype,
                       workspace, workspace_bytes, stream);
}

int fa_bwd(const void* Q, const void* K, const void* V, const void* O, const void* dO, const float* LSE, void* dQ,
           void* dK, void* dV, int B, int H, int N, int d, float scale, int causal, int dtype, void* workspace,
           size_t workspace_bytes, void* stream) {
  return fa_bwd_window(Q, K, V, O, dO, LSE, dQ, dK, dV, B, H, H, N, d, scale, -1, causal ? 0 : -1, dtype,
                       workspace, workspace_bytes, stream);
}

int fa_merge_partial(float* O_acc, float* LSE_acc, const void* O_part, const float* LSE_part, void* O_out, int B,
                     int H, int N, int d, int init, void* stream) {
  int rc = check_shape(B, H, N, d, FA_BF16);
  if (rc) return rc;
  if (static_cast<long long>(B) * H * N == 0) return FA_OK;
  if (!O_acc || !LSE_acc || !O_part || !LSE_part) return FA_ERR_INVALID_ARG;
  if (!aligned16(O_acc) || !aligned16(O_part) || (O_out && !aligned16(O_out)) ||
      (reinterpret_cast<uintptr_t>(LSE_acc) & 3u) || (reinterpret_cast<uintptr_t>(LSE_part) & 3u))
    return FA_ERR_MISALIGNED;
  DeviceState* st = nullptr;
  if ((rc = device_state(&st))) return rc;
  cudaError_t e = launch_merge(O_acc, LSE_acc, O_part, LSE_part, O_out, B, H, N, d, init ? 1 : 0,
                               static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail_cuda(e);
  return FA_OK;
}

int fa_accumulate_bf16(float* acc, const void* part, long long n, int init, void* stream) {
  if (n < 0 || n % 8 != 0) return FA_ERR_INVALID_ARG;
  if (n == 0) return FA_OK;
  if (!acc || !part) return FA_ERR_INVALID_ARG;
  if (!aligned16(acc) || !aligned16(part)) return FA_ERR_MISALIGNED;
  DeviceState* st = nullptr;
  int rc = device_state(&st);
  if (rc) return rc;
  cudaError_t e = launch_accumulate(acc, part, n, init ? 1 : 0, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail_cuda(e);
  return FA_OK;
}

int fa_cast_bf16(void* out, const float* in, long long n, void* stream) {
  if (n < 0 || n % 8 != 0) return FA_ERR_INVALID_ARG;
  if (n == 0) return FA_OK;
  if (!out || !in) return FA_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(in)) return FA_ERR_MISALIGNED;
  DeviceState* st = nullptr;
  int rc = device_state(&st);
  if (rc) return rc;
  cudaError_t e = launch_cast(out, in, n, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail_cuda(e);
  return FA_OK;
}

}  // extern "C"

// ---------------------------------------------------------------------------
// One decode step over a paged KV cache
// ---------------------------------------------------------------------------
namespace {

struct DecodePlan {
  int hgroups, splits, chunk;
  size_t ws;  // workspace bytes the plan needs (0 with one chunk)
};

bool pow2_in(int x, int lo, int hi) { return x >= lo && x <= hi && (x & (x - 1)) == 0; }

int check_decode(int B, int H, int Hkv, int d, int page_size, int num_pages, int max_pages, float scale) {
  if (B < 0 || H < 1 || num_pages < 1 || max_pages < 1) return FA_ERR_INVALID_ARG;
  int rc = check_kv_heads(H, Hkv);
  if (rc) return rc;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (!pow2_in(page_size, 8, 4096)) return FA_ERR_UNSUPPORTED;
  if ((rc = check_scale(scale))) return rc;
  const long long hg = (H / Hkv + 15) / 16;
  if (static_cast<long long>(num_pages) * page_size > 0x7fffffffLL ||
      static_cast<long long>(max_pages) * page_size > 0x7fffffffLL || B > 65535 || Hkv * hg > 65535)
    return FA_ERR_TOO_LARGE;
  return FA_OK;
}

size_t decode_ws_bytes(int B, int H, int d, int splits) {
  if (splits <= 1) return 0;
  const size_t rows = static_cast<size_t>(splits) * B * H;
  return align256(rows * d * sizeof(float)) + align256(rows * sizeof(float));
}

// Chunks per (sequence, head group).  Each CTA pays a fixed start (length and
// page checks, the first loads in flight) and end (merge of its warps), so chunks
// hold at least 512 KB of K/V (16 tiles at d = 128, 32 at d = 64).  A batch with
// fewer (sequence, head group) pairs than CTA slots (148 SMs x 2) is split into
// about two waves of CTAs; a larger batch into about four, the later waves'
// chunks being the short or empty ends of the sequences.  No more chunks than
// the workspace holds.
DecodePlan decode_plan(int B, int H, int Hkv, int d, int page_size, int max_pages, size_t ws_cap) {
  DecodePlan p;
  p.hgroups = (H / Hkv + 15) / 16;
  const long long max_keys = static_cast<long long>(max_pages) * page_size;
  const long long tiles = (max_keys + 63) / 64;
  const long long ctas = static_cast<long long>(B) * Hkv * p.hgroups;
  const long long slots = 2 * 148;
  const long long waves = 4;  // for batches that fill the slots
  const long long min_tiles = d == 128 ? 16 : 32;
  // a small batch: two waves (one wave suits equal lengths best, but a long
  // sequence among shorter ones then runs alone at the end)
  const long long w = ctas < slots ? 2 : waves;
  long long want = ctas <= 0 ? 1 : (w * slots + ctas - 1) / ctas;
  want = std::max(1LL, std::min({want, tiles / min_tiles, 65535LL}));
  for (;;) {
    const long long chunk_tiles = (tiles + want - 1) / want;
    p.splits = static_cast<int>((tiles + chunk_tiles - 1) / chunk_tiles);
    p.chunk = static_cast<int>(chunk_tiles * 64);
    p.ws = decode_ws_bytes(B, H, d, p.splits);
    if (p.splits == 1 || p.ws <= ws_cap) break;
    want = p.splits - 1;
  }
  return p;
}

}  // namespace

extern "C" {

size_t fa_decode_workspace_size(int B, int H, int Hkv, int d, int page_size, int max_pages) {
  if (check_decode(B, H, Hkv, d, page_size, 1, max_pages, 1.0f) != FA_OK) return 0;
  return decode_plan(B, H, Hkv, d, page_size, max_pages, SIZE_MAX).ws;
}

int fa_decode_paged(const void* Q, const void* K_cache, const void* V_cache, const int* block_table,
                    const int* seqlens, void* O, float* LSE, int B, int H, int Hkv, int d, int page_size,
                    int num_pages, int max_pages, float scale, void* workspace, size_t workspace_bytes,
                    void* stream) {
  int rc = check_decode(B, H, Hkv, d, page_size, num_pages, max_pages, scale);
  if (rc) return rc;
  if (B == 0) return FA_OK;
  if (!Q || !K_cache || !V_cache || !block_table || !seqlens || !O || !LSE) return FA_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(K_cache) || !aligned16(V_cache) || !aligned16(O) ||
      (reinterpret_cast<uintptr_t>(LSE) & 3u) || (reinterpret_cast<uintptr_t>(block_table) & 3u) ||
      (reinterpret_cast<uintptr_t>(seqlens) & 3u))
    return FA_ERR_MISALIGNED;
  if (workspace && !aligned16(workspace)) return FA_ERR_WORKSPACE;
  DeviceState* st = nullptr;
  if ((rc = device_state(&st))) return rc;
  const DecodePlan plan = decode_plan(B, H, Hkv, d, page_size, max_pages, workspace ? workspace_bytes : 0);
  DecodeArgs a;
  a.B = B;
  a.H = H;
  a.Hkv = Hkv;
  a.d = d;
  a.page_size = page_size;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.hgroups = plan.hgroups;
  a.splits = plan.splits;
  a.chunk = plan.chunk;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.Q = Q;
  a.block_table = block_table;
  a.seqlens = seqlens;
  a.O = O;
  a.LSE = LSE;
  const size_t rows = static_cast<size_t>(plan.splits) * B * H;
  a.Opart = plan.splits > 1 ? static_cast<float*>(workspace) : nullptr;
  a.LSEpart = plan.splits > 1 ? reinterpret_cast<float*>(static_cast<char*>(workspace) + align256(rows * d * 4))
                              : nullptr;
  CUtensorMap tk, tv;
  CUresult r;
  if ((r = make_paged_map(&tk, K_cache, num_pages, page_size, Hkv, d)) != CUDA_SUCCESS ||
      (r = make_paged_map(&tv, V_cache, num_pages, page_size, Hkv, d)) != CUDA_SUCCESS)
    return fail_encode(r);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (t_ev_start) cudaEventRecord(t_ev_start, s);
  cudaError_t e = launch_decode(tk, tv, a, make_ctl(*st), s);
  if (t_ev_stop && e == cudaSuccess) cudaEventRecord(t_ev_stop, s);
  if (e != cudaSuccess) return fail_cuda(e);
  return FA_OK;
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Norm and rotation of query and key heads
// ---------------------------------------------------------------------------
namespace {

constexpr int kRopeBlockWarps = 4;
constexpr int kRopeBwdBlocks = 148 * 3;  // resident together
constexpr int kRopePairs = 148 * 5 * 4 * 2;  // row groups (of 512 / d heads) of the warps resident together, two each
// Row groups of a warp in one round.  Backward, bf16 d128: B4 N8192 H32 + 8 160 us with 4, 166 with
// 8; B1 N16384 H32 + 32 130 and 133; d64 B8 N4096 H32 + 32 129 and 128.  Forward: B1 N4096 H64 + 8
// 25.8 and 25.5, N2048 H32 + 8 8.5 and 7.8 (a position's start costs it more).
constexpr int kRopeFwdRound = 8;
constexpr int kRopeBwdRound = 4;

bool aligned_strides(const long long* s, int dtype) {
  const long long m = dtype == FA_BF16 ? 8 : 4;  // 16 bytes
  return s == nullptr || (s[0] % m == 0 && s[1] % m == 0 && s[2] % m == 0);
}

void set_strides(const long long* s, int N, int heads, int d, long long* sb, long long* sn, long long* sh) {
  *sh = s ? s[2] : d;
  *sn = s ? s[1] : static_cast<long long>(heads) * d;
  *sb = s ? s[0] : static_cast<long long>(N) * heads * d;
}

int check_rope(const void* Q, const void* K, const void* wq, const void* wk, const float* cos_t, const float* sin_t,
               const void* Qo, const void* Ko, const int* positions, int B, int N, int H, int Hkv, int d,
               int table_rows, float eps, int interleaved, int dtype, int weight_dtype) {
  int rc = check_shape(B, H, N, d, dtype);
  if (rc) return rc;
  if (Hkv < 0 || table_rows < 0) return FA_ERR_INVALID_ARG;
  if (Hkv > 65535 || static_cast<long long>(B) * N > 0x7fffffffLL ||
      static_cast<double>(B) * N * Hkv * d >= 1099511627776.0)  // 2^40
    return FA_ERR_TOO_LARGE;
  if ((interleaved != 0 && interleaved != 1) || (weight_dtype != FA_BF16 && weight_dtype != FA_FP32))
    return FA_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.f) return FA_ERR_INVALID_ARG;
  if ((wq == nullptr) != (wk == nullptr)) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * N == 0 || H + Hkv == 0) return FA_OK;
  if (!positions && N > table_rows) return FA_ERR_INVALID_ARG;
  if ((H > 0 && (!Q || !Qo)) || (Hkv > 0 && (!K || !Ko)) || !cos_t || !sin_t) return FA_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(Qo) || !aligned16(Ko) || !aligned16(wq) || !aligned16(wk) ||
      !aligned16(cos_t) || !aligned16(sin_t) || (reinterpret_cast<uintptr_t>(positions) & 3u))
    return FA_ERR_MISALIGNED;
  return FA_OK;
}

RopeArgs rope_args(const void* Q, const void* K, const void* wq, const void* wk, const float* cos_t, const float* sin_t,
                   const int* positions, void* Qo, void* Ko, int B, int N, int H, int Hkv, int d,
                   const long long* qs, const long long* ks, int table_rows, float eps, int interleaved,
                   int weight_dtype, int* status) {
  RopeArgs a = {};
  a.q.x = Q;
  a.k.x = K;
  set_strides(qs, N, H, d, &a.q.sb, &a.q.sn, &a.q.sh);
  set_strides(ks, N, Hkv, d, &a.k.sb, &a.k.sn, &a.k.sh);
  a.q.out = Qo;
  a.k.out = Ko;
  a.q.w = wq;
  a.k.w = wk;
  a.cos_t = cos_t;
  a.sin_t = sin_t;
  a.positions = positions;
  a.tokens = B * N;
  a.N = N;
  a.H = H;
  a.Hkv = Hkv;
  a.table = table_rows;
  a.interleaved = interleaved;
  a.w_f32 = weight_dtype == FA_FP32;
  a.eps = eps;
  a.status = status;
  const int rows = 512 / d;
  a.q_groups = (H + rows - 1) / rows;
  a.k_groups = (Hkv + rows - 1) / rows;
  return a;
}

// Blocks that walk the row groups in rounds: as many as fill the GPU, shared between q
// and k by their work.
void rope_rounds(RopeArgs* a, int per, long long most) {
  a->per = per;
  // two row groups or more a warp
  const long long qu = static_cast<long long>(a->tokens) * a->q_groups, ku = static_cast<long long>(a->tokens) * a->k_groups;
  const int least = 2 * kRopeBlockWarps;
  const long long qw = (qu + least - 1) / least, kw = (ku + least - 1) / least;
  if (qw + kw <= most) {
    a->q_blocks = static_cast<int>(qw);
    a->blocks = static_cast<int>(qw + kw);
    return;
  }
  // by their row groups, and one more for each position's start
  const long long qc = a->q_groups + (a->H > 0), kc = a->k_groups + (a->Hkv > 0);
  const long long want = std::max<long long>(a->H ? 1 : 0, most * qc / (qc + kc));
  a->q_blocks = static_cast<int>(std::min(qw, std::min<long long>(want, most - (a->Hkv ? 1 : 0))));
  a->blocks = a->q_blocks + static_cast<int>(std::min(kw, most - a->q_blocks));
}

}  // namespace

extern "C" {

int fa_qk_norm_rope(const void* Q, const void* K, const void* q_weight, const void* k_weight, const float* cos_table,
                    const float* sin_table, const int* positions, void* Q_out, void* K_out, int B, int N, int H,
                    int Hkv, int d, const long long* q_strides, const long long* k_strides, int table_rows, float eps,
                    int interleaved, int dtype, int weight_dtype, void* stream) {
  int rc = check_rope(Q, K, q_weight, k_weight, cos_table, sin_table, Q_out, K_out, positions, B, N, H, Hkv, d,
                      table_rows, eps, interleaved, dtype, weight_dtype);
  if (rc) return rc;
  if (static_cast<long long>(B) * N == 0 || H + Hkv == 0) return FA_OK;
  if (!aligned_strides(q_strides, dtype) || !aligned_strides(k_strides, dtype)) return FA_ERR_MISALIGNED;
  DeviceState* st = nullptr;
  if ((rc = device_state(&st))) return rc;
  RopeArgs a = rope_args(Q, K, q_weight, k_weight, cos_table, sin_table, positions, Q_out, K_out, B, N, H, Hkv, d,
                               q_strides, k_strides, table_rows, eps, interleaved, weight_dtype, st->status);
  const long long groups = static_cast<long long>(a.tokens) * (a.q_groups + a.k_groups);
  if (groups >= kRopePairs) {
    // B1 H32 + 8 d128 bf16: 5120 groups (N512) 3.5 us against 3.2 by pairs; 7000 (N700) 4.0
    // against 4.5, 20480 (N2048) 7.7 against 9.3.  From 256 MB on three blocks per SM, because
    // memory takes more requests in flight badly: B4 N8192 H32 + 8 (671 MB) 111 us against 122 with
    // four, B1 N16384 H32 + 32 (537 MB) 86 against 97, B2 N8192 H32 + 8 (336 MB) 57 against 60;
    // B1 N4096 H64 + 8 (151 MB) 27.4 against 25.5.
    const double bytes = 2.0 * a.tokens * (H + Hkv) * d * (dtype == FA_FP32 ? 4 : 2);
    rope_rounds(&a, kRopeFwdRound, bytes < 256e6 ? 148 * 4 : 148 * 3);
  } else {  // pairs of groups, a warp each
    a.q_groups = (a.q_groups + 1) / 2;
    a.k_groups = (a.k_groups + 1) / 2;
  }
  const cudaError_t e = launch_rope_fwd(a, d, dtype == FA_FP32, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : fail_cuda(e);
}

size_t fa_qk_norm_rope_workspace_size(int d) {
  if (d != 64 && d != 128) return 0;
  return align256(static_cast<size_t>(kRopeBwdBlocks) * d * sizeof(float));
}

int fa_qk_norm_rope_bwd(const void* Q, const void* K, const void* q_weight, const void* k_weight,
                        const float* cos_table, const float* sin_table, const int* positions, const void* dQ_out,
                        const void* dK_out, void* dQ, void* dK, void* dq_weight, void* dk_weight, int B, int N, int H,
                        int Hkv, int d, const long long* q_strides, const long long* k_strides,
                        const long long* dq_out_strides, const long long* dk_out_strides, int table_rows, float eps,
                        int interleaved, int dtype, int weight_dtype, void* workspace, size_t workspace_bytes,
                        void* stream) {
  int rc = check_rope(Q, K, q_weight, k_weight, cos_table, sin_table, dQ, dK, positions, B, N, H, Hkv, d, table_rows,
                      eps, interleaved, dtype, weight_dtype);
  if (rc) return rc;
  const bool norm = q_weight != nullptr;
  const bool empty = static_cast<long long>(B) * N == 0 || H + Hkv == 0;
  if (!norm && empty) return FA_OK;
  if (norm && (!dq_weight || !dk_weight)) return FA_ERR_INVALID_ARG;
  if (!empty && ((H > 0 && !dQ_out) || (Hkv > 0 && !dK_out))) return FA_ERR_INVALID_ARG;
  if (!aligned16(dQ_out) || !aligned16(dK_out) || !aligned16(dq_weight) || !aligned16(dk_weight) ||
      !aligned_strides(q_strides, dtype) || !aligned_strides(k_strides, dtype) ||
      !aligned_strides(dq_out_strides, dtype) || !aligned_strides(dk_out_strides, dtype))
    return FA_ERR_MISALIGNED;
  if (norm && (!workspace || workspace_bytes < fa_qk_norm_rope_workspace_size(d) ||
               (reinterpret_cast<uintptr_t>(workspace) & 255u)))
    return FA_ERR_WORKSPACE;
  DeviceState* st = nullptr;
  if ((rc = device_state(&st))) return rc;
  RopeArgs a = rope_args(Q, K, q_weight, k_weight, cos_table, sin_table, positions, dQ, dK, B, N, H, Hkv, d, q_strides,
                         k_strides, table_rows, eps, interleaved, weight_dtype, st->status);
  a.q.g = dQ_out;
  a.k.g = dK_out;
  set_strides(dq_out_strides, N, H, d, &a.q.gb, &a.q.gn, &a.q.gh);
  set_strides(dk_out_strides, N, Hkv, d, &a.k.gb, &a.k.gn, &a.k.gh);
  if (!empty) rope_rounds(&a, kRopeBwdRound, kRopeBwdBlocks);
  a.partial = static_cast<float*>(workspace);
  a.dwq = dq_weight;
  a.dwk = dk_weight;
  const cudaError_t e = launch_rope_bwd(a, d, dtype == FA_FP32, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : fail_cuda(e);
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Paged cache: writing new tokens, reading cached positions, 8-bit decode
// ---------------------------------------------------------------------------
namespace {

int check_cache(const void* K_cache, const void* V_cache, const void* kv_scale, const int* block_table,
                const int* lengths, int B, int N, int Hkv, int d, int page_size, int num_pages, int max_pages,
                int fp8) {
  if (B < 0 || N < 0 || Hkv < 1 || num_pages < 1 || max_pages < 1 || (fp8 != 0 && fp8 != 1)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (!pow2_in(page_size, 8, 4096)) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_pages) * page_size > 0x7fffffffLL ||
      static_cast<long long>(max_pages) * page_size > (1LL << 30) || N > (1 << 30) || B > 65535 || Hkv > 65535)
    return FA_ERR_TOO_LARGE;
  // one warp per (sequence, 512 / d positions, head)
  const long long groups = (static_cast<long long>(N) * d + 511) / 512;
  if (static_cast<double>(B) * groups * Hkv >= 4294967296.0) return FA_ERR_TOO_LARGE;
  if (B == 0 || N == 0) return FA_OK;
  if (!K_cache || !V_cache || !block_table || !lengths || (fp8 && !kv_scale)) return FA_ERR_INVALID_ARG;
  if (!aligned16(K_cache) || !aligned16(V_cache) || (fp8 && !aligned16(kv_scale)) ||
      (reinterpret_cast<uintptr_t>(block_table) & 3u) || (reinterpret_cast<uintptr_t>(lengths) & 3u))
    return FA_ERR_MISALIGNED;
  return FA_OK;
}

// An append's warp takes up to 8 groups of positions, as long as that leaves every SM its 64
// warps: the rows behind a prompt's end then cost few warps that only look up a count
// (8 prompts of 0 to 4096 tokens, 8 heads, d = 128: 17.4 us, 20.7 with one group a
// warp, 23 with half as many warps).  A read writes the rows behind the end, too: one group.
constexpr long long kCacheWarps = 148LL * 64;
constexpr int kAppendGroups = 8;

CacheArgs cache_args(void* K_cache, void* V_cache, void* kv_scale, const int* block_table, const int* lengths, int B,
                     int N, int Hkv, int d, int page_size, int num_pages, int max_pages, int most, int* status) {
  CacheArgs a = {};
  a.t[0].pool = K_cache;
  a.t[1].pool = V_cache;
  a.kv_scale = static_cast<uint8_t*>(kv_scale);
  a.block_table = block_table;
  a.start = lengths;
  a.N = N;
  a.Hkv = Hkv;
  a.page_size = page_size;
  while ((1 << a.page_shift) < page_size) ++a.page_shift;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  const long long groups = (static_cast<long long>(N) * d + 511) / 512;
  a.per = static_cast<int>(std::max(1LL, std::min<long long>(most, B * groups * Hkv / kCacheWarps)));
  a.groups = static_cast<unsigned int>((groups + a.per - 1) / a.per);
  a.units = static_cast<unsigned int>(B) * a.groups * static_cast<unsigned int>(Hkv);
  a.status = status;
  return a;
}

}  // namespace

extern "C" {

int fa_cache_append(const void* K, const void* V, void* K_cache, void* V_cache, void* kv_scale, const int* block_table,
                    const int* start, const int* count, int B, int N, int Hkv, int d, const long long* k_strides,
                    const long long* v_strides, int page_size, int num_pages, int max_pages, int fp8, void* stream) {
  int rc = check_cache(K_cache, V_cache, kv_scale, block_table, start, B, N, Hkv, d, page_size, num_pages, max_pages, fp8);
  if (rc) return rc;
  if (B == 0 || N == 0) return FA_OK;
  if (!K || !V) return FA_ERR_INVALID_ARG;
  if (!aligned16(K) || !aligned16(V) || !aligned_strides(k_strides, FA_BF16) || !aligned_strides(v_strides, FA_BF16) ||
      (reinterpret_cast<uintptr_t>(count) & 3u))
    return FA_ERR_MISALIGNED;
  DeviceState* st = nullptr;
  if ((rc = device_state(&st))) return rc;
  CacheArgs a = cache_args(K_cache, V_cache, kv_scale, block_table, start, B, N, Hkv, d, page_size, num_pages,
                           max_pages, kAppendGroups, st->status);
  a.t[0].x = K;
  a.t[1].x = V;
  set_strides(k_strides, N, Hkv, d, &a.t[0].sb, &a.t[0].sn, &a.t[0].sh);
  set_strides(v_strides, N, Hkv, d, &a.t[1].sb, &a.t[1].sn, &a.t[1].sh);
  a.count = count;
  const cudaError_t e = launch_cache(a, d, fp8 != 0, true, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : fail_cuda(e);
}

int fa_cache_read(const void* K_cache, const void* V_cache, const void* kv_scale, const int* block_table,
                  const int* seqlens, void* K, void* V, int B, int N, int Hkv, int d, int page_size, int num_pages,
                  int max_pages, int fp8, void* stream) {
  int rc = check_cache(K_cache, V_cache, kv_scale, block_table, seqlens, B, N, Hkv, d, page_size, num_pages, max_pages,
                       fp8);
  if (rc) return rc;
  if (B == 0 || N == 0) return FA_OK;
  if (!K || !V) return FA_ERR_INVALID_ARG;
  if (!aligned16(K) || !aligned16(V)) return FA_ERR_MISALIGNED;
  DeviceState* st = nullptr;
  if ((rc = device_state(&st))) return rc;
  CacheArgs a = cache_args(const_cast<void*>(K_cache), const_cast<void*>(V_cache), const_cast<void*>(kv_scale),
                           block_table, seqlens, B, N, Hkv, d, page_size, num_pages, max_pages, 1, st->status);
  a.t[0].out = K;
  a.t[1].out = V;
  const cudaError_t e = launch_cache(a, d, fp8 != 0, false, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : fail_cuda(e);
}

}  // extern "C"

namespace {

struct Decode8Plan {
  int nt, hgroups, ranges;
  size_t ws;
};

int check_decode8(int B, int H, int Hkv, int d, int page_size, int num_pages, int max_pages, float scale, int window) {
  int rc = check_decode(B, H, Hkv, d, page_size, num_pages, max_pages, scale);
  if (rc) return rc;
  if (window < -1) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(max_pages) * page_size > (1LL << 30)) return FA_ERR_TOO_LARGE;
  // the kernel counts the tiles of all sequences in an int
  if (static_cast<long long>(B) * ((static_cast<long long>(max_pages) * page_size + 127) / 128) > (1LL << 30))
    return FA_ERR_TOO_LARGE;
  return FA_OK;
}

// A lone CTA takes 1.2 us for a tile; cutting a list into ranges and joining them costs 3 us
// more than one CTA per sequence (measured, one sequence, 8 K/V heads, d = 128: 3 tiles
// 7.1 us whole and 7.6 in ranges of one tile, 4 tiles 8.3 and 7.7, 16 tiles 23 and 8.6).
constexpr int kDecode8WholeTiles = 3;

size_t decode8_ws_bytes(int H, int d, int ranges) {
  const size_t rows = static_cast<size_t>(ranges) * 2 * H;
  return align256(rows * d * sizeof(float)) + align256(rows * sizeof(float)) + align256(ranges * sizeof(int4));
}

// How the tiles (128 positions) of all sequences are shared out.  Where no table row
// holds more than kDecode8WholeTiles, or the workspace holds no two ranges, one CTA takes
// one sequence of one head group.  Else as many ranges as CTAs fit on the GPU beside one
// another.
Decode8Plan decode8_plan(int B, int H, int Hkv, int d, int page_size, int max_pages, int window, size_t ws_cap) {
  Decode8Plan p = {};
  const int G = H / Hkv;
  p.nt = G <= 8 ? 1 : 2;
  p.hgroups = (G + 8 * p.nt - 1) / (8 * p.nt);
  long long span = static_cast<long long>(max_pages) * page_size;
  // a window's first position lies anywhere in its first tile
  if (window >= 0) span = std::min(span, static_cast<long long>(window) + 1 + 127);
  const long long tiles = (span + 127) / 128;
  const long long slots = 148LL * fa::decode_fp8_ctas_per_sm(d, p.nt);
  const long long per_range = static_cast<long long>(Hkv) * p.hgroups;
  if (tiles <= kDecode8WholeTiles || B == 0) return p;
  long long want = std::max(1LL, slots / per_range);
  want = std::min({want, tiles * B, 65535LL});
  while (want > 1 && decode8_ws_bytes(H, d, static_cast<int>(want)) > ws_cap) --want;
  if (want < 2) return p;
  p.ranges = static_cast<int>(want);
  p.ws = decode8_ws_bytes(H, d, p.ranges);
  return p;
}

}  // namespace

extern "C" {

size_t fa_decode_fp8_workspace_size(int B, int H, int Hkv, int d, int page_size, int max_pages, int window_left) {
  if (check_decode8(B, H, Hkv, d, page_size, 1, max_pages, 1.0f, window_left) != FA_OK) return 0;
  return decode8_plan(B, H, Hkv, d, page_size, max_pages, window_left, SIZE_MAX).ws;
}

int fa_decode_paged_fp8(const void* Q, const void* K_cache, const void* V_cache, const void* kv_scale,
                        const int* block_table, const int* seqlens, void* O, float* LSE, int B, int H, int Hkv, int d,
                        int page_size, int num_pages, int max_pages, float scale, int window_left, void* workspace,
                        size_t workspace_bytes, void* stream) {
  int rc = check_decode8(B, H, Hkv, d, page_size, num_pages, max_pages, scale, window_left);
  if (rc) return rc;
  if (B == 0) return FA_OK;
  if (!Q || !K_cache || !V_cache || !kv_scale || !block_table || !seqlens || !O || !LSE) return FA_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(K_cache) || !aligned16(V_cache) || !aligned16(kv_scale) || !aligned16(O) ||
      (reinterpret_cast<uintptr_t>(LSE) & 3u) || (reinterpret_cast<uintptr_t>(block_table) & 3u) ||
      (reinterpret_cast<uintptr_t>(seqlens) & 3u))
    return FA_ERR_MISALIGNED;
  if (workspace && !aligned16(workspace)) return FA_ERR_WORKSPACE;
  DeviceState* st = nullptr;
  if ((rc = device_state(&st))) return rc;
  const Decode8Plan plan =
      decode8_plan(B, H, Hkv, d, page_size, max_pages, window_left, workspace ? workspace_bytes : 0);
  Decode8Args a = {};
  a.B = B;
  a.H = H;
  a.Hkv = Hkv;
  a.page_size = page_size;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.hgroups = plan.hgroups;
  a.ranges = plan.ranges;
  a.window = window_left;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.Q = Q;
  a.kv_scale = static_cast<const uint8_t*>(kv_scale);
  a.block_table = block_table;
  a.seqlens = seqlens;
  a.O = O;
  a.LSE = LSE;
  if (plan.ranges) {
    const size_t rows = static_cast<size_t>(plan.ranges) * 2 * H;
    char* ws = static_cast<char*>(workspace);
    a.Opart = reinterpret_cast<float*>(ws);
    ws += align256(rows * d * sizeof(float));
    a.LSEpart = reinterpret_cast<float*>(ws);
    a.borders = reinterpret_cast<int4*>(ws + align256(rows * sizeof(float)));
  }
  CUtensorMap tk, tv;
  CUresult r;
  if ((r = make_paged_map_u8(&tk, K_cache, num_pages, page_size, Hkv, d)) != CUDA_SUCCESS ||
      (r = make_paged_map_u8(&tv, V_cache, num_pages, page_size, Hkv, d)) != CUDA_SUCCESS)
    return fail_encode(r);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (t_ev_start) cudaEventRecord(t_ev_start, s);
  cudaError_t e = launch_decode_fp8(tk, tv, a, d, plan.nt, make_ctl(*st), s);
  if (t_ev_stop && e == cudaSuccess) cudaEventRecord(t_ev_stop, s);
  if (e != cudaSuccess) return fail_cuda(e);
  return FA_OK;
}

}  // extern "C"
