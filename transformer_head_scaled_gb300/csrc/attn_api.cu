// attn_api.cu -- the library's C ABI (declared in include/attn.h): argument
// checks, per-device set-up, TMA tensor-map encoding and kernel dispatch.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cstdint>
#include <cmath>
#include <mutex>

#include "attn.h"
#include "attn_internal.cuh"

namespace attn {
namespace {

// Errors a kernel finds (a bounded wait that ran out) are recorded here, one
// word per device, and read back by attn_check().
__device__ int g_status;

constexpr int kMaxDevices = 64;
constexpr uint64_t kDefaultLimitNs = 2000000000ull;

// attn_fwd_host splits the batch into at most this many slices, so that the
// copies of one slice overlap the kernel and the copies of its neighbours.
constexpr int kHostSlices = 8;
// Copy streams per direction (slices alternate between them); two measured no
// faster than one: the host link, not the copy engines, sets the rate.
constexpr int kCopyStreams = 1;

struct DeviceInfo {
  bool ready = false;
  bool supported = false;
  int num_sms = 0;
  int* status = nullptr;
  // attn_fwd_host: copy-in and copy-out streams and the events that order
  // them with the caller's stream (created on first use; issued under
  // host_mu so that concurrent callers do not share an event in flight).
  cudaStream_t copy_in[kCopyStreams] = {}, copy_out[kCopyStreams] = {};
  cudaEvent_t ev_start = nullptr, ev_done[kCopyStreams] = {};
  cudaEvent_t ev_in[kHostSlices] = {}, ev_kernel[kHostSlices] = {};
  std::mutex host_mu;
};

std::mutex g_mu;
DeviceInfo g_dev[kMaxDevices];
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::atomic<uint64_t> g_limit_ns{kDefaultLimitNs};
std::atomic<uint64_t> g_launches{0};
std::atomic<int> g_last_cuda_error{0};

int cuda_fail(cudaError_t e) {
  g_last_cuda_error.store(static_cast<int>(e));
  return ATTN_ERR_CUDA;
}

// Per-device set-up on first use: SM count, architecture check, address of
// the status word, the driver's tensor-map encoder.
int device_info(DeviceInfo** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= kMaxDevices) return ATTN_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceInfo& di = g_dev[dev];
  if (!di.ready) {
    int major = 0, minor = 0, sms = 0;
    if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess)
      return cuda_fail(e);
    if ((e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess)
      return cuda_fail(e);
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
      return cuda_fail(e);
    di.supported = (major == 10 && minor == 3);  // the kernels are built for sm_103a only
    di.num_sms = sms;
    if (di.supported) {
      void* addr = nullptr;
      if ((e = cudaGetSymbolAddress(&addr, g_status)) != cudaSuccess) return cuda_fail(e);
      di.status = static_cast<int*>(addr);
    }
    if (g_encode == nullptr) {
      void* fn = nullptr;
      cudaDriverEntryPointQueryResult q;
      e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                           &q);
      if (e != cudaSuccess) return cuda_fail(e);
      if (q != cudaDriverEntryPointSuccess || fn == nullptr) return cuda_fail(cudaErrorNotSupported);
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    di.ready = true;
  }
  if (!di.supported) return ATTN_ERR_UNSUPPORTED;
  *out = &di;
  return ATTN_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_common(const void* q, const void* k, const void* v, const void* o, const float* lse,
                 int B, int h, int n_q, int n_k, int d_k, float scale, int mask_kind,
                 const int* key_lens, size_t elem) {
  if (!q || !k || !v || !o) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return ATTN_ERR_INVALID_ARG;
  if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)) return ATTN_ERR_INVALID_ARG;
  if (B < 1 || h < 1 || n_q < 1 || n_k < 1 || d_k < 1) return ATTN_ERR_INVALID_ARG;
  if (!(std::isfinite(scale) && scale > 0.f)) return ATTN_ERR_INVALID_ARG;
  if (mask_kind != ATTN_MASK_NONE && mask_kind != ATTN_MASK_CAUSAL &&
      mask_kind != ATTN_MASK_KEY_PADDING)
    return ATTN_ERR_INVALID_ARG;
  if (mask_kind == ATTN_MASK_KEY_PADDING &&
      (key_lens == nullptr || (reinterpret_cast<uintptr_t>(key_lens) & 3u)))
    return ATTN_ERR_INVALID_ARG;
  // Index arithmetic: B*h fits a TMA coordinate and a grid; every tensor
  // stays below 2^40 bytes (the TMA stride limit).
  const long long bh = static_cast<long long>(B) * h;
  if (bh > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
  const long long n = n_q > n_k ? n_q : n_k;
  if (bh * n * d_k * static_cast<long long>(elem) >= (1LL << 40)) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

// (d, n, B*H) fp32 view with a (min(d, 32), 64, 1) box in the swizzle of its
// 4*min(d, 32)-byte rows (the backward's dQ accumulator, added into by TMA
// reduce).
int encode_3d_f32(CUtensorMap* map, const void* base, int d, int n, long long bh) {
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(n),
                        static_cast<cuuint64_t>(bh)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 4,
                           static_cast<cuuint64_t>(d) * 4 * static_cast<cuuint64_t>(n)};
  const int inner = d < 32 ? d : 32;
  cuuint32_t box[3] = {static_cast<cuuint32_t>(inner), 64u, 1u};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  const CUtensorMapSwizzle swz = inner == 32   ? CU_TENSOR_MAP_SWIZZLE_128B
                                 : inner == 16 ? CU_TENSOR_MAP_SWIZZLE_64B
                                               : CU_TENSOR_MAP_SWIZZLE_32B;
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? ATTN_OK : cuda_fail(cudaErrorInvalidValue);
}

// Head sizes the tensor-core forward covers.
bool tc_head_size(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

// Element strides of a [B, h, n, d] tensor view (d contiguous).
using Strides = RowStrides;

Strides bhsd(int h, int n, int d) {
  return Strides{static_cast<long long>(h) * n * d, static_cast<long long>(n) * d, d};
}

// A stride the TMA can use: positive and a multiple of 16 bytes.
bool stride_ok(long long elems) {
  return elems > 0 && (elems * 2) % 16 == 0 && elems * 2 < (1LL << 40);
}

// (d, n, h, B) bf16 view with the given strides and a (min(d, 64), rows, 1, 1)
// box in the widest swizzle its 2*min(d, 64)-byte rows fit.
int encode_4d(CUtensorMap* map, const void* base, int d, int n, int h, int B, Strides st,
              int box_rows) {
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(n),
                        static_cast<cuuint64_t>(h), static_cast<cuuint64_t>(B)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(st.n) * 2, static_cast<cuuint64_t>(st.h) * 2,
                           static_cast<cuuint64_t>(st.b) * 2};
  const int inner = d < 64 ? d : 64;
  const CUtensorMapSwizzle swz = inner == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
                                 : inner == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                               : CU_TENSOR_MAP_SWIZZLE_32B;
  cuuint32_t box[4] = {static_cast<cuuint32_t>(inner), static_cast<cuuint32_t>(box_rows), 1u, 1u};
  cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ERR_INVALID_ARG;
}

// The forward's four maps: Q and O with 128-row boxes, K and V with the key
// tile of this head size.  st = strides of q, k, v, o, or null for
// contiguous [B, h, n, d].
int encode_fwd_maps(CUtensorMap* tmq, CUtensorMap* tmk, CUtensorMap* tmv, CUtensorMap* tmo,
                    const void* q, const void* k, const void* v, const void* o, int d, int n_q,
                    int n_k, int h, int B, const Strides* st) {
  const int kv_rows = fwd_tc_kv_rows(d);
  const Strides sq = st ? st[0] : bhsd(h, n_q, d), sk = st ? st[1] : bhsd(h, n_k, d),
                sv = st ? st[2] : bhsd(h, n_k, d), so = st ? st[3] : bhsd(h, n_q, d);
  int rc;
  if ((rc = encode_4d(tmq, q, d, n_q, h, B, sq, 128)) != ATTN_OK) return rc;
  if ((rc = encode_4d(tmk, k, d, n_k, h, B, sk, kv_rows)) != ATTN_OK) return rc;
  if ((rc = encode_4d(tmv, v, d, n_k, h, B, sv, kv_rows)) != ATTN_OK) return rc;
  return encode_4d(tmo, o, d, n_q, h, B, so, 128);
}

int encode_2d(CUtensorMap* map, const void* base) {
  cuuint64_t dims[2] = {64, 128};
  cuuint64_t strides[1] = {128};
  cuuint32_t box[2] = {64, 128};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? ATTN_OK : cuda_fail(cudaErrorInvalidValue);
}

// Scratch for attn_decode_noalloc: a fixed-size array in the library's own
// device memory, created when the library's module is loaded on a device and
// kept until the process exits.  Host code only knows the symbol; the device
// address is looked up once per device (scratch_on_device) and handed to the
// kernels as a plain pointer.
static __device__ __align__(256) unsigned char g_decode_scratch[ATTN_DECODE_NOALLOC_SCRATCH_BYTES];
void* g_scratch_addr[kMaxDevices] = {};

// Device address of g_decode_scratch on the current device (looked up on the
// first call per device, under the set-up lock).
int scratch_on_device(void** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= kMaxDevices) return ATTN_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_mu);
  if (g_scratch_addr[dev] == nullptr) {
    void* addr = nullptr;
    if ((e = cudaGetSymbolAddress(&addr, g_decode_scratch)) != cudaSuccess) return cuda_fail(e);
    if (addr == nullptr) return cuda_fail(cudaErrorInvalidSymbol);
    g_scratch_addr[dev] = addr;
  }
  *out = g_scratch_addr[dev];
  return ATTN_OK;
}

// K and V caches with 128-key boxes, then with 32-key boxes for partial tiles.
int encode_decode_maps(CUtensorMap* maps, const void* k_cache, const void* v_cache, int d_k,
                       int L_max, int B, int h, Strides sk, Strides sv) {
  int rc;
  if ((rc = encode_4d(&maps[0], k_cache, d_k, L_max, h, B, sk, 128)) != ATTN_OK) return rc;
  if ((rc = encode_4d(&maps[1], v_cache, d_k, L_max, h, B, sv, 128)) != ATTN_OK) return rc;
  if ((rc = encode_4d(&maps[2], k_cache, d_k, L_max, h, B, sk, 32)) != ATTN_OK) return rc;
  return encode_4d(&maps[3], v_cache, d_k, L_max, h, B, sv, 32);
}

// Device staging of attn_fwd_host: Q, K, V, O (bf16), LSE (fp32) and the key
// lengths (int32), each at a 256-byte boundary, for the whole batch.
struct HostLayout {
  size_t q, k, v, o, lse, lens, bytes;
};

HostLayout host_layout(int B, int h, int n_q, int n_k, int d) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const size_t bh = static_cast<size_t>(B) * h;
  HostLayout l;
  size_t off = 0;
  l.q = off;
  off += up(bh * n_q * d * 2);
  l.k = off;
  off += up(bh * n_k * d * 2);
  l.v = off;
  off += up(bh * n_k * d * 2);
  l.o = off;
  off += up(bh * n_q * d * 2);
  l.lse = off;
  off += up(bh * n_q * 4);
  l.lens = off;
  off += up(static_cast<size_t>(B) * 4);
  l.bytes = off;
  return l;
}

// The copy streams and events of attn_fwd_host, created once per device.
int host_streams(DeviceInfo* di) {
  std::lock_guard<std::mutex> lock(g_mu);
  if (di->copy_in[0] != nullptr) return ATTN_OK;
  cudaError_t e;
  cudaStream_t st[2 * kCopyStreams];
  for (int i = 0; i < 2 * kCopyStreams; ++i)
    if ((e = cudaStreamCreateWithFlags(&st[i], cudaStreamNonBlocking)) != cudaSuccess)
      return cuda_fail(e);
  cudaEvent_t* evs[1 + kCopyStreams + 2 * kHostSlices];
  int n = 0;
  evs[n++] = &di->ev_start;
  for (int i = 0; i < kCopyStreams; ++i) evs[n++] = &di->ev_done[i];
  for (int i = 0; i < kHostSlices; ++i) {
    evs[n++] = &di->ev_in[i];
    evs[n++] = &di->ev_kernel[i];
  }
  for (int i = 0; i < n; ++i)
    if ((e = cudaEventCreateWithFlags(evs[i], cudaEventDisableTiming)) != cudaSuccess)
      return cuda_fail(e);
  for (int i = kCopyStreams - 1; i >= 0; --i) {
    di->copy_out[i] = st[kCopyStreams + i];
    di->copy_in[i] = st[i];  // copy_in[0] last: marks the set as complete
  }
  return ATTN_OK;
}

LaunchCtx make_ctx(const DeviceInfo& di, cudaStream_t stream) {
  LaunchCtx ctx;
  ctx.num_sms = di.num_sms;
  ctx.limit_ns = g_limit_ns.load();
  ctx.status = di.status;
  ctx.stream = stream;
  return ctx;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

int attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int h,
             int n_q, int n_k, int d_k, float scale, int mask_kind, const int* key_lens,
             struct CUstream_st* stream) {
  int rc = check_common(q, k, v, o, lse, B, h, n_q, n_k, d_k, scale, mask_kind, key_lens, 2);
  if (rc != ATTN_OK) return rc;
  if (!tc_head_size(d_k)) return ATTN_ERR_UNSUPPORTED;
  DeviceInfo* di = nullptr;
  if ((rc = device_info(&di)) != ATTN_OK) return rc;
  CUtensorMap tmq, tmk, tmv, tmo;
  if ((rc = encode_fwd_maps(&tmq, &tmk, &tmv, &tmo, q, k, v, o, d_k, n_q, n_k, h, B, nullptr)) !=
      ATTN_OK)
    return rc;
  Problem pb{q, k, v, o, lse, B, h, n_q, n_k, d_k, scale, mask_kind,
             mask_kind == ATTN_MASK_KEY_PADDING ? key_lens : nullptr};
  cudaError_t e = launch_fwd_tc(pb, tmq, tmk, tmv, tmo, make_ctx(*di, stream));
  if (e != cudaSuccess) return cuda_fail(e);
  g_launches.fetch_add(1);
  return ATTN_OK;
}

int attn_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int B, int h,
                    int n_q, int n_k, int d_k, float scale, int window_left, int window_right,
                    struct CUstream_st* stream) {
  int rc = check_common(q, k, v, o, lse, B, h, n_q, n_k, d_k, scale, ATTN_MASK_NONE, nullptr, 2);
  if (rc != ATTN_OK) return rc;
  if (window_left < 0 || window_right < 0) return ATTN_ERR_INVALID_ARG;
  if (!tc_head_size(d_k)) return ATTN_ERR_UNSUPPORTED;
  DeviceInfo* di = nullptr;
  if ((rc = device_info(&di)) != ATTN_OK) return rc;
  CUtensorMap tmq, tmk, tmv, tmo;
  if ((rc = encode_fwd_maps(&tmq, &tmk, &tmv, &tmo, q, k, v, o, d_k, n_q, n_k, h, B, nullptr)) !=
      ATTN_OK)
    return rc;
  // a side longer than both sequences changes nothing; clamping keeps the
  // kernel's index arithmetic within int
  const int reach = n_q + n_k;
  Problem pb{q, k, v, o, lse, B, h, n_q, n_k, d_k, scale, kMaskBand, nullptr,
             window_left < reach ? window_left : reach, window_right < reach ? window_right : reach};
  cudaError_t e = launch_fwd_tc(pb, tmq, tmk, tmv, tmo, make_ctx(*di, stream));
  if (e != cudaSuccess) return cuda_fail(e);
  g_launches.fetch_add(1);
  return ATTN_OK;
}

int attn_fwd_strided(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                     int h, int n_q, int n_k, int d_k, const int64_t* q_strides,
                     const int64_t* k_strides, const int64_t* v_strides, const int64_t* o_strides,
                     float scale, int mask_kind, const int* key_lens, int window_left,
                     int window_right, struct CUstream_st* stream) {
  if (!q || !k || !v || !o) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return ATTN_ERR_INVALID_ARG;
  if (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)) return ATTN_ERR_INVALID_ARG;
  if (B < 1 || h < 1 || n_q < 1 || n_k < 1 || d_k < 1) return ATTN_ERR_INVALID_ARG;
  if (!(std::isfinite(scale) && scale > 0.f)) return ATTN_ERR_INVALID_ARG;
  if (mask_kind < ATTN_MASK_NONE || mask_kind > ATTN_MASK_WINDOW) return ATTN_ERR_INVALID_ARG;
  if (mask_kind == ATTN_MASK_KEY_PADDING &&
      (key_lens == nullptr || (reinterpret_cast<uintptr_t>(key_lens) & 3u)))
    return ATTN_ERR_INVALID_ARG;
  if (mask_kind == ATTN_MASK_WINDOW && (window_left < 0 || window_right < 0))
    return ATTN_ERR_INVALID_ARG;
  if (!q_strides || !k_strides || !v_strides || !o_strides) return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * h > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
  Strides st[4];
  const int64_t* in[4] = {q_strides, k_strides, v_strides, o_strides};
  for (int i = 0; i < 4; ++i) {
    st[i] = Strides{in[i][0], in[i][1], in[i][2]};
    if (!stride_ok(st[i].b) || !stride_ok(st[i].h) || !stride_ok(st[i].n))
      return ATTN_ERR_INVALID_ARG;
  }
  if (!tc_head_size(d_k)) return ATTN_ERR_UNSUPPORTED;
  DeviceInfo* di = nullptr;
  int rc;
  if ((rc = device_info(&di)) != ATTN_OK) return rc;
  CUtensorMap tmq, tmk, tmv, tmo;
  if ((rc = encode_fwd_maps(&tmq, &tmk, &tmv, &tmo, q, k, v, o, d_k, n_q, n_k, h, B, st)) !=
      ATTN_OK)
    return rc;
  const int reach = n_q + n_k;
  Problem pb{q, k, v, o, lse, B, h, n_q, n_k, d_k, scale,
             mask_kind == ATTN_MASK_WINDOW ? static_cast<int>(kMaskBand) : mask_kind,
             mask_kind == ATTN_MASK_KEY_PADDING ? key_lens : nullptr,
             window_left < reach ? window_left : reach, window_right < reach ? window_right : reach};
  cudaError_t e = launch_fwd_tc(pb, tmq, tmk, tmv, tmo, make_ctx(*di, stream));
  if (e != cudaSuccess) return cuda_fail(e);
  g_launches.fetch_add(1);
  return ATTN_OK;
}

size_t attn_fwd_host_buffer_bytes(int B, int h, int n_q, int n_k, int d_k) {
  if (B < 1 || h < 1 || n_q < 1 || n_k < 1 || !tc_head_size(d_k)) return 0;
  if (static_cast<long long>(B) * h > 0x7fffffffLL) return 0;
  return host_layout(B, h, n_q, n_k, d_k).bytes;
}

int attn_fwd_host(const void* q, const void* k, const void* v, void* o, float* lse, int B, int h,
                  int n_q, int n_k, int d_k, float scale, int mask_kind, const int* key_lens,
                  int window_left, int window_right, void* dev_buf, size_t dev_buf_bytes,
                  struct CUstream_st* stream) {
  const bool window = mask_kind == ATTN_MASK_WINDOW;
  if (mask_kind < ATTN_MASK_NONE || mask_kind > ATTN_MASK_WINDOW) return ATTN_ERR_INVALID_ARG;
  if (window && (window_left < 0 || window_right < 0)) return ATTN_ERR_INVALID_ARG;
  if (!q || !k || !v || !o) return ATTN_ERR_INVALID_ARG;
  if (mask_kind == ATTN_MASK_KEY_PADDING && key_lens == nullptr) return ATTN_ERR_INVALID_ARG;
  // sizes, scale and the device-side limits, checked as for attn_fwd on the
  // staging buffer (the host buffers need no alignment)
  const void* stage = dev_buf;
  int rc = check_common(stage, stage, stage, stage, nullptr, B, h, n_q, n_k, d_k, scale,
                        mask_kind == ATTN_MASK_KEY_PADDING ? ATTN_MASK_KEY_PADDING : ATTN_MASK_NONE,
                        static_cast<const int*>(stage), 2);
  if (rc != ATTN_OK) return rc;
  if (reinterpret_cast<uintptr_t>(dev_buf) & 255u) return ATTN_ERR_INVALID_ARG;
  if (!tc_head_size(d_k)) return ATTN_ERR_UNSUPPORTED;
  const HostLayout lay = host_layout(B, h, n_q, n_k, d_k);
  if (dev_buf_bytes < lay.bytes) return ATTN_ERR_INVALID_ARG;
  DeviceInfo* di = nullptr;
  if ((rc = device_info(&di)) != ATTN_OK) return rc;
  if ((rc = host_streams(di)) != ATTN_OK) return rc;
  std::lock_guard<std::mutex> lock(di->host_mu);

  uint8_t* dbuf = static_cast<uint8_t*>(dev_buf);
  const size_t qrow = static_cast<size_t>(h) * n_q * d_k * 2;  // bytes of one batch entry
  const size_t krow = static_cast<size_t>(h) * n_k * d_k * 2;
  const size_t lrow = static_cast<size_t>(h) * n_q * 4;
  const bool padding = mask_kind == ATTN_MASK_KEY_PADDING;
  const int reach = n_q + n_k;
  const int slices = B < kHostSlices ? B : kHostSlices;
  cudaError_t e;
  // the staging buffer and the host buffers may still be in use by work
  // enqueued earlier on the caller's stream
  if ((e = cudaEventRecord(di->ev_start, stream)) != cudaSuccess) return cuda_fail(e);
  for (int i = 0; i < kCopyStreams; ++i) {
    if ((e = cudaStreamWaitEvent(di->copy_in[i], di->ev_start, 0)) != cudaSuccess)
      return cuda_fail(e);
    if ((e = cudaStreamWaitEvent(di->copy_out[i], di->ev_start, 0)) != cudaSuccess)
      return cuda_fail(e);
  }
  const cudaMemcpyKind h2d = cudaMemcpyHostToDevice, d2h = cudaMemcpyDeviceToHost;
  for (int s = 0; s < slices; ++s) {
    const int b0 = static_cast<int>(static_cast<long long>(B) * s / slices);
    const int b1 = static_cast<int>(static_cast<long long>(B) * (s + 1) / slices);
    const int nb = b1 - b0;
    uint8_t* dq = dbuf + lay.q + b0 * qrow;
    uint8_t* dk = dbuf + lay.k + b0 * krow;
    uint8_t* dv = dbuf + lay.v + b0 * krow;
    uint8_t* dout = dbuf + lay.o + b0 * qrow;
    float* dlse = reinterpret_cast<float*>(dbuf + lay.lse + b0 * lrow);
    int* dlens = reinterpret_cast<int*>(dbuf + lay.lens) + b0;
    cudaStream_t copy_in = di->copy_in[s % kCopyStreams];
    cudaStream_t copy_out = di->copy_out[s % kCopyStreams];
    // copy in (one copy per tensor slice)
    if ((e = cudaMemcpyAsync(dq, static_cast<const uint8_t*>(q) + b0 * qrow, nb * qrow, h2d,
                             copy_in)) != cudaSuccess)
      return cuda_fail(e);
    if ((e = cudaMemcpyAsync(dk, static_cast<const uint8_t*>(k) + b0 * krow, nb * krow, h2d,
                             copy_in)) != cudaSuccess)
      return cuda_fail(e);
    if ((e = cudaMemcpyAsync(dv, static_cast<const uint8_t*>(v) + b0 * krow, nb * krow, h2d,
                             copy_in)) != cudaSuccess)
      return cuda_fail(e);
    if (padding && (e = cudaMemcpyAsync(dlens, key_lens + b0, nb * sizeof(int), h2d, copy_in)) !=
                       cudaSuccess)
      return cuda_fail(e);
    if ((e = cudaEventRecord(di->ev_in[s], copy_in)) != cudaSuccess) return cuda_fail(e);
    // the forward of this slice on the caller's stream
    if ((e = cudaStreamWaitEvent(stream, di->ev_in[s], 0)) != cudaSuccess) return cuda_fail(e);
    CUtensorMap tmq, tmk, tmv, tmo;
    if ((rc = encode_fwd_maps(&tmq, &tmk, &tmv, &tmo, dq, dk, dv, dout, d_k, n_q, n_k, h, nb,
                              nullptr)) != ATTN_OK)
      return rc;
    Problem pb{dq, dk, dv, dout, lse ? dlse : nullptr, nb, h, n_q, n_k, d_k, scale,
               window ? static_cast<int>(kMaskBand) : mask_kind, padding ? dlens : nullptr,
               window_left < reach ? window_left : reach,
               window_right < reach ? window_right : reach};
    if ((e = launch_fwd_tc(pb, tmq, tmk, tmv, tmo, make_ctx(*di, stream))) != cudaSuccess)
      return cuda_fail(e);
    g_launches.fetch_add(1);
    if ((e = cudaEventRecord(di->ev_kernel[s], stream)) != cudaSuccess) return cuda_fail(e);
    // copy out
    if ((e = cudaStreamWaitEvent(copy_out, di->ev_kernel[s], 0)) != cudaSuccess) return cuda_fail(e);
    if ((e = cudaMemcpyAsync(static_cast<uint8_t*>(o) + b0 * qrow, dout, nb * qrow, d2h,
                             copy_out)) != cudaSuccess)
      return cuda_fail(e);
    if (lse && (e = cudaMemcpyAsync(reinterpret_cast<uint8_t*>(lse) + b0 * lrow, dlse, nb * lrow,
                                    d2h, copy_out)) != cudaSuccess)
      return cuda_fail(e);
  }
  // the caller's stream resumes once every copy out is done
  for (int i = 0; i < kCopyStreams; ++i) {
    if ((e = cudaEventRecord(di->ev_done[i], di->copy_out[i])) != cudaSuccess) return cuda_fail(e);
    if ((e = cudaStreamWaitEvent(stream, di->ev_done[i], 0)) != cudaSuccess) return cuda_fail(e);
  }
  return ATTN_OK;
}

int attn_fwd_f32(const float* q, const float* k, const float* v, float* o, float* lse, int B,
                 int h, int n_q, int n_k, int d_k, float scale, int mask_kind,
                 const int* key_lens, struct CUstream_st* stream) {
  int rc = check_common(q, k, v, o, lse, B, h, n_q, n_k, d_k, scale, mask_kind, key_lens, 4);
  if (rc != ATTN_OK) return rc;
  if (d_k != 16 && d_k != 32 && d_k != 64 && d_k != 128) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * h > 65535) return ATTN_ERR_UNSUPPORTED;  // grid.y
  DeviceInfo* di = nullptr;
  if ((rc = device_info(&di)) != ATTN_OK) return rc;
  Problem pb{q, k, v, o, lse, B, h, n_q, n_k, d_k, scale, mask_kind,
             mask_kind == ATTN_MASK_KEY_PADDING ? key_lens : nullptr};
  cudaError_t e = launch_fwd_f32(pb, make_ctx(*di, stream));
  if (e != cudaSuccess) return cuda_fail(e);
  g_launches.fetch_add(1);
  return ATTN_OK;
}

size_t attn_decode_workspace_bytes(int B, int h, int n_q, int L_max, int d_k) {
  if (B < 1 || h < 1 || n_q < 1 || n_q > kDecodeMaxQueries || L_max < 1 || !tc_head_size(d_k))
    return 0;
  DeviceInfo* di = nullptr;
  if (device_info(&di) != ATTN_OK) return 0;
  return decode_plan(B, h, n_q, L_max, d_k, di->num_sms).workspace_bytes;
}

size_t attn_decode_window_workspace_bytes(int B, int h, int n_q, int L_max, int d_k, int window) {
  if (window < 0) return 0;
  // the splits cover the window's keys only
  return attn_decode_workspace_bytes(B, h, n_q, window < L_max ? window + 1 : L_max, d_k);
}

}  // extern "C"

namespace attn {
namespace {
// st: strides of q, k_cache, v_cache, o, or null for contiguous tensors.
// scratch_noalloc: take the partials' space from the library's own array
// instead of the caller's workspace.  window: restricted self-attention
// (keys [len - 1 - window, len)), or -1 for all cached keys.
static int decode_impl(const void* q, const void* k_cache, const void* v_cache, void* o,
                       float* lse, int B, int h, int n_q, int L_max, int d_k, const Strides* st,
                       float scale, const int* cache_lens, void* workspace,
                       size_t workspace_bytes, bool scratch_noalloc, struct CUstream_st* stream,
                       int window = -1) {
  int rc = check_common(q, k_cache, v_cache, o, lse, B, h, n_q, L_max, d_k, scale,
                        ATTN_MASK_NONE, nullptr, 2);
  if (rc != ATTN_OK) return rc;
  if (cache_lens && (reinterpret_cast<uintptr_t>(cache_lens) & 3u)) return ATTN_ERR_INVALID_ARG;
  if (!tc_head_size(d_k) || n_q > kDecodeMaxQueries) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * h > 65535) return ATTN_ERR_UNSUPPORTED;  // grid.y
  DeviceInfo* di = nullptr;
  if ((rc = device_info(&di)) != ATTN_OK) return rc;
  // the most keys one query sees: what the cache is split by
  const int seen = window >= 0 && window < L_max ? window + 1 : L_max;
  const DecodePlan plan = decode_plan(B, h, n_q, seen, d_k, di->num_sms);
  if (scratch_noalloc) {
    if (plan.workspace_bytes > ATTN_DECODE_NOALLOC_SCRATCH_BYTES)
      return ATTN_ERR_SCRATCH_TOO_SMALL;
    // only a split cache writes partials: the array is not touched otherwise
    workspace = nullptr;
    if (plan.workspace_bytes > 0 && (rc = scratch_on_device(&workspace)) != ATTN_OK) return rc;
  } else if (plan.workspace_bytes > 0 && (workspace == nullptr ||
                                          workspace_bytes < plan.workspace_bytes ||
                                          !aligned16(workspace))) {
    return ATTN_ERR_INVALID_ARG;
  }
  const Strides sq = st ? st[0] : bhsd(h, n_q, d_k), sk = st ? st[1] : bhsd(h, L_max, d_k),
                sv = st ? st[2] : bhsd(h, L_max, d_k), so = st ? st[3] : bhsd(h, n_q, d_k);
  CUtensorMap maps[4];
  if (d_k == 64 &&
      (rc = encode_decode_maps(maps, k_cache, v_cache, d_k, L_max, B, h, sk, sv)) != ATTN_OK)
    return rc;
  DecodeProblem pb{q,  k_cache, v_cache, o,          lse, B,  h,  n_q, L_max,
                   d_k, scale,  cache_lens, sq, sk, sv, so, window};
  cudaError_t e = launch_decode(pb, maps, plan, static_cast<float*>(workspace),
                                make_ctx(*di, stream));
  if (e != cudaSuccess) return cuda_fail(e);
  g_launches.fetch_add(plan.splits > 1 ? 2 : 1);
  return ATTN_OK;
}
}  // namespace
}  // namespace attn

extern "C" {

int attn_decode(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                int B, int h, int n_q, int L_max, int d_k, float scale, const int* cache_lens,
                void* workspace, size_t workspace_bytes, struct CUstream_st* stream) {
  return decode_impl(q, k_cache, v_cache, o, lse, B, h, n_q, L_max, d_k, nullptr, scale,
                     cache_lens, workspace, workspace_bytes, false, stream);
}

int attn_decode_window(const void* q, const void* k_cache, const void* v_cache, void* o,
                       float* lse, int B, int h, int n_q, int L_max, int d_k, float scale,
                       const int* cache_lens, int window, void* workspace,
                       size_t workspace_bytes, struct CUstream_st* stream) {
  if (window < 0) return ATTN_ERR_INVALID_ARG;
  return decode_impl(q, k_cache, v_cache, o, lse, B, h, n_q, L_max, d_k, nullptr, scale,
                     cache_lens, workspace, workspace_bytes, false, stream, window);
}

int attn_decode_noalloc(const void* q, const void* k_cache, const void* v_cache, void* o,
                        float* lse, int B, int h, int n_q, int L_max, int d_k, float scale,
                        const int* cache_lens, struct CUstream_st* stream) {
  return decode_impl(q, k_cache, v_cache, o, lse, B, h, n_q, L_max, d_k, nullptr, scale,
                     cache_lens, nullptr, 0, true, stream);
}

int attn_decode_strided(const void* q, const void* k_cache, const void* v_cache, void* o,
                        float* lse, int B, int h, int n_q, int L_max, int d_k,
                        const int64_t* strides, float scale, const int* cache_lens,
                        void* workspace, size_t workspace_bytes, struct CUstream_st* stream) {
  if (strides == nullptr) return ATTN_ERR_INVALID_ARG;
  Strides st[4];
  for (int i = 0; i < 4; ++i) {
    st[i] = Strides{strides[3 * i], strides[3 * i + 1], strides[3 * i + 2]};
    if (!stride_ok(st[i].b) || !stride_ok(st[i].h) || !stride_ok(st[i].n))
      return ATTN_ERR_INVALID_ARG;
  }
  return decode_impl(q, k_cache, v_cache, o, lse, B, h, n_q, L_max, d_k, st, scale, cache_lens,
                     workspace, workspace_bytes, false, stream);
}

size_t attn_bwd_workspace_bytes(int B, int h, int n_q, int d_k) {
  if (B < 1 || h < 1 || n_q < 1 || !bwd_head_size_ok(d_k)) return 0;
  if (static_cast<long long>(B) * h > 0x7fffffffLL) return 0;
  return bwd_layout(B, h, n_q, d_k).bytes;
}

}  // extern "C"

namespace attn {
namespace {
// st: strides of q, k, v, o, dout, dq, dk, dv, or null for contiguous
// [B, h, n, d] tensors.
static int bwd_impl(const void* q, const void* k, const void* v, const void* o, const void* dout,
                    const float* lse, void* dq, void* dk, void* dv, int B, int h, int n_q,
                    int n_k, int d_k, const Strides* st, float scale, int mask_kind,
                    const int* key_lens, int window_left, int window_right, void* workspace,
                    size_t workspace_bytes, struct CUstream_st* stream) {
  const bool window = mask_kind == kMaskBand;
  int rc = check_common(q, k, v, o, lse, B, h, n_q, n_k, d_k, scale,
                        window ? ATTN_MASK_NONE : mask_kind, key_lens, 2);
  if (rc != ATTN_OK) return rc;
  if (!dout || !lse || !dq || !dk || !dv || !workspace) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(dout) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv) ||
      !aligned16(workspace))
    return ATTN_ERR_INVALID_ARG;
  if (!bwd_head_size_ok(d_k)) return ATTN_ERR_UNSUPPORTED;
  const BwdLayout lay = bwd_layout(B, h, n_q, d_k);
  if (workspace_bytes < lay.bytes) return ATTN_ERR_INVALID_ARG;
  DeviceInfo* di = nullptr;
  if ((rc = device_info(&di)) != ATTN_OK) return rc;
  const long long bh = static_cast<long long>(B) * h;
  const Strides rq = bhsd(h, n_q, d_k), rk = bhsd(h, n_k, d_k);
  const Strides sq = st ? st[0] : rq, sk = st ? st[1] : rk, sv = st ? st[2] : rk,
                so = st ? st[3] : rq, sdo = st ? st[4] : rq, sdq = st ? st[5] : rq,
                sdk = st ? st[6] : rk, sdv = st ? st[7] : rk;
  CUtensorMap maps[8];
  if ((rc = encode_4d(&maps[0], q, d_k, n_q, h, B, sq, 128)) != ATTN_OK) return rc;
  if ((rc = encode_4d(&maps[1], k, d_k, n_k, h, B, sk, 128)) != ATTN_OK) return rc;
  if ((rc = encode_4d(&maps[2], v, d_k, n_k, h, B, sv, 128)) != ATTN_OK) return rc;
  if ((rc = encode_4d(&maps[3], dout, d_k, n_q, h, B, sdo, 128)) != ATTN_OK) return rc;
  if ((rc = encode_4d(&maps[4], dk, d_k, n_k, h, B, sdk, 64)) != ATTN_OK) return rc;
  if ((rc = encode_4d(&maps[5], dv, d_k, n_k, h, B, sdv, 64)) != ATTN_OK) return rc;
  if ((rc = encode_3d_f32(&maps[6], static_cast<uint8_t*>(workspace) + lay.dq_acc_off, d_k, n_q,
                          bh)) != ATTN_OK)
    return rc;
  maps[7] = maps[6];  // used with changed scores only
  const int reach = n_q + n_k;
  BwdProblem pb{q, k, v, o, dout, lse, dq, dk, dv, B, h, n_q, n_k, d_k, scale, mask_kind,
                mask_kind == ATTN_MASK_KEY_PADDING ? key_lens : nullptr,
                window_left < reach ? window_left : reach,
                window_right < reach ? window_right : reach, so, sdo, sdq};
  cudaError_t e = launch_bwd(pb, maps, workspace, make_ctx(*di, stream));
  if (e != cudaSuccess) return cuda_fail(e);
  g_launches.fetch_add(3);
  return ATTN_OK;
}
}  // namespace
}  // namespace attn

extern "C" {

int attn_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout,
             const float* lse, void* dq, void* dk, void* dv, int B, int h, int n_q, int n_k,
             int d_k, float scale, int mask_kind, const int* key_lens, void* workspace,
             size_t workspace_bytes, struct CUstream_st* stream) {
  if (mask_kind == ATTN_MASK_WINDOW) return ATTN_ERR_INVALID_ARG;  // attn_bwd_window
  return bwd_impl(q, k, v, o, dout, lse, dq, dk, dv, B, h, n_q, n_k, d_k, nullptr, scale,
                  mask_kind, key_lens, 0, 0, workspace, workspace_bytes, stream);
}

int attn_bwd_window(const void* q, const void* k, const void* v, const void* o, const void* dout,
                    const float* lse, void* dq, void* dk, void* dv, int B, int h, int n_q,
                    int n_k, int d_k, float scale, int window_left, int window_right,
                    void* workspace, size_t workspace_bytes, struct CUstream_st* stream) {
  if (window_left < 0 || window_right < 0) return ATTN_ERR_INVALID_ARG;
  return bwd_impl(q, k, v, o, dout, lse, dq, dk, dv, B, h, n_q, n_k, d_k, nullptr, scale,
                  kMaskBand, nullptr, window_left, window_right, workspace, workspace_bytes,
                  stream);
}

int attn_bwd_strided(const void* q, const void* k, const void* v, const void* o, const void* dout,
                     const float* lse, void* dq, void* dk, void* dv, int B, int h, int n_q,
                     int n_k, int d_k, const int64_t* strides, float scale, int mask_kind,
                     const int* key_lens, int window_left, int window_right, void* workspace,
                     size_t workspace_bytes, struct CUstream_st* stream) {
  if (mask_kind < ATTN_MASK_NONE || mask_kind > ATTN_MASK_WINDOW) return ATTN_ERR_INVALID_ARG;
  if (mask_kind == ATTN_MASK_WINDOW && (window_left < 0 || window_right < 0))
    return ATTN_ERR_INVALID_ARG;
  if (strides == nullptr) return ATTN_ERR_INVALID_ARG;
  Strides st[8];
  for (int i = 0; i < 8; ++i) {
    st[i] = Strides{strides[3 * i], strides[3 * i + 1], strides[3 * i + 2]};
    if (!stride_ok(st[i].b) || !stride_ok(st[i].h) || !stride_ok(st[i].n))
      return ATTN_ERR_INVALID_ARG;
  }
  const bool window = mask_kind == ATTN_MASK_WINDOW;
  return bwd_impl(q, k, v, o, dout, lse, dq, dk, dv, B, h, n_q, n_k, d_k, st, scale,
                  window ? static_cast<int>(kMaskBand) : mask_kind, window ? nullptr : key_lens,
                  window ? window_left : 0, window ? window_right : 0, workspace,
                  workspace_bytes, stream);
}

int attn_check(struct CUstream_st* stream) {
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return cuda_fail(e);
  DeviceInfo* di = nullptr;
  int rc = device_info(&di);
  if (rc != ATTN_OK) return rc;
  int status = 0;
  if ((e = cudaMemcpyFromSymbol(&status, g_status, sizeof(int))) != cudaSuccess) return cuda_fail(e);
  if (status != kDevOk) {
    const int zero = 0;
    if ((e = cudaMemcpyToSymbol(g_status, &zero, sizeof(int))) != cudaSuccess) return cuda_fail(e);
    return status == kDevWrongPlan ? ATTN_ERR_WRONG_PLAN : ATTN_ERR_TIMEOUT;
  }
  return ATTN_OK;
}

const char* attn_status_string(int status) {
  switch (status) {
    case ATTN_OK: return "ok";
    case ATTN_ERR_INVALID_ARG: return "invalid argument";
    case ATTN_ERR_UNSUPPORTED: return "unsupported head size or device";
    case ATTN_ERR_CUDA: return "CUDA error";
    case ATTN_ERR_TIMEOUT: return "a bounded wait inside a kernel timed out";
    case ATTN_ERR_SCRATCH_TOO_SMALL:
      return "these sizes need more scratch than the library's fixed scratch array holds";
    case ATTN_ERR_WRONG_PLAN: return "a mask plan was made for other sizes";
    default: return "unknown status";
  }
}

int attn_last_cuda_error(void) { return g_last_cuda_error.load(); }

uint64_t attn_set_wait_limit_ns(uint64_t limit_ns) {
  return g_limit_ns.exchange(limit_ns == 0 ? kDefaultLimitNs : limit_ns);
}

uint64_t attn_launch_count(void) { return g_launches.load(); }

int attn_diag_tile(const void* q, const void* k, const void* p, const void* v, float* s,
                   float* o, struct CUstream_st* stream) {
  if (!q || !k || !p || !v || !s || !o) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(p) || !aligned16(v) || !aligned16(s) ||
      !aligned16(o))
    return ATTN_ERR_INVALID_ARG;
  DeviceInfo* di = nullptr;
  int rc = device_info(&di);
  if (rc != ATTN_OK) return rc;
  CUtensorMap tmq, tmk, tmv;
  if ((rc = encode_2d(&tmq, q)) != ATTN_OK) return rc;
  if ((rc = encode_2d(&tmk, k)) != ATTN_OK) return rc;
  if ((rc = encode_2d(&tmv, v)) != ATTN_OK) return rc;
  cudaError_t e = launch_diag_tile(tmq, tmk, tmv, p, s, o, make_ctx(*di, stream));
  if (e != cudaSuccess) return cuda_fail(e);
  g_launches.fetch_add(1);
  return ATTN_OK;
}

int attn_diag_wait_timeout(uint64_t limit_ns, struct CUstream_st* stream) {
  if (limit_ns == 0 || limit_ns > 10000000000ull) return ATTN_ERR_INVALID_ARG;
  DeviceInfo* di = nullptr;
  int rc = device_info(&di);
  if (rc != ATTN_OK) return rc;
  cudaError_t e = launch_diag_wait_timeout(limit_ns, make_ctx(*di, stream));
  if (e != cudaSuccess) return cuda_fail(e);
  g_launches.fetch_add(1);
  return ATTN_OK;
}

}  // extern "C"

namespace attn {
namespace {
// A row stride in elements of `elem` bytes that keeps rows 16-byte aligned.
bool stride16_ok(long long elems, int elem) {
  return elems > 0 && elems < (1LL << 40) / elem && (elems * elem) % 16 == 0;
}

constexpr int kMostCached = 1 << 30;  // tokens of a sequence in a cache

bool block_tokens_ok(int t) { return t == 16 || t == 32 || t == 64 || t == 128; }

// Strides of `count` [B, h, n, d] tensors from a host array of 3 * count
// element counts, or contiguous ones when the array is null.
bool read_strides(Strides* st, const int64_t* in, int count, const int* heads, const int* rows,
                  int d, const int* elem) {
  for (int i = 0; i < count; ++i) {
    st[i] = in ? Strides{in[3 * i], in[3 * i + 1], in[3 * i + 2]} : bhsd(heads[i], rows[i], d);
    if (!stride16_ok(st[i].b, elem[i]) || !stride16_ok(st[i].h, elem[i]) ||
        !stride16_ok(st[i].n, elem[i]))
      return false;
  }
  return true;
}

// 0 (none), or large enough that the tanh's argument per unit of q.k is finite, and
// no larger than 2^64, so that this argument times a code's scale and the cap in log2
// units stay normal numbers (at 1e36 and above scores of 8-bit caches were wrong).
bool softcap_ok(float softcap, float scale) {
  return softcap >= 0.f && softcap <= 0x1p64f &&
         (softcap == 0.f || std::isfinite(4.f * scale / softcap));
}

bool int_ptr_ok(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A cache as 4-D (row bytes, L_max, h, B) bytes with a (min(row bytes, 128),
// tile keys, 1, 1) box, with the 128-byte swizzle where box rows are 128 bytes;
// strides in elements of `elem` bytes.
int encode_4d_bytes(CUtensorMap* map, const void* base, int row_bytes, int n, int h, int B,
                    Strides st, int elem, int box_rows) {
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(n),
                        static_cast<cuuint64_t>(h), static_cast<cuuint64_t>(B)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(st.n) * elem,
                           static_cast<cuuint64_t>(st.h) * elem,
                           static_cast<cuuint64_t>(st.b) * elem};
  const int inner = row_bytes < 128 ? row_bytes : 128;
  const CUtensorMapSwizzle swz =
      inner == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE;
  cuuint32_t box[4] = {static_cast<cuuint32_t>(inner), static_cast<cuuint32_t>(box_rows), 1u, 1u};
  cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ERR_INVALID_ARG;
}

int elem_bytes(int cache_format) { return cache_format == ATTN_CACHE_BF16 ? 2 : 1; }

// The most keys n_q queries with this window see.
int scored_seen(int n_q, int L_max, int window) {
  return window >= 0 && window < L_max - n_q ? window + n_q : L_max;
}

// Sizes of attn_decode_scored, shared with its workspace query.
int scored_decode_sizes(int B, int h, int h_kv, int n_q, int L_max, int d_k, int cache_format,
                        int window) {
  if (B < 1 || h < 1 || h_kv < 1 || n_q < 1 || L_max < 1 || d_k < 1 || h % h_kv != 0)
    return ATTN_ERR_INVALID_ARG;
  if (cache_format < ATTN_CACHE_BF16 || cache_format > ATTN_CACHE_INT8 || window < -1)
    return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * h > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
  if (!tc_head_size(d_k) || n_q > kDecodeMaxQueries) return ATTN_ERR_UNSUPPORTED;
  // the kernel counts the visible cache's tiles of 16 keys or more, over all
  // sequences and key heads (and tiles of query rows), in 31 bits
  if (static_cast<long long>(B) * h * n_q > (1LL << 24) || L_max > kMostCached ||
      static_cast<long long>(B) * h_kv * ((h / h_kv * n_q + 31) / 32) * (L_max / 16 + 2LL) >
          0x7fffffffLL)
    return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}
}  // namespace
}  // namespace attn

extern "C" {

int attn_cache_append(const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                      float* k_scale, float* v_scale, int B, int h, int n_new, int L_max, int d_k,
                      const int64_t* strides, int cache_format, int block_tokens,
                      const int* cache_lens, const int* new_lens, struct CUstream_st* stream) {
  if (!k_new || !v_new || !k_cache || !v_cache || !k_scale || !v_scale) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !int_ptr_ok(k_scale) || !int_ptr_ok(v_scale) || !int_ptr_ok(cache_lens) ||
      !int_ptr_ok(new_lens))
    return ATTN_ERR_INVALID_ARG;
  if (B < 1 || h < 1 || n_new < 1 || L_max < 1 || d_k < 1) return ATTN_ERR_INVALID_ARG;
  if (cache_format != ATTN_CACHE_E4M3 && cache_format != ATTN_CACHE_INT8)
    return ATTN_ERR_INVALID_ARG;
  if (!block_tokens_ok(block_tokens)) return ATTN_ERR_INVALID_ARG;
  const int heads[4] = {h, h, h, h}, rows[4] = {n_new, n_new, L_max, L_max}, elem[4] = {2, 2, 1, 1};
  Strides st[4];
  if (tc_head_size(d_k) && !read_strides(st, strides, 4, heads, rows, d_k, elem))
    return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * h > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
  if (!tc_head_size(d_k)) return ATTN_ERR_UNSUPPORTED;
  // (a row's number and its block's end stay inside int)
  if (L_max > kMostCached) return ATTN_ERR_UNSUPPORTED;
  // one block of threads at most per cache block that can be touched
  if (static_cast<double>(B) * h * cache_blocks_touched(n_new, L_max, block_tokens) * 2.0 >
      2147483647.0)
    return ATTN_ERR_UNSUPPORTED;
  DeviceInfo* di = nullptr;
  int rc;
  if ((rc = device_info(&di)) != ATTN_OK) return rc;
  CacheAppendProblem pb{k_new, v_new, k_cache, v_cache, k_scale, v_scale, B, h, n_new, L_max, d_k,
                        cache_format == ATTN_CACHE_E4M3, block_tokens, cache_lens, new_lens,
                        st[0], st[1], st[2], st[3]};
  cudaError_t e = launch_cache_append(pb, make_ctx(*di, stream));
  if (e != cudaSuccess) return cuda_fail(e);
  g_launches.fetch_add(1);
  return ATTN_OK;
}

size_t attn_decode_scored_workspace_bytes(int B, int h, int h_kv, int n_q, int L_max, int d_k,
                                          int cache_format, int window) {
  if (scored_decode_sizes(B, h, h_kv, n_q, L_max, d_k, cache_format, window) != ATTN_OK) return 0;
  DeviceInfo* di = nullptr;
  if (device_info(&di) != ATTN_OK) return 0;
  return scored_decode_plan(B, h, h_kv, n_q, scored_seen(n_q, L_max, window), d_k,
                            elem_bytes(cache_format), di->num_sms)
      .workspace_bytes;
}

int attn_decode_scored(const void* q, const void* k_cache, const void* v_cache,
                       const float* k_scale, const float* v_scale, void* o, float* lse, int B,
                       int h, int h_kv, int n_q, int L_max, int d_k, const int64_t* strides,
                       int cache_format, int block_tokens, float scale, float softcap,
                       const float* slopes, const int* cache_lens, int window, void* workspace,
                       size_t workspace_bytes, struct CUstream_st* stream) {
  if (!q || !k_cache || !v_cache || !o) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) ||
      !int_ptr_ok(k_scale) || !int_ptr_ok(v_scale) || !int_ptr_ok(lse) || !int_ptr_ok(slopes) ||
      !int_ptr_ok(cache_lens))
    return ATTN_ERR_INVALID_ARG;
  int rc = scored_decode_sizes(B, h, h_kv, n_q, L_max, d_k, cache_format, window);
  if (rc == ATTN_ERR_INVALID_ARG) return rc;
  if (!(std::isfinite(scale) && scale > 0.f)) return ATTN_ERR_INVALID_ARG;
  if (!softcap_ok(softcap, scale)) return ATTN_ERR_INVALID_ARG;
  const bool q8 = cache_format != ATTN_CACHE_BF16;
  if (q8 && (!k_scale || !v_scale || !block_tokens_ok(block_tokens))) return ATTN_ERR_INVALID_ARG;
  const int e1 = elem_bytes(cache_format);
  const int heads[4] = {h, h_kv, h_kv, h}, rows[4] = {n_q, L_max, L_max, n_q},
            elem[4] = {2, e1, e1, 2};
  Strides st[4];
  if (rc == ATTN_OK && !read_strides(st, strides, 4, heads, rows, d_k, elem))
    return ATTN_ERR_INVALID_ARG;
  if (rc != ATTN_OK) return rc;
  DeviceInfo* di = nullptr;
  if ((rc = device_info(&di)) != ATTN_OK) return rc;
  const ScoredDecodePlan plan = scored_decode_plan(
      B, h, h_kv, n_q, scored_seen(n_q, L_max, window), d_k, e1, di->num_sms);
  if (plan.workspace_bytes > 0 &&
      (workspace == nullptr || workspace_bytes < plan.workspace_bytes || !aligned16(workspace)))
    return ATTN_ERR_INVALID_ARG;
  CUtensorMap maps[2];
  if ((rc = encode_4d_bytes(&maps[0], k_cache, d_k * e1, L_max, h_kv, B, st[1], e1,
                            plan.tile_keys)) != ATTN_OK)
    return rc;
  if ((rc = encode_4d_bytes(&maps[1], v_cache, d_k * e1, L_max, h_kv, B, st[2], e1,
                            plan.tile_keys)) != ATTN_OK)
    return rc;
  ScoredDecodeProblem pb{q, k_cache, v_cache, k_scale, v_scale, o, lse, B, h, h_kv, n_q, L_max,
                         d_k, q8 ? block_tokens : 128, scale, softcap, slopes, cache_lens,
                         window < L_max ? window : -1, st[0], st[1], st[2], st[3]};
  const LaunchCtx ctx = make_ctx(*di, stream);
  float* ws = static_cast<float*>(workspace);
  const cudaError_t e = cache_format == ATTN_CACHE_BF16   ? launch_decode_scored_bf16(pb, maps, plan, ws, ctx)
                        : cache_format == ATTN_CACHE_E4M3 ? launch_decode_scored_e4m3(pb, maps, plan, ws, ctx)
                                                          : launch_decode_scored_int8(pb, maps, plan, ws, ctx);
  if (e != cudaSuccess) return cuda_fail(e);
  g_launches.fetch_add(plan.whole ? 1 : 2);
  return ATTN_OK;
}

}  // extern "C"

namespace attn {

ScoredDecodePlan scored_decode_plan(int B, int H, int HK, int n_q, int seen, int d, int elem_bytes,
                                    int num_sms) {
  ScoredDecodePlan plan;
  const int rows = H / HK * n_q;
  plan.row_tile = rows <= 8 ? 8 : (rows <= 16 ? 16 : 32);
  plan.row_tiles = (rows + plan.row_tile - 1) / plan.row_tile;
  const int row_bytes = d * elem_bytes;
  const long long units = static_cast<long long>(B) * HK * plan.row_tiles;
  auto tiles_of = [&](int kt) { return (seen + 2LL * kt - 2) / kt; };  // a window may start inside one
  // whole units per warp when there are enough of them to occupy the SMs and the
  // longest is at most 32 small tiles (about 20 us of one warp)
  int kt = scored_decode_tile_keys(row_bytes, false);
  const long long small = static_cast<long long>(num_sms) * scored_decode_warps(row_bytes, plan.row_tile, false);
  plan.whole = units * 2 >= small && tiles_of(kt) <= 32;
  plan.tile_keys = kt;
  if (plan.whole) {
    plan.warps = static_cast<int>(units < small ? units : small);
    plan.part_off = plan.workspace_bytes = 0;
    return plan;
  }
  // every resident warp takes a share of the tiles, if there are that many
  const bool big = scored_decode_big(row_bytes, plan.row_tile, false);
  plan.tile_keys = kt = scored_decode_tile_keys(row_bytes, big);
  const long long resident = static_cast<long long>(num_sms) * scored_decode_warps(row_bytes, plan.row_tile, big);
  const long long useful =
      (units * tiles_of(kt) + scored_decode_min_tiles() - 1) / scored_decode_min_tiles();
  plan.warps = static_cast<int>(useful < resident ? useful : resident);
  // the sequences' first tiles, then two partial results per warp
  plan.part_off = (static_cast<size_t>(B) + 1 + 3) / 4 * 4;
  plan.workspace_bytes = (plan.part_off + static_cast<size_t>(plan.warps) * 2 * plan.row_tile *
                                              (d + kPartTail)) * sizeof(float);
  return plan;
}

}  // namespace attn

namespace attn {
namespace {

constexpr int kMostTokens = 1 << 30;  // of a sequence: a place and a side of a mask add up in int

constexpr float kLeastScale = 0x1p-64f;  // where something is divided by it

int check_mask_sizes(int B, int n_q, int n_k) {
  if (B < 1 || n_q < 1 || n_k < 1) return ATTN_ERR_INVALID_ARG;
  const long long n = n_q > n_k ? n_q : n_k;
  if (n > kMostTokens || B * ((n + kMaskTile - 1) / kMaskTile) > 0x7fffffffLL)
    return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

// What attn_fwd_scored and attn_bwd_scored check alike.
int check_scored(const void* q, const void* k, const void* v, const void* o, const float* lse,
                 int B, int h, int h_kv, int n_q, int n_k, int d_k, float scale, float softcap,
                 const float* slopes, const void* plan, size_t plan_bytes) {
  int rc = check_common(q, k, v, o, lse, B, h, n_q, n_k, d_k, scale, ATTN_MASK_NONE, nullptr, 2);
  if (rc != ATTN_OK) return rc;
  if (h_kv < 1 || h % h_kv != 0) return ATTN_ERR_INVALID_ARG;
  if (!softcap_ok(softcap, scale) || !int_ptr_ok(slopes))
    return ATTN_ERR_INVALID_ARG;
  // the bias is added in units of q.k: slope / scale
  if (slopes != nullptr && scale < kLeastScale) return ATTN_ERR_INVALID_ARG;
  if ((rc = check_mask_sizes(B, n_q, n_k)) != ATTN_OK) return rc;
  // one work item per 256 queries, or per 128 keys, of a head
  const long long n = n_q > n_k ? n_q : n_k;
  if (static_cast<long long>(B) * h * ((n + 127) / 128) > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  if (plan != nullptr && (!aligned16(plan) || plan_bytes < mask_layout(B, n_q, n_k).bytes))
    return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

ScoreMod score_mod(float softcap, const float* slopes, int h, int h_kv, const void* plan, int B,
                   int n_q, int n_k, const Strides* st) {
  ScoreMod mod{softcap, slopes, h / h_kv, {}, plan != nullptr, st[0], st[1], st[2], {}, {}, 1};
  if (plan != nullptr) mod.plan = mask_plan_at(plan, B, n_q, n_k);
  return mod;
}

}  // namespace
}  // namespace attn

extern "C" {

size_t attn_mask_plan_bytes(int B, int n_q, int n_k) {
  return check_mask_sizes(B, n_q, n_k) == ATTN_OK ? mask_layout(B, n_q, n_k).bytes : 0;
}

int attn_mask_plan(int B, int n_q, int n_k, int window_left, int window_right,
                   const int* key_lens, const int* doc_ids, const int* prefix_lens, void* plan,
                   size_t plan_bytes, struct CUstream_st* stream) {
  int rc = check_mask_sizes(B, n_q, n_k);
  if (rc == ATTN_ERR_INVALID_ARG) return rc;
  if (window_left < -1 || window_right < -1) return ATTN_ERR_INVALID_ARG;
  if (!int_ptr_ok(key_lens) || !int_ptr_ok(doc_ids) || !int_ptr_ok(prefix_lens))
    return ATTN_ERR_INVALID_ARG;
  if (doc_ids != nullptr && n_q != n_k) return ATTN_ERR_INVALID_ARG;
  if (prefix_lens != nullptr && window_left >= 0) return ATTN_ERR_INVALID_ARG;
  if (plan == nullptr || !aligned16(plan)) return ATTN_ERR_INVALID_ARG;
  if (rc != ATTN_OK) return rc;
  if (plan_bytes < mask_layout(B, n_q, n_k).bytes) return ATTN_ERR_INVALID_ARG;
  DeviceInfo* di = nullptr;
  if ((rc = device_info(&di)) != ATTN_OK) return rc;
  const MaskProblem pb{B,
                       n_q,
                       n_k,
                       window_left < n_q ? window_left : -1,  // a longer side bounds nothing
                       window_right < n_k ? window_right : -1,
                       key_lens,
                       doc_ids,
                       prefix_lens};
  const cudaError_t e = launch_mask_plan(pb, plan, make_ctx(*di, stream));
  if (e != cudaSuccess) return cuda_fail(e);
  g_launches.fetch_add(doc_ids == nullptr ? 1 : (mask_plan_ordered(pb) ? 3 : 2));
  return ATTN_OK;
}

int attn_fwd_scored(const void* q, const void* k, const void* v, void* o, float* lse, int B, int h,
                    int h_kv, int n_q, int n_k, int d_k, const int64_t* strides, float scale,
                    float softcap, const float* slopes, const void* plan, size_t plan_bytes,
                    struct CUstream_st* stream) {
  int rc = check_scored(q, k, v, o, lse, B, h, h_kv, n_q, n_k, d_k, scale, softcap, slopes, plan,
                        plan_bytes);
  if (rc != ATTN_OK) return rc;
  if (!tc_head_size(d_k)) return ATTN_ERR_UNSUPPORTED;
  const int heads[4] = {h, h_kv, h_kv, h}, rows[4] = {n_q, n_k, n_k, n_q}, elem[4] = {2, 2, 2, 2};
  Strides st[4];
  if (!read_strides(st, strides, 4, heads, rows, d_k, elem)) return ATTN_ERR_INVALID_ARG;
  DeviceInfo* di = nullptr;
  if ((rc = device_info(&di)) != ATTN_OK) return rc;
  CUtensorMap tmq, tmk, tmv, tmo;
  const int kv_rows = fwd_tc_kv_rows(d_k);
  if ((rc = encode_4d(&tmq, q, d_k, n_q, h, B, st[0], 128)) != ATTN_OK) return rc;
  if ((rc = encode_4d(&tmk, k, d_k, n_k, h_kv, B, st[1], kv_rows)) != ATTN_OK) return rc;
  if ((rc = encode_4d(&tmv, v, d_k, n_k, h_kv, B, st[2], kv_rows)) != ATTN_OK) return rc;
  if ((rc = encode_4d(&tmo, o, d_k, n_q, h, B, st[3], 128)) != ATTN_OK) return rc;
  const Problem pb{q, k, v, o, lse, B, h, n_q, n_k, d_k, scale, kMaskNone, nullptr, 0, 0};
  const ScoreMod mod = score_mod(softcap, slopes, h, h_kv, plan, B, n_q, n_k, st);
  const cudaError_t e = launch_fwd_tc(pb, tmq, tmk, tmv, tmo, make_ctx(*di, stream), &mod);
  if (e != cudaSuccess) return cuda_fail(e);
  g_launches.fetch_add(1);
  return ATTN_OK;
}

size_t attn_bwd_scored_workspace_bytes(int B, int h, int h_kv, int n_q, int n_k, int d_k) {
  if (h < 1 || h_kv < 1 || h % h_kv != 0 || check_mask_sizes(B, n_q, n_k) != ATTN_OK ||
      !bwd_head_size_ok(d_k) || static_cast<long long>(B) * h > 0x7fffffffLL)
    return 0;
  return bwd_scored_layout(B, h, h_kv, n_q, n_k, d_k).scored_bytes;
}

int attn_bwd_scored(const void* q, const void* k, const void* v, const void* o, const void* dout,
                    const float* lse, void* dq, void* dk, void* dv, int B, int h, int h_kv,
                    int n_q, int n_k, int d_k, const int64_t* strides, float scale, float softcap,
                    const float* slopes, const void* plan, size_t plan_bytes, void* workspace,
                    size_t workspace_bytes, struct CUstream_st* stream) {
  int rc = check_scored(q, k, v, o, lse, B, h, h_kv, n_q, n_k, d_k, scale, softcap, slopes, plan,
                        plan_bytes);
  if (rc != ATTN_OK) return rc;
  if (!dout || !lse || !dq || !dk || !dv || !workspace) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(dout) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv) ||
      !aligned16(workspace))
    return ATTN_ERR_INVALID_ARG;
  if (scale < kLeastScale) return ATTN_ERR_INVALID_ARG;  // LSE comes off in units of q.k
  if (!bwd_head_size_ok(d_k)) return ATTN_ERR_UNSUPPORTED;
  // order: q, k, v, o, dout, dq, dk, dv
  const int heads[8] = {h, h_kv, h_kv, h, h, h, h_kv, h_kv},
            rows[8] = {n_q, n_k, n_k, n_q, n_q, n_q, n_k, n_k}, elem[8] = {2, 2, 2, 2, 2, 2, 2, 2};
  Strides st[8];
  if (!read_strides(st, strides, 8, heads, rows, d_k, elem)) return ATTN_ERR_INVALID_ARG;
  const BwdLayout lay = bwd_scored_layout(B, h, h_kv, n_q, n_k, d_k);
  if (workspace_bytes < lay.scored_bytes) return ATTN_ERR_INVALID_ARG;
  // (the parts of dK and dV are one tensor of 2^31 - 1 heads at most)
  if (2LL * lay.parts * B * h_kv > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  DeviceInfo* di = nullptr;
  if ((rc = device_info(&di)) != ATTN_OK) return rc;
  CUtensorMap maps[8];
  if ((rc = encode_4d(&maps[0], q, d_k, n_q, h, B, st[0], 128)) != ATTN_OK) return rc;
  if ((rc = encode_4d(&maps[1], k, d_k, n_k, h_kv, B, st[1], 128)) != ATTN_OK) return rc;
  if ((rc = encode_4d(&maps[2], v, d_k, n_k, h_kv, B, st[2], 128)) != ATTN_OK) return rc;
  if ((rc = encode_4d(&maps[3], dout, d_k, n_q, h, B, st[4], 128)) != ATTN_OK) return rc;
  if ((rc = encode_4d(&maps[4], dk, d_k, n_k, h_kv, B, st[6], 64)) != ATTN_OK) return rc;
  if ((rc = encode_4d(&maps[5], dv, d_k, n_k, h_kv, B, st[7], 64)) != ATTN_OK) return rc;
  if ((rc = encode_3d_f32(&maps[6], static_cast<uint8_t*>(workspace) + lay.dq_acc_off, d_k, n_q,
                          static_cast<long long>(B) * h)) != ATTN_OK)
    return rc;
  const BwdProblem pb{q, k, v, o, dout, lse, dq, dk, dv, B, h, n_q, n_k, d_k, scale,
                      kMaskNone, nullptr, 0, 0, st[3], st[4], st[5]};
  ScoreMod mod = score_mod(softcap, slopes, h, h_kv, plan, B, n_q, n_k, st);
  mod.sdk = st[6];
  mod.sdv = st[7];
  mod.parts = lay.parts;
  maps[7] = maps[6];
  if (lay.parts > 1 &&
      (rc = encode_3d_f32(&maps[7], static_cast<uint8_t*>(workspace) + lay.part_off, d_k, n_k,
                          2LL * lay.parts * B * h_kv)) != ATTN_OK)
    return rc;
  const cudaError_t e = launch_bwd(pb, maps, workspace, make_ctx(*di, stream), &mod);
  if (e != cudaSuccess) return cuda_fail(e);
  g_launches.fetch_add(3 + (bwd_few_possible(mod.masked, n_k) ? 1 : 0) + (lay.parts > 1 ? 1 : 0));
  return ATTN_OK;
}

}  // extern "C"

// ---------------------------------------------------------------- drafted tokens

namespace attn {
namespace {
// Sizes of attn_decode_tree, shared with its workspace query.
int tree_decode_sizes(int B, int h, int h_kv, int n, int L_max, int d_k, int cache_format,
                      int window) {
  if (B < 1 || h < 1 || h_kv < 1 || n < 1 || L_max < 1 || d_k < 1 || h % h_kv != 0)
    return ATTN_ERR_INVALID_ARG;
  if (cache_format < ATTN_CACHE_BF16 || cache_format > ATTN_CACHE_INT8 || window < -1)
    return ATTN_ERR_INVALID_ARG;
  if (!tc_head_size(d_k) || n > kMostNodes || L_max > kMostCached) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * h > (1LL << 24) / n) return ATTN_ERR_UNSUPPORTED;
  // the kernels count the visible cache's tiles of 16 keys or more, over all sequences
  // and key heads (and tiles of query rows), in 31 bits
  const long long tiles = (static_cast<long long>(h / h_kv) * n + 31) / 32;
  if (static_cast<long long>(B) * h_kv * tiles > 0x7fffffffLL / (L_max / 16 + 8LL))
    return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

// Bytes that a call reads or writes, and whether two such have any in common.
struct Extent {
  const void* at;
  long long bytes;
};
bool overlap(const Extent& a, const Extent& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  return x < y ? y - x < static_cast<uintptr_t>(a.bytes) : x - y < static_cast<uintptr_t>(b.bytes);
}
}  // namespace

ScoredDecodePlan tree_few_plan(int B, int H, int HK, int n, int seen, int d, int elem_bytes,
                               int num_sms) {
  ScoredDecodePlan plan = scored_decode_plan(B, H, HK, n, seen, d, elem_bytes, num_sms);
  // behind what the plan needs: the results of units that one warp took
  const size_t units = static_cast<size_t>(B) * HK * plan.row_tiles;
  plan.done_off = (plan.workspace_bytes / sizeof(float) + 3) / 4 * 4;
  plan.workspace_bytes = (plan.done_off + units * plan.row_tile * (d + kPartTail)) * sizeof(float);
  return plan;
}

TreePlan tree_plan(int B, int HK, int rows, int n, int L_max, int d, int window, int num_sms) {
  TreePlan plan;
  plan.blocks = (rows + 255) / 256;
  plan.block_rows = rows < 256 ? rows : 256;
  const int kt = tree_tile_keys(d);
  plan.tree_tiles = (n + kt - 1) / kt;
  const long long units = static_cast<long long>(B) * HK * plan.blocks;
  // most tiles of a unit (a window may begin inside one)
  const long long seen = window >= 0 && window < L_max ? window + kt - 1LL : L_max;
  const long long tiles = (seen + kt - 1) / kt + plan.tree_tiles;
  plan.whole = tiles <= 8;
  const long long useful = plan.whole ? units : (units * tiles + tree_min_tiles() - 1) / tree_min_tiles();
  plan.ctas = static_cast<int>(useful < num_sms ? useful : num_sms);
  plan.part_off = plan.workspace_bytes = 0;
  if (plan.whole) return plan;
  // the sequences' first tiles, then two parts per CTA
  plan.part_off = (static_cast<size_t>(B) + 1 + 3) / 4 * 4;
  plan.workspace_bytes = (plan.part_off + static_cast<size_t>(plan.ctas) * 2 * plan.block_rows *
                                              (d + kPartTail)) * sizeof(float);
  return plan;
}
}  // namespace attn

extern "C" {

size_t attn_decode_tree_workspace_bytes(int B, int h, int h_kv, int n, int L_max, int d_k,
                                        int cache_format, int window) {
  if (tree_decode_sizes(B, h, h_kv, n, L_max, d_k, cache_format, window) != ATTN_OK) return 0;
  DeviceInfo* di = nullptr;
  if (device_info(&di) != ATTN_OK) return 0;
  if (tree_few(B, h_kv, h / h_kv * n, d_k))
    return tree_few_plan(B, h, h_kv, n, scored_seen(n, L_max, window), d_k,
                         elem_bytes(cache_format), di->num_sms)
        .workspace_bytes;
  return tree_plan(B, h_kv, h / h_kv * n, n, L_max, d_k, window, di->num_sms).workspace_bytes;
}

int attn_decode_tree(const void* q, const void* k_tree, const void* v_tree, const void* k_cache,
                     const void* v_cache, const float* k_scale, const float* v_scale,
                     const int* parents, void* o, float* lse, int B, int h, int h_kv, int n,
                     int L_max, int d_k, const int64_t* strides, int cache_format,
                     int block_tokens, float scale, float softcap, const float* slopes,
                     const int* cache_lens, int window, void* workspace, size_t workspace_bytes,
                     struct CUstream_st* stream) {
  if (!q || !k_tree || !v_tree || !k_cache || !v_cache || !parents || !o)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_tree) || !aligned16(v_tree) || !aligned16(k_cache) ||
      !aligned16(v_cache) || !aligned16(o) || !int_ptr_ok(parents) || !int_ptr_ok(k_scale) ||
      !int_ptr_ok(v_scale) || !int_ptr_ok(lse) || !int_ptr_ok(slopes) || !int_ptr_ok(cache_lens))
    return ATTN_ERR_INVALID_ARG;
  int rc = tree_decode_sizes(B, h, h_kv, n, L_max, d_k, cache_format, window);
  if (rc == ATTN_ERR_INVALID_ARG) return rc;
  if (!(std::isfinite(scale) && scale > 0.f)) return ATTN_ERR_INVALID_ARG;
  if (!softcap_ok(softcap, scale)) return ATTN_ERR_INVALID_ARG;
  const bool q8 = cache_format != ATTN_CACHE_BF16;
  if (q8 && (!k_scale || !v_scale || !block_tokens_ok(block_tokens))) return ATTN_ERR_INVALID_ARG;
  const int e1 = elem_bytes(cache_format);
  const int heads[6] = {h, h_kv, h_kv, h_kv, h_kv, h}, rows[6] = {n, n, n, L_max, L_max, n},
            elem[6] = {2, 2, 2, e1, e1, 2};
  Strides st[6];
  if (rc == ATTN_OK && !read_strides(st, strides, 6, heads, rows, d_k, elem))
    return ATTN_ERR_INVALID_ARG;
  if (rc != ATTN_OK) return rc;
  DeviceInfo* di = nullptr;
  if ((rc = device_info(&di)) != ATTN_OK) return rc;
  // (the tree's own keys are that far back too)
  const int near = window < L_max + n ? window : -1;
  const LaunchCtx ctx = make_ctx(*di, stream);
  CUtensorMap maps[4];
  if (tree_few(B, h_kv, h / h_kv * n, d_k)) {
    const ScoredDecodePlan plan = tree_few_plan(B, h, h_kv, n, scored_seen(n, L_max, window), d_k,
                                                e1, di->num_sms);
    if (workspace == nullptr || workspace_bytes < plan.workspace_bytes || !aligned16(workspace))
      return ATTN_ERR_INVALID_ARG;
    for (int i = 0; i < 2; ++i)
      if ((rc = encode_4d_bytes(&maps[i], i ? v_cache : k_cache, d_k * e1, L_max, h_kv, B,
                                st[3 + i], e1, plan.tile_keys)) != ATTN_OK)
        return rc;
    const ScoredDecodeProblem pb{q, k_cache, v_cache, k_scale, v_scale, o, lse, B, h, h_kv, n,
                                 L_max, d_k, q8 ? block_tokens : 128, scale, softcap, slopes,
                                 cache_lens, near, st[0], st[3], st[4], st[5]};
    const TreeOwn tree{parents, k_tree, v_tree, st[1], st[2]};
    float* ws = static_cast<float*>(workspace);
    const cudaError_t e =
        cache_format == ATTN_CACHE_BF16   ? launch_tree_few_bf16(pb, maps, plan, ws, ctx, tree)
        : cache_format == ATTN_CACHE_E4M3 ? launch_tree_few_e4m3(pb, maps, plan, ws, ctx, tree)
                                          : launch_tree_few_int8(pb, maps, plan, ws, ctx, tree);
    if (e != cudaSuccess) return cuda_fail(e);
    g_launches.fetch_add(2);
    return ATTN_OK;
  }
  const TreeDecodeProblem pb{q, k_tree, v_tree, k_cache, v_cache, k_scale, v_scale, parents, o, lse,
                             B, h, h_kv, n, L_max, d_k, cache_format, q8 ? block_tokens : 128,
                             scale, softcap, slopes, cache_lens, near, st[0], st[1], st[2], st[3],
                             st[4], st[5]};
  const TreePlan plan = tree_plan(B, h_kv, h / h_kv * n, n, L_max, d_k, window, di->num_sms);
  if (plan.workspace_bytes > 0 &&
      (workspace == nullptr || workspace_bytes < plan.workspace_bytes || !aligned16(workspace)))
    return ATTN_ERR_INVALID_ARG;
  const int kt = tree_tile_keys(d_k);
  for (int i = 0; i < 2; ++i) {
    const void* cache = i ? v_cache : k_cache;
    rc = q8 ? encode_4d_bytes(&maps[i], cache, d_k, L_max, h_kv, B, st[3 + i], 1, kt)
            : encode_4d(&maps[i], cache, d_k, L_max, h_kv, B, st[3 + i], kt);
    if (rc != ATTN_OK) return rc;
    if ((rc = encode_4d(&maps[2 + i], i ? v_tree : k_tree, d_k, n, h_kv, B, st[1 + i], kt)) !=
        ATTN_OK)
      return rc;
  }
  const cudaError_t e =
      cache_format == ATTN_CACHE_BF16   ? launch_decode_tree_bf16(pb, maps, plan, workspace, ctx)
      : cache_format == ATTN_CACHE_E4M3 ? launch_decode_tree_e4m3(pb, maps, plan, workspace, ctx)
                                        : launch_decode_tree_int8(pb, maps, plan, workspace, ctx);
  if (e != cudaSuccess) return cuda_fail(e);
  g_launches.fetch_add(plan.whole ? 1 : 2);
  return ATTN_OK;
}

int attn_tree_verify(const void* target, const void* draft, const int* tokens,
                     const int* parents, const float* uniforms, int* path, int* path_lens,
                     int* next_tokens, int B, int n, int V, const int64_t* strides, int prob_type,
                     struct CUstream_st* stream) {
  if (!target || !tokens || !parents || !uniforms || !path || !path_lens || !next_tokens)
    return ATTN_ERR_INVALID_ARG;
  if (prob_type != ATTN_PROB_F32 && prob_type != ATTN_PROB_BF16) return ATTN_ERR_INVALID_ARG;
  const uintptr_t off = prob_type == ATTN_PROB_BF16 ? 1u : 3u;
  if ((reinterpret_cast<uintptr_t>(target) & off) || (reinterpret_cast<uintptr_t>(draft) & off) ||
      !int_ptr_ok(tokens) || !int_ptr_ok(parents) || !int_ptr_ok(uniforms) || !int_ptr_ok(path) ||
      !int_ptr_ok(path_lens) || !int_ptr_ok(next_tokens))
    return ATTN_ERR_INVALID_ARG;
  if (B < 1 || n < 1 || V < 1) return ATTN_ERR_INVALID_ARG;
  if (n > kMostNodes || V > (1 << 24) || B > (1 << 24)) return ATTN_ERR_UNSUPPORTED;
  long long st[4] = {static_cast<long long>(n) * V, V, static_cast<long long>(n) * V, V};
  for (int i = 0; strides != nullptr && i < (draft ? 4 : 2); ++i) {
    if (strides[i] < 0 || strides[i] >= (1LL << 40)) return ATTN_ERR_INVALID_ARG;
    st[i] = strides[i];
  }
  // every CTA of a sequence's cluster walks for itself, over what it has read while another
  // may write already: walks that differ would wait for each other's barriers
  const long long ints = 4LL * B * n;
  const int es = prob_type == ATTN_PROB_BF16 ? 2 : 4;
  auto rows = [&](int i) {  // (strides may be larger than any memory)
    const double x = ((B - 1.0) * st[i] + (n - 1.0) * st[i + 1] + V) * es;
    return static_cast<long long>(x < 0x1p60 ? x : 0x1p60);
  };
  const Extent in[5] = {{target, rows(0)}, {draft, draft ? rows(2) : 0}, {tokens, ints},
                        {parents, ints}, {uniforms, ints}};
  const Extent out[3] = {{path, ints}, {path_lens, 4LL * B}, {next_tokens, 4LL * B}};
  for (int i = 0; i < 3; ++i) {
    for (const Extent& x : in)
      if (overlap(out[i], x)) return ATTN_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return ATTN_ERR_INVALID_ARG;
  }
  DeviceInfo* di = nullptr;
  int rc;
  if ((rc = device_info(&di)) != ATTN_OK) return rc;
  TreeVerifyProblem pb{target, draft, tokens, parents, uniforms, path, path_lens, next_tokens, B, n,
                       V, st[0], st[1], st[2], st[3], prob_type == ATTN_PROB_BF16};
  const cudaError_t e = launch_tree_verify(pb, make_ctx(*di, stream));
  if (e != cudaSuccess) return cuda_fail(e);
  g_launches.fetch_add(1);
  return ATTN_OK;
}

int attn_cache_append_tree(const void* k_tree, const void* v_tree, const int* path,
                           const int* path_lens, void* k_cache, void* v_cache, float* k_scale,
                           float* v_scale, int layers, int B, int h, int n, int L_max, int d_k,
                           const int64_t* strides, int cache_format, int block_tokens,
                           const int* cache_lens, struct CUstream_st* stream) {
  if (!k_tree || !v_tree || !path || !path_lens || !k_cache || !v_cache)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned16(k_tree) || !aligned16(v_tree) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !int_ptr_ok(path) || !int_ptr_ok(path_lens) || !int_ptr_ok(k_scale) ||
      !int_ptr_ok(v_scale) || !int_ptr_ok(cache_lens))
    return ATTN_ERR_INVALID_ARG;
  if (layers < 1 || B < 1 || h < 1 || n < 1 || L_max < 1 || d_k < 1) return ATTN_ERR_INVALID_ARG;
  if (cache_format < ATTN_CACHE_BF16 || cache_format > ATTN_CACHE_INT8)
    return ATTN_ERR_INVALID_ARG;
  const bool q8 = cache_format != ATTN_CACHE_BF16;
  if (q8 && (!k_scale || !v_scale || !block_tokens_ok(block_tokens))) return ATTN_ERR_INVALID_ARG;
  if (!tc_head_size(d_k) || n > kMostNodes || L_max > kMostCached) return ATTN_ERR_UNSUPPORTED;
  const int e1 = elem_bytes(cache_format);
  LayerStrides st[4];
  for (int i = 0; i < 4; ++i) {
    const int rows = i < 2 ? n : L_max, es = i < 2 ? 2 : e1;
    if (strides != nullptr) {
      st[i].layer = strides[4 * i];
      st[i].row = Strides{strides[4 * i + 1], strides[4 * i + 2], strides[4 * i + 3]};
    } else {
      st[i].row = bhsd(h, rows, d_k);
      st[i].layer = st[i].row.b * B;
    }
    if (!stride16_ok(st[i].layer, es) || !stride16_ok(st[i].row.b, es) ||
        !stride16_ok(st[i].row.h, es) || !stride16_ok(st[i].row.n, es))
      return ATTN_ERR_INVALID_ARG;
  }
  // one block of threads at most per cache block that can be touched
  const int touched = q8 ? cache_blocks_touched(n, L_max, block_tokens) : 1;
  if (static_cast<double>(layers) * B * h * touched * 2.0 > 2147483647.0)
    return ATTN_ERR_UNSUPPORTED;
  DeviceInfo* di = nullptr;
  int rc;
  if ((rc = device_info(&di)) != ATTN_OK) return rc;
  CacheTreeProblem pb{k_tree, v_tree, k_cache, v_cache, k_scale, v_scale, layers, B, h, n, L_max,
                      d_k, !q8, cache_format == ATTN_CACHE_E4M3, q8 ? block_tokens : 128, path,
                      path_lens, cache_lens, {st[0], st[1]}, {st[2], st[3]}};
  const cudaError_t e = launch_cache_append_tree(pb, make_ctx(*di, stream));
  if (e != cudaSuccess) return cuda_fail(e);
  g_launches.fetch_add(1);
  return ATTN_OK;
}

}  // extern "C"
