// qat_api.cu -- the C ABI declared in include/qat_attn.h: host-side validation, the
// backward workspace layout, kernel launches on the caller's stream, status codes and
// the device-side error word.  No entry point here allocates device memory.
#include "qat_attn.h"
#include "qat_internal.h"
#include "sm100.cuh"

#include <cuda_runtime.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <mutex>

namespace qat {

// The error word that kernels whose bounded waits expire set (read and cleared by
// qat_attn_device_status), followed by the limit of those waits.
__device__ sm100::DeviceState g_device_state = {0u, 0u, sm100::kWaitLimitNs};

cudaError_t read_and_clear_device_error(unsigned int* out, cudaStream_t s) {
  cudaError_t e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return e;
  e = cudaMemcpyFromSymbol(out, g_device_state, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0u;
  return cudaMemcpyToSymbol(g_device_state, &zero, sizeof(unsigned int));
}

namespace {
constexpr int kMaxDevices = 64;
std::mutex g_ctx_mu;
int g_num_sms[kMaxDevices] = {};
}  // namespace

cudaError_t device_context(unsigned int** err, int* num_sms) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  // a host-side lookup (no allocation), repeated on every call: a cached address would
  // go stale when the device's context is destroyed and recreated
  void* p = nullptr;
  e = cudaGetSymbolAddress(&p, g_device_state);
  if (e != cudaSuccess) return e;
  *err = static_cast<unsigned int*>(p);
  std::lock_guard<std::mutex> lock(g_ctx_mu);
  if (g_num_sms[dev] == 0) {
    int n = 0;
    e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    g_num_sms[dev] = n;
  }
  *num_sms = g_num_sms[dev];
  return cudaSuccess;
}

}  // namespace qat

namespace {

using qat::aligned16;
using qat::check_sizes;
using qat::kMaxRows;

constexpr float kLog2e = 1.4426950408889634f;
constexpr size_t kAlign = 256;
constexpr int kMostKeys = 1 << 30;  // positions of a sequence in the cache

// With QAT_VERBOSE=1 in the environment, CUDA errors are also printed to stderr.
qat_status_t from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return QAT_OK;
  cudaGetLastError();  // reported here: not left for a later call's check of its launch
  static const bool verbose = [] {
    const char* v = getenv("QAT_VERBOSE");
    return v != nullptr && v[0] == '1';
  }();
  if (verbose) fprintf(stderr, "qat_attn: CUDA error %d: %s\n", static_cast<int>(e), cudaGetErrorString(e));
  return QAT_ERR_CUDA;
}

}  // namespace

extern "C" {

const char* qat_status_string(qat_status_t status) {
  switch (status) {
    case QAT_OK: return "QAT_OK";
    case QAT_ERR_INVALID_ARG: return "QAT_ERR_INVALID_ARG: invalid argument";
    case QAT_ERR_UNSUPPORTED: return "QAT_ERR_UNSUPPORTED: unsupported configuration";
    case QAT_ERR_CUDA: return "QAT_ERR_CUDA: CUDA runtime or launch error";
    case QAT_ERR_TIMEOUT: return "QAT_ERR_TIMEOUT: a bounded device wait expired";
    case QAT_ERR_WORKSPACE: return "QAT_ERR_WORKSPACE: workspace missing or too small";
    case QAT_ERR_BAD_PAGE: return "QAT_ERR_BAD_PAGE: a page index or length outside the cache";
  }
  return "QAT_ERR_UNKNOWN: unknown status code";
}

}  // extern "C"

namespace {

// A window's arguments as the kernels take them: both within the keys there are.
qat_status_t window_args(int N, int window, int sinks, int* w, int* s) {
  if (window < 1 || sinks < 0) return QAT_ERR_INVALID_ARG;
  if (N > (1 << 30)) return QAT_ERR_UNSUPPORTED;  // positions plus a window are 32-bit sums
  *w = window < N ? window : N;
  *s = sinks < N ? sinks : N;
  return QAT_OK;
}

qat_status_t fwd_impl(const void* q, const void* k, const void* v, void* o_q, void* o_hp, float* lse, int B, int H,
                      int Nq, int Nkv, int D, float sm_scale, int causal, int window, int sinks, int quant_mode,
                      void* stream) {
  bool empty = false;
  const qat_status_t st = check_sizes(B, H, Nq, Nkv, D, sm_scale, causal, quant_mode, &empty);
  if (st != QAT_OK || empty) return st;
  const void* ptrs[] = {q, k, v, o_q, lse};
  for (const void* p : ptrs)
    if (p == nullptr || !aligned16(p)) return QAT_ERR_INVALID_ARG;
  if (!aligned16(o_hp) || (o_hp == nullptr && window == 0)) return QAT_ERR_INVALID_ARG;
  qat::FwdArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.o_q = static_cast<uint16_t*>(o_q);
  a.o_hp = static_cast<uint16_t*>(o_hp);
  a.lse = lse;
  a.B = B; a.H = H; a.Nq = Nq; a.Nkv = Nkv; a.D = D;
  a.sm_scale = sm_scale;
  a.qk_scale = sm_scale * kLog2e;
  a.causal = causal;
  a.window = window;
  a.sinks = sinks;
  a.quant = quant_mode != QAT_QUANT_NONE;
  a.kv_head_rows = Nkv;
  a.o_q_f32 = nullptr;
  a.o_hp_f32 = nullptr;
  if (window > 0) {
    a.o_hp_f32 = static_cast<float*>(o_hp);
    a.o_hp = nullptr;
  }
  unsigned int* err = nullptr;
  int num_sms = 0;
  cudaError_t e = qat::device_context(&err, &num_sms);
  if (e == cudaSuccess) e = qat::launch_fwd_tc(a, err, num_sms, static_cast<cudaStream_t>(stream));
  return from_cuda(e);
}

}  // namespace

extern "C" {

qat_status_t qat_attn_fwd(const void* q, const void* k, const void* v, void* o_q, void* o_hp,
                          float* lse, int B, int H, int Nq, int Nkv, int D, float sm_scale,
                          int causal, int quant_mode, void* stream) {
  return fwd_impl(q, k, v, o_q, o_hp, lse, B, H, Nq, Nkv, D, sm_scale, causal, 0, 0, quant_mode, stream);
}

qat_status_t qat_attn_fwd_window(const void* q, const void* k, const void* v, void* o_q, float* o_hp, float* lse,
                                 int B, int H, int N, int D, float sm_scale, int window, int sinks, int quant_mode,
                                 void* stream) {
  int w = 0, s = 0;
  const qat_status_t st = window_args(N, window, sinks, &w, &s);
  if (st != QAT_OK) return st;
  return fwd_impl(q, k, v, o_q, o_hp, lse, B, H, N, N, D, sm_scale, 1, w, s, quant_mode, stream);
}

qat_status_t qat_attn_fwd_chunk(const void* q, const void* k, const void* v, float* o_q,
                                float* o_hp, float* lse, int B, int H, int Nq, int Nkv_total,
                                int kv_begin, int kv_len, int D, float sm_scale, int quant_mode,
                                void* stream) {
  bool empty = false;
  const qat_status_t st = check_sizes(B, H, Nq, Nkv_total, D, sm_scale, 0, quant_mode, &empty);
  if (st != QAT_OK || empty) return st;
  if (kv_begin < 0 || kv_len < 1 || static_cast<long long>(kv_begin) + kv_len > Nkv_total)
    return QAT_ERR_INVALID_ARG;
  if (kv_begin % 64 != 0) return QAT_ERR_UNSUPPORTED;  // a quantization tile would be split
  const void* ptrs[] = {q, k, v, o_q, o_hp, lse};
  for (const void* p : ptrs)
    if (p == nullptr || !aligned16(p)) return QAT_ERR_INVALID_ARG;
  const size_t off = static_cast<size_t>(kv_begin) * D;
  qat::FwdArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k) + off;
  a.v = static_cast<const uint16_t*>(v) + off;
  a.o_q = nullptr;
  a.o_hp = nullptr;
  a.lse = lse;
  a.B = B; a.H = H; a.Nq = Nq; a.Nkv = kv_len; a.D = D;
  a.sm_scale = sm_scale;
  a.qk_scale = sm_scale * kLog2e;
  a.causal = 0;
  a.window = a.sinks = 0;
  a.quant = quant_mode != QAT_QUANT_NONE;
  a.kv_head_rows = Nkv_total;
  a.o_q_f32 = o_q;
  a.o_hp_f32 = o_hp;
  unsigned int* err = nullptr;
  int num_sms = 0;
  cudaError_t e = qat::device_context(&err, &num_sms);
  if (e == cudaSuccess) e = qat::launch_fwd_tc(a, err, num_sms, static_cast<cudaStream_t>(stream));
  return from_cuda(e);
}

qat_status_t qat_attn_merge(float* o_q_acc, float* o_hp_acc, float* lse_acc,
                            const float* o_q_part, const float* o_hp_part, const float* lse_part,
                            void* o_q_out, void* o_hp_out, int B, int H, int Nq, int D,
                            void* stream) {
  if (B < 0 || H < 0 || Nq < 0 || (D != 64 && D != 128)) return QAT_ERR_INVALID_ARG;
  const long long rows = static_cast<long long>(B) * H * Nq;
  if (rows > kMaxRows) return QAT_ERR_INVALID_ARG;
  if (rows == 0) return QAT_OK;
  const void* ptrs[] = {o_q_acc, o_hp_acc, lse_acc, o_q_part, o_hp_part, lse_part};
  for (const void* p : ptrs)
    if (p == nullptr || !aligned16(p)) return QAT_ERR_INVALID_ARG;
  if ((o_q_out != nullptr && !aligned16(o_q_out)) || (o_hp_out != nullptr && !aligned16(o_hp_out)))
    return QAT_ERR_INVALID_ARG;
  unsigned int* err = nullptr;
  int num_sms = 0;
  cudaError_t e = qat::device_context(&err, &num_sms);
  if (e == cudaSuccess)
    e = qat::launch_merge(o_q_acc, o_hp_acc, lse_acc, o_q_part, o_hp_part, lse_part,
                          static_cast<uint16_t*>(o_q_out), static_cast<uint16_t*>(o_hp_out), rows,
                          D, num_sms, static_cast<cudaStream_t>(stream));
  return from_cuda(e);
}

size_t qat_attn_bwd_workspace_bytes(int B, int H, int Nq, int Nkv, int D) {
  bool empty = false;
  if (check_sizes(B, H, Nq, Nkv, D, 1.0f, 0, 0, &empty) != QAT_OK) return 0;
  return qat::bwd_workspace_layout(B, H, Nq, Nkv, D, qat::bwd_stream_k_ctas(B, H, Nq, Nkv)).total;
}

size_t qat_attn_bwd_window_workspace_bytes(int B, int H, int N, int D, int window, int sinks) {
  bool empty = false;
  int w = 0, s = 0;
  if (check_sizes(B, H, N, N, D, 1.0f, 1, 0, &empty) != QAT_OK || window_args(N, window, sinks, &w, &s) != QAT_OK)
    return 0;
  return qat::bwd_workspace_layout(B, H, N, N, D, 0).total + (empty ? 0 : qat::window_part_bytes(B, H, N, D, w, s));
}

}  // extern "C"

namespace {

qat_status_t bwd_impl(const void* q, const void* k, const void* v, const void* o_hp,
                      const float* lse, const void* dO, void* dq, void* dk, void* dv,
                      const float* k_mean, int B, int H, int Nq, int Nkv, int D, float sm_scale,
                      int causal, int window, int sinks, int quant_mode, void* workspace, size_t workspace_bytes,
                      void* stream) {
  bool empty = false;
  const qat_status_t st = check_sizes(B, H, Nq, Nkv, D, sm_scale, causal, quant_mode, &empty);
  if (st != QAT_OK) return st;
  if (B == 0 || H == 0) return QAT_OK;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t kv_bytes = static_cast<size_t>(B) * H * Nkv * D * sizeof(uint16_t);
  if (Nq == 0) {  // no queries: every key gets zero gradient
    if (dk == nullptr || dv == nullptr || !aligned16(dk) || !aligned16(dv))
      return QAT_ERR_INVALID_ARG;
    cudaError_t e = cudaMemsetAsync(dk, 0, kv_bytes, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(dv, 0, kv_bytes, s);
    return from_cuda(e);
  }
  const void* ptrs[] = {q, k, v, o_hp, lse, dO, dq, dk, dv};
  for (const void* p : ptrs)
    if (p == nullptr || !aligned16(p)) return QAT_ERR_INVALID_ARG;
  // the stream-K split of the dK/dV work runs only when the workspace also holds its
  // segment sums (qat_attn_bwd_workspace_bytes does; the no-alloc scratch may not)
  const size_t base = qat::bwd_workspace_layout(B, H, Nq, Nkv, D, 0).total;
  const size_t need = base + (window > 0 ? qat::window_part_bytes(B, H, Nq, D, window, sinks) : 0);
  if (workspace == nullptr || workspace_bytes < need) return QAT_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) != 0) return QAT_ERR_INVALID_ARG;
  int sk = causal ? 0 : qat::bwd_stream_k_ctas(B, H, Nq, Nkv);
  if (sk > 0 && workspace_bytes < qat::bwd_workspace_layout(B, H, Nq, Nkv, D, sk).total) sk = 0;

  qat::BwdArgs a;
  const qat::BwdWorkspace wl = qat::bwd_workspace_layout(B, H, Nq, Nkv, D, sk);
  char* ws = static_cast<char*>(workspace);
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.o_hp = static_cast<const uint16_t*>(o_hp);
  a.lse = lse;
  a.dO = static_cast<const uint16_t*>(dO);
  a.dq = static_cast<uint16_t*>(dq);
  a.dk = static_cast<uint16_t*>(dk);
  a.dv = static_cast<uint16_t*>(dv);
  a.lse_pad = reinterpret_cast<float*>(ws + wl.off_lse);
  a.delta = reinterpret_cast<float*>(ws + wl.off_delta);
  a.lse_ext = reinterpret_cast<uint16_t*>(ws + wl.off_lse_ext);
  a.d_ext = reinterpret_cast<uint16_t*>(ws + wl.off_d_ext);
  a.ones = reinterpret_cast<uint16_t*>(ws + wl.off_ones);
  a.part = sk > 0 || need > base ? reinterpret_cast<float*>(ws + wl.off_part) : nullptr;
  a.o_f32 = nullptr;
  if (window > 0 && quant_mode != QAT_QUANT_P_FP8E4M3_ROW_TILE64_PAGE_BWD) {
    a.o_f32 = static_cast<const float*>(o_hp);
    a.o_hp = nullptr;
  }
  a.window = window;
  a.sinks = sinks;
  a.sink_pieces = window > 0 ? qat::window_sink_pieces(B, H, Nq, window, sinks) : 1;
  a.k_mean = k_mean;
  a.sk_ctas = sk;
  a.B = B; a.H = H; a.Nq = Nq; a.Nkv = Nkv; a.D = D;
  a.sm_scale = sm_scale;
  a.qk_scale = sm_scale * kLog2e;
  a.causal = causal;
  a.page_bwd = quant_mode == QAT_QUANT_P_FP8E4M3_ROW_TILE64_PAGE_BWD;
  unsigned int* err = nullptr;
  int num_sms = 0;
  cudaError_t e = qat::device_context(&err, &num_sms);
  if (e == cudaSuccess) e = qat::launch_bwd_tc(a, err, num_sms, s);
  return from_cuda(e);
}

}  // namespace

extern "C" {

qat_status_t qat_attn_bwd(const void* q, const void* k, const void* v, const void* o_hp,
                          const float* lse, const void* dO, void* dq, void* dk, void* dv,
                          int B, int H, int Nq, int Nkv, int D, float sm_scale, int causal,
                          int quant_mode, void* workspace, size_t workspace_bytes,
                          void* stream) {
  return bwd_impl(q, k, v, o_hp, lse, dO, dq, dk, dv, nullptr, B, H, Nq, Nkv, D, sm_scale,
                  causal, 0, 0, quant_mode, workspace, workspace_bytes, stream);
}

qat_status_t qat_attn_bwd_window(const void* q, const void* k, const void* v, const void* o_hp, const float* lse,
                                 const void* dO, void* dq, void* dk, void* dv, const float* k_mean, int B, int H,
                                 int N, int D, float sm_scale, int window, int sinks, int quant_mode,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  int w = 0, s = 0;
  const qat_status_t st = window_args(N, window, sinks, &w, &s);
  if (st != QAT_OK) return st;
  if (k_mean != nullptr && !aligned16(k_mean)) return QAT_ERR_INVALID_ARG;
  return bwd_impl(q, k, v, o_hp, lse, dO, dq, dk, dv, k_mean, B, H, N, N, D, sm_scale, 1, w, s, quant_mode,
                  workspace, workspace_bytes, stream);
}

qat_status_t qat_attn_bwd_smooth_k(const void* q, const void* k, const void* v,
                                   const void* o_hp, const float* lse, const void* dO, void* dq,
                                   void* dk, void* dv, const float* k_mean, int B, int H, int Nq,
                                   int Nkv, int D, float sm_scale, int causal, int quant_mode,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  if (k_mean == nullptr || !aligned16(k_mean)) return QAT_ERR_INVALID_ARG;
  return bwd_impl(q, k, v, o_hp, lse, dO, dq, dk, dv, k_mean, B, H, Nq, Nkv, D, sm_scale,
                  causal, 0, 0, quant_mode, workspace, workspace_bytes, stream);
}

qat_status_t qat_debug_set_wait_limit_us(int limit_us, void* stream) {
  if (limit_us < 0 || limit_us > 4000000) return QAT_ERR_INVALID_ARG;
  // no kernel of the library may be running while the limit changes
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  const unsigned long long ns =
      limit_us == 0 ? 1ull : static_cast<unsigned long long>(limit_us) * 1000ull;
  if (e == cudaSuccess)
    e = cudaMemcpyToSymbol(qat::g_device_state, &ns, sizeof(ns),
                           offsetof(qat::sm100::DeviceState, wait_limit_ns));
  return from_cuda(e);
}

qat_status_t qat_attn_device_status(void* stream) {
  unsigned int word = 0u;
  const cudaError_t e = qat::read_and_clear_device_error(&word, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return QAT_ERR_CUDA;
  if (word & qat::kErrTimeout) return QAT_ERR_TIMEOUT;
  return word ? QAT_ERR_BAD_PAGE : QAT_OK;
}

qat_status_t qat_channel_mean(const void* x, float* mean, int B, int H, int N, int D,
                              void* stream) {
  if (B < 0 || H < 0 || N < 0 || (D != 64 && D != 128)) return QAT_ERR_INVALID_ARG;
  if (mean == nullptr || (reinterpret_cast<uintptr_t>(mean) & 3u) != 0) return QAT_ERR_INVALID_ARG;
  const long long rows = static_cast<long long>(B) * H * N;
  if (rows > kMaxRows) return QAT_ERR_INVALID_ARG;
  if (rows > 0 && (x == nullptr || !aligned16(x))) return QAT_ERR_INVALID_ARG;
  unsigned int* err = nullptr;
  int num_sms = 0;
  cudaError_t e = qat::device_context(&err, &num_sms);
  if (e == cudaSuccess)
    e = qat::launch_channel_mean(static_cast<const uint16_t*>(x), mean, rows, D, num_sms,
                                 static_cast<cudaStream_t>(stream));
  return from_cuda(e);
}

qat_status_t qat_fake_quant_tokens(const void* x, const float* mean, void* out, float* scales,
                                   int B, int H, int N, int D, void* stream) {
  if (B < 0 || H < 0 || N < 0 || (D != 64 && D != 128)) return QAT_ERR_INVALID_ARG;
  const long long bh = static_cast<long long>(B) * H;
  if (bh * N > kMaxRows || bh * ((N + 31) / 32) > kMaxRows) return QAT_ERR_INVALID_ARG;
  if (bh * N == 0) return QAT_OK;
  if (x == nullptr || out == nullptr || !aligned16(x) || !aligned16(out)) return QAT_ERR_INVALID_ARG;
  if (mean != nullptr && (reinterpret_cast<uintptr_t>(mean) & 3u) != 0) return QAT_ERR_INVALID_ARG;
  if (scales != nullptr && (reinterpret_cast<uintptr_t>(scales) & 3u) != 0)
    return QAT_ERR_INVALID_ARG;
  return from_cuda(qat::launch_fake_quant_tokens(
      static_cast<const uint16_t*>(x), mean, static_cast<uint16_t*>(out), scales,
      static_cast<int>(bh), N, D, static_cast<cudaStream_t>(stream)));
}

qat_status_t qat_subtract_mean(const void* x, const float* mean, void* out, int B, int H, int N,
                               int D, void* stream) {
  if (B < 0 || H < 0 || N < 0 || (D != 64 && D != 128)) return QAT_ERR_INVALID_ARG;
  const long long rows = static_cast<long long>(B) * H * N;
  if (rows > kMaxRows) return QAT_ERR_INVALID_ARG;
  if (rows == 0) return QAT_OK;
  if (x == nullptr || out == nullptr || mean == nullptr || !aligned16(x) || !aligned16(out) ||
      !aligned16(mean))
    return QAT_ERR_INVALID_ARG;
  unsigned int* err = nullptr;
  int num_sms = 0;
  cudaError_t e = qat::device_context(&err, &num_sms);
  if (e == cudaSuccess)
    e = qat::launch_subtract_mean(static_cast<const uint16_t*>(x), mean,
                                  static_cast<uint16_t*>(out), rows, D, num_sms,
                                  static_cast<cudaStream_t>(stream));
  return from_cuda(e);
}

}  // extern "C"

namespace {

// Element strides {b, h, n} of a [B, H, N, D] tensor, contiguous by default.  Rows start on
// 16-byte boundaries, so strides along axes longer than one are multiples of 8.
struct Strides {
  long long b, h, n;
};

bool get_strides(const long long* s, int B, int H, int N, int D, Strides* out) {
  if (s == nullptr) {
    out->n = D;
    out->h = static_cast<long long>(N) * D;
    out->b = out->h * H;
    return true;
  }
  *out = {s[0], s[1], s[2]};
  if (B <= 1) out->b = 0;
  if (H <= 1) out->h = 0;
  if (N <= 1) out->n = 0;
  for (long long x : {out->b, out->h, out->n})
    if (x < 0 || x % 8 != 0 || x > (1ll << 40)) return false;
  return true;
}

// Checks shared by the norm + rotation pass and its backward; fills in what both need.
qat_status_t norm_rope_args(qat::NormRopeArgs* a, const void* q, const long long* q_strides,
                            const void* k, const long long* k_strides, const int* positions,
                            long long position_stride, const unsigned long long* phases,
                            const void* q_weight, const void* k_weight, int weight_bf16, int B,
                            int Hq, int Hk, int N, int D, int rotary_dim, int interleaved,
                            float amplitude, float eps) {
  if (B < 0 || Hq < 0 || Hk < 0 || N < 0 || (D != 64 && D != 128)) return QAT_ERR_INVALID_ARG;
  if (rotary_dim < 0 || rotary_dim > D || rotary_dim % 16 != 0) return QAT_ERR_INVALID_ARG;
  if ((interleaved != 0 && interleaved != 1) || (weight_bf16 != 0 && weight_bf16 != 1))
    return QAT_ERR_INVALID_ARG;
  if (!isfinite(amplitude) || !isfinite(eps) || !(eps > 0.f)) return QAT_ERR_INVALID_ARG;
  const long long tokens = static_cast<long long>(B) * N;
  if (tokens > kMaxRows || tokens * Hq > kMaxRows || tokens * Hk > kMaxRows)
    return QAT_ERR_INVALID_ARG;
  a->tokens = tokens;
  if (tokens == 0) return QAT_OK;
  if (rotary_dim > 0 && (positions == nullptr || phases == nullptr ||
                         (reinterpret_cast<uintptr_t>(positions) & 3u) != 0 ||
                         (reinterpret_cast<uintptr_t>(phases) & 7u) != 0 || position_stride < 0))
    return QAT_ERR_INVALID_ARG;
  if ((Hq > 0 && Hk > 0) && (q_weight == nullptr) != (k_weight == nullptr))
    return QAT_ERR_INVALID_ARG;  // both are normed, or neither
  auto tensor = [&](qat::NormRopeTensor* t, const void* x, const long long* strides,
                    const void* w, int H) {
    *t = {};
    t->H = H;
    if (H == 0) return true;
    Strides s;
    if (x == nullptr || !aligned16(x) || !get_strides(strides, B, H, N, D, &s)) return false;
    if (w != nullptr && !aligned16(w)) return false;
    t->x = static_cast<const uint16_t*>(x);
    t->sb = s.b; t->sh = s.h; t->sn = s.n;
    t->w = w;
    return true;
  };
  if (!tensor(&a->q, q, q_strides, q_weight, Hq) || !tensor(&a->k, k, k_strides, k_weight, Hk))
    return QAT_ERR_INVALID_ARG;
  a->positions = positions;
  a->pos_sb = position_stride;
  a->phases = phases;
  a->B = B; a->N = N; a->R = rotary_dim;
  a->interleaved = interleaved;
  a->w_bf16 = weight_bf16;
  a->amplitude = amplitude;
  a->eps = eps;
  a->part = nullptr;
  return QAT_OK;
}

// log2 of a page size the cache accepts (16, 32, 64, 128 or 256 tokens), or -1.
int page_shift(int page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

// The cache's own sizes, for the append, the read and the attention over it; the pointers are
// looked at only by calls that have work.
qat_status_t check_cache_sizes(int H, int D, int num_pages, int page_size, int max_pages) {
  if (H < 1 || (D != 64 && D != 128) || num_pages < 1 || max_pages < 1) return QAT_ERR_INVALID_ARG;
  if (page_shift(page_size) < 0) return QAT_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_pages) * page_size > (1ll << 30)) return QAT_ERR_UNSUPPORTED;
  // rows are numbered in 32 bits (2^32 rows of 64 channels are 550 GB of codes)
  if (static_cast<double>(num_pages) * H * page_size > 4294967000.0) return QAT_ERR_UNSUPPORTED;
  return QAT_OK;
}

bool cache_pointers_ok(const void* k_codes, const void* v_codes, const float* k_scales,
                       const float* v_scales, const int* block_table, const int* seq_lens) {
  for (const void* p : {k_codes, v_codes, static_cast<const void*>(k_scales),
                        static_cast<const void*>(v_scales)})
    if (p == nullptr || !aligned16(p)) return false;
  for (const int* p : {block_table, seq_lens})
    if (p == nullptr || (reinterpret_cast<uintptr_t>(p) & 3u) != 0) return false;
  return true;
}

}  // namespace

extern "C" {

qat_status_t qat_qk_norm_rope(const void* q, const long long* q_strides, const void* k,
                              const long long* k_strides, void* q_out, void* k_out,
                              const int* positions, long long position_stride,
                              const unsigned long long* phases, const void* q_weight,
                              const void* k_weight, int weight_bf16, int B, int Hq, int Hk, int N,
                              int D, int rotary_dim, int interleaved, float amplitude, float eps,
                              void* stream) {
  qat::NormRopeArgs a;
  const qat_status_t st = norm_rope_args(&a, q, q_strides, k, k_strides, positions,
                                         position_stride, phases, q_weight, k_weight, weight_bf16,
                                         B, Hq, Hk, N, D, rotary_dim, interleaved, amplitude, eps);
  if (st != QAT_OK || a.tokens == 0 || (Hq == 0 && Hk == 0)) return st;
  if ((Hq > 0 && (q_out == nullptr || !aligned16(q_out))) ||
      (Hk > 0 && (k_out == nullptr || !aligned16(k_out))))
    return QAT_ERR_INVALID_ARG;
  a.q.y = static_cast<uint16_t*>(q_out);
  a.k.y = static_cast<uint16_t*>(k_out);
  unsigned int* err = nullptr;
  int num_sms = 0;
  cudaError_t e = qat::device_context(&err, &num_sms);
  if (e == cudaSuccess) e = qat::launch_norm_rope(a, D, num_sms, static_cast<cudaStream_t>(stream));
  return from_cuda(e);
}

size_t qat_qk_norm_rope_bwd_workspace_bytes(int D) {
  if (D != 64 && D != 128) return 0;
  return sizeof(float) * static_cast<size_t>(qat::kNormRopeBwdBlocks) * D;
}

qat_status_t qat_qk_norm_rope_bwd(
    const void* q, const long long* q_strides, const void* k, const long long* k_strides,
    const void* dq_out, const long long* dq_out_strides, const void* dk_out,
    const long long* dk_out_strides, const int* positions, long long position_stride,
    const unsigned long long* phases, const void* q_weight, const void* k_weight, int weight_bf16,
    void* dq, const long long* dq_strides, void* dk, const long long* dk_strides, void* dq_weight,
    void* dk_weight, int B, int Hq, int Hk, int N, int D, int rotary_dim, int interleaved,
    float amplitude, float eps, void* workspace, size_t workspace_bytes, void* stream) {
  qat::NormRopeArgs a;
  const qat_status_t st = norm_rope_args(&a, q, q_strides, k, k_strides, positions,
                                         position_stride, phases, q_weight, k_weight, weight_bf16,
                                         B, Hq, Hk, N, D, rotary_dim, interleaved, amplitude, eps);
  if (st != QAT_OK) return st;
  for (const void* w : {dq_weight, dk_weight})
    if (w != nullptr && !aligned16(w)) return QAT_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.tokens == 0 || (Hq == 0 && Hk == 0)) {  // no rows: zero weight gradients
    const size_t bytes = static_cast<size_t>(D) * (weight_bf16 ? 2 : 4);
    for (void* w : {dq_weight, dk_weight})
      if (w != nullptr)
        if (const cudaError_t e = cudaMemsetAsync(w, 0, bytes, s); e != cudaSuccess) return from_cuda(e);
    return QAT_OK;
  }
  auto tensor = [&](qat::NormRopeTensor* t, const void* dy, const long long* dy_strides, void* dx,
                    const long long* dx_strides, void* dw) {
    if (t->H == 0) return dw == nullptr;
    Strides g, d;
    if (dy == nullptr || !aligned16(dy) || dx == nullptr || !aligned16(dx)) return false;
    if (!get_strides(dy_strides, B, t->H, N, D, &g) || !get_strides(dx_strides, B, t->H, N, D, &d))
      return false;
    if (dw != nullptr && t->w == nullptr) return false;
    t->dy = static_cast<const uint16_t*>(dy);
    t->dy_sb = g.b; t->dy_sh = g.h; t->dy_sn = g.n;
    t->y = static_cast<uint16_t*>(dx);
    t->y_sb = d.b; t->y_sh = d.h; t->y_sn = d.n;
    t->dw = dw;
    return true;
  };
  if (!tensor(&a.q, dq_out, dq_out_strides, dq, dq_strides, dq_weight) ||
      !tensor(&a.k, dk_out, dk_out_strides, dk, dk_strides, dk_weight))
    return QAT_ERR_INVALID_ARG;
  if (a.q.w != nullptr || a.k.w != nullptr) {
    if (workspace == nullptr || workspace_bytes < qat_qk_norm_rope_bwd_workspace_bytes(D))
      return QAT_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) != 0) return QAT_ERR_INVALID_ARG;
    a.part = static_cast<float*>(workspace);
  }
  unsigned int* err = nullptr;
  int num_sms = 0;
  cudaError_t e = qat::device_context(&err, &num_sms);
  if (e == cudaSuccess) e = qat::launch_norm_rope_bwd(a, D, num_sms, s);
  return from_cuda(e);
}

qat_status_t qat_kv_cache_append(const void* k, const long long* k_strides, const void* v,
                                 const long long* v_strides, void* k_codes, void* v_codes,
                                 float* k_scales, float* v_scales, const int* block_table,
                                 const int* seq_lens, const int* new_lens, int B, int H, int N,
                                 int D, int num_pages, int page_size, int max_pages,
                                 void* stream) {
  if (B < 0 || N < 0) return QAT_ERR_INVALID_ARG;
  const qat_status_t st = check_cache_sizes(H, D, num_pages, page_size, max_pages);
  if (st != QAT_OK) return st;
  if (new_lens != nullptr && (reinterpret_cast<uintptr_t>(new_lens) & 3u) != 0)
    return QAT_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * H > kMaxRows || static_cast<long long>(B) * H * N > kMaxRows)
    return QAT_ERR_INVALID_ARG;
  if (B == 0 || N == 0) return QAT_OK;
  if (!cache_pointers_ok(k_codes, v_codes, k_scales, v_scales, block_table, seq_lens))
    return QAT_ERR_INVALID_ARG;
  Strides ks, vs;
  if (k == nullptr || v == nullptr || !aligned16(k) || !aligned16(v) ||
      !get_strides(k_strides, B, H, N, D, &ks) || !get_strides(v_strides, B, H, N, D, &vs))
    return QAT_ERR_INVALID_ARG;
  qat::KvCacheArgs a = {};
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.k_sb = ks.b; a.k_sh = ks.h; a.k_sn = ks.n;
  a.v_sb = vs.b; a.v_sh = vs.h; a.v_sn = vs.n;
  a.k_codes = static_cast<uint8_t*>(k_codes);
  a.v_codes = static_cast<uint8_t*>(v_codes);
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  a.table = block_table;
  a.seq_lens = seq_lens;
  a.new_lens = new_lens;
  a.B = B; a.H = H; a.N = N;
  a.by_n = qat::FastDiv(N);
  a.by_h = qat::FastDiv(H);
  a.num_pages = num_pages;
  a.page_shift = page_shift(page_size);
  a.max_pages = max_pages;
  int num_sms = 0;
  cudaError_t e = qat::device_context(&a.err, &num_sms);
  if (e == cudaSuccess) e = qat::launch_kv_append(a, D, static_cast<cudaStream_t>(stream));
  return from_cuda(e);
}

qat_status_t qat_kv_cache_read(const void* k_codes, const void* v_codes, const float* k_scales,
                               const float* v_scales, const int* block_table, const int* seq_lens,
                               void* k_out, void* v_out, int B, int H, int begin, int N, int D,
                               int num_pages, int page_size, int max_pages, void* stream) {
  if (B < 0 || N < 0 || begin < 0) return QAT_ERR_INVALID_ARG;
  const qat_status_t st = check_cache_sizes(H, D, num_pages, page_size, max_pages);
  if (st != QAT_OK) return st;
  if (static_cast<long long>(B) * H > kMaxRows || static_cast<long long>(B) * H * N > kMaxRows)
    return QAT_ERR_INVALID_ARG;
  if (B == 0 || N == 0) return QAT_OK;
  if (!cache_pointers_ok(k_codes, v_codes, k_scales, v_scales, block_table, seq_lens))
    return QAT_ERR_INVALID_ARG;
  if (k_out == nullptr || v_out == nullptr || !aligned16(k_out) || !aligned16(v_out))
    return QAT_ERR_INVALID_ARG;
  qat::KvCacheArgs a = {};
  a.k_codes = static_cast<uint8_t*>(const_cast<void*>(k_codes));
  a.v_codes = static_cast<uint8_t*>(const_cast<void*>(v_codes));
  a.k_scales = const_cast<float*>(k_scales);
  a.v_scales = const_cast<float*>(v_scales);
  a.table = block_table;
  a.seq_lens = seq_lens;
  a.k_out = static_cast<uint16_t*>(k_out);
  a.v_out = static_cast<uint16_t*>(v_out);
  a.B = B; a.H = H; a.N = N;
  a.by_n = qat::FastDiv(N);
  a.by_h = qat::FastDiv(H);
  a.begin = begin;
  a.num_pages = num_pages;
  a.page_shift = page_shift(page_size);
  a.max_pages = max_pages;
  int num_sms = 0;
  cudaError_t e = qat::device_context(&a.err, &num_sms);
  if (e == cudaSuccess) e = qat::launch_kv_read(a, D, static_cast<cudaStream_t>(stream));
  return from_cuda(e);
}

}  // extern "C"

namespace {

size_t over_cache_workspace(int Hq, int Hkv, int T, int D, int most) {
  if ((D != 64 && D != 128) || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || T < 0 || T > most) return 0;
  const long long R = static_cast<long long>(Hq / Hkv) * T;
  const size_t few = qat::decode_workspace_bytes(static_cast<int>(R < 16 ? R : 16), D);
  if (most != qat::kTreeMaxTokens || !qat::tree_is_wide(R, D)) return few;
  // what holds a tree's partials holds a smaller tree's too
  const size_t many = qat::tree_workspace_bytes(static_cast<int>(R < kMaxRows ? R : kMaxRows), D);
  return few > many ? few : many;
}

// The attention of new tokens over the cache, `most` of them: decoding, with a window (0: none), or of a tree.
qat_status_t over_cache(const void* q, const void* k_codes, const void* v_codes, const float* k_scales,
                        const float* v_scales, const int* block_table, const int* seq_lens,
                        const unsigned long long* tree, long long tree_stride, void* o, float* lse, int B, int Hq,
                        int Hkv, int T, int most, int D, int num_pages, int page_size, int max_pages, float sm_scale,
                        int window, int sinks, int quant_mode, void* workspace, size_t workspace_bytes,
                        void* stream) {
  if (B < 0 || Hq < 1 || T < 0 || !(sm_scale > 0.f) || !isfinite(sm_scale * kLog2e))
    return QAT_ERR_INVALID_ARG;
  if (quant_mode != QAT_QUANT_NONE && quant_mode != QAT_QUANT_P_FP8E4M3_ROW_TILE64)
    return QAT_ERR_INVALID_ARG;
  const qat_status_t st = check_cache_sizes(Hkv, D, num_pages, page_size, max_pages);
  if (st != QAT_OK) return st;
  if (Hq % Hkv != 0) return QAT_ERR_INVALID_ARG;
  if (T > most || B > qat::kDecodeMaxBatch) return QAT_ERR_UNSUPPORTED;
  const long long rows = static_cast<long long>(Hq / Hkv) * T;
  if (rows > kMaxRows || static_cast<long long>(B) * Hkv > kMaxRows) return QAT_ERR_UNSUPPORTED;
  const long long units = (static_cast<long long>(max_pages) * page_size + 63) / 64;
  const double all = static_cast<double>(units) * B * Hkv * static_cast<double>((rows + 15) / 16);
  if (all > 1073741823.0) return QAT_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return QAT_OK;
  if (!cache_pointers_ok(k_codes, v_codes, k_scales, v_scales, block_table, seq_lens))
    return QAT_ERR_INVALID_ARG;
  if (q == nullptr || o == nullptr || !aligned16(q) || !aligned16(o)) return QAT_ERR_INVALID_ARG;
  if (lse != nullptr && (reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return QAT_ERR_INVALID_ARG;
  if (most == qat::kTreeMaxTokens && (tree == nullptr || (reinterpret_cast<uintptr_t>(tree) & 7u) != 0))
    return QAT_ERR_INVALID_ARG;
  if (workspace == nullptr || workspace_bytes < over_cache_workspace(Hq, Hkv, T, D, most)) return QAT_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) != 0) return QAT_ERR_INVALID_ARG;
  qat::DecodeArgs a = {};
  a.q = static_cast<const uint16_t*>(q);
  a.k_codes = static_cast<const uint8_t*>(k_codes);
  a.v_codes = static_cast<const uint8_t*>(v_codes);
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  a.table = block_table;
  a.seq_lens = seq_lens;
  a.o = static_cast<uint16_t*>(o);
  a.lse = lse;
  a.ws = workspace;
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.T = T;
  a.num_pages = num_pages;
  a.page_shift = page_shift(page_size);
  a.max_pages = max_pages;
  a.quant = quant_mode != QAT_QUANT_NONE;
  a.qk_scale = sm_scale * kLog2e;
  a.window = window < kMostKeys ? window : kMostKeys;  // of 2^30 positions, so that sums stay 32-bit
  a.sinks = sinks < kMostKeys ? sinks : kMostKeys;
  a.tree = tree;
  a.tree_sb = tree_stride;
  int num_sms = 0;
  cudaError_t e = qat::device_context(&a.err, &num_sms);
  if (e == cudaSuccess) e = qat::launch_decode(a, D, num_sms, static_cast<cudaStream_t>(stream));
  return from_cuda(e);
}

}  // namespace

extern "C" {

size_t qat_attn_decode_workspace_bytes(int Hq, int Hkv, int T, int D) {
  return over_cache_workspace(Hq, Hkv, T, D, qat::kDecodeMaxTokens);
}

qat_status_t qat_attn_decode(const void* q, const void* k_codes, const void* v_codes,
                             const float* k_scales, const float* v_scales, const int* block_table,
                             const int* seq_lens, void* o, float* lse, int B, int Hq, int Hkv,
                             int T, int D, int num_pages, int page_size, int max_pages,
                             float sm_scale, int quant_mode, void* workspace,
                             size_t workspace_bytes, void* stream) {
  return over_cache(q, k_codes, v_codes, k_scales, v_scales, block_table, seq_lens, nullptr, 0, o, lse, B, Hq, Hkv,
                    T, qat::kDecodeMaxTokens, D, num_pages, page_size, max_pages, sm_scale, 0, 0, quant_mode,
                    workspace, workspace_bytes, stream);
}

qat_status_t qat_attn_decode_window(const void* q, const void* k_codes, const void* v_codes, const float* k_scales,
                                    const float* v_scales, const int* block_table, const int* seq_lens, void* o,
                                    float* lse, int B, int Hq, int Hkv, int T, int D, int num_pages, int page_size,
                                    int max_pages, float sm_scale, int window, int sinks, int quant_mode,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  if (window < 1 || sinks < 0) return QAT_ERR_INVALID_ARG;
  return over_cache(q, k_codes, v_codes, k_scales, v_scales, block_table, seq_lens, nullptr, 0, o, lse, B, Hq, Hkv,
                    T, qat::kDecodeMaxTokens, D, num_pages, page_size, max_pages, sm_scale, window, sinks,
                    quant_mode, workspace, workspace_bytes, stream);
}

size_t qat_attn_tree_workspace_bytes(int Hq, int Hkv, int T, int D) {
  return over_cache_workspace(Hq, Hkv, T, D, qat::kTreeMaxTokens);
}

qat_status_t qat_attn_tree(const void* q, const void* k_codes, const void* v_codes, const float* k_scales,
                           const float* v_scales, const int* block_table, const int* seq_lens,
                           const unsigned long long* tree, long long tree_stride, void* o, float* lse, int B, int Hq,
                           int Hkv, int T, int D, int num_pages, int page_size, int max_pages, float sm_scale,
                           int window, int sinks, int quant_mode, void* workspace, size_t workspace_bytes,
                           void* stream) {
  if (window < 0 || sinks < 0 || tree_stride < 0 || (window == 0 && sinks > 0)) return QAT_ERR_INVALID_ARG;
  return over_cache(q, k_codes, v_codes, k_scales, v_scales, block_table, seq_lens, tree, tree_stride, o, lse, B, Hq,
                    Hkv, T, qat::kTreeMaxTokens, D, num_pages, page_size, max_pages, sm_scale, window, sinks,
                    quant_mode, workspace, workspace_bytes, stream);
}

qat_status_t qat_draft_tree(const int* parents, long long parents_stride, const int* seq_lens,
                            unsigned long long* tree, int* positions, int B, int T, void* stream) {
  if (B < 0 || T < 0 || parents_stride < 0) return QAT_ERR_INVALID_ARG;
  if (T > qat::kTreeMaxTokens) return QAT_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * T > kMaxRows) return QAT_ERR_INVALID_ARG;
  if (B == 0 || T == 0) return QAT_OK;
  for (const void* p : {static_cast<const void*>(parents), static_cast<const void*>(seq_lens),
                        static_cast<const void*>(positions)})
    if (p == nullptr || (reinterpret_cast<uintptr_t>(p) & 3u) != 0) return QAT_ERR_INVALID_ARG;
  if (tree == nullptr || (reinterpret_cast<uintptr_t>(tree) & 7u) != 0) return QAT_ERR_INVALID_ARG;
  const qat::DraftTreeArgs a = {parents, parents_stride, seq_lens, tree, positions, B, T};
  return from_cuda(qat::launch_draft_tree(a, static_cast<cudaStream_t>(stream)));
}

qat_status_t qat_kv_cache_keep(void* k_codes, void* v_codes, float* k_scales, float* v_scales,
                               const int* block_table, const int* seq_lens, const int* path, const int* path_lens,
                               int* new_lens, int B, int H, int T, int L, int D, int num_pages, int page_size,
                               int max_pages, void* stream) {
  if (B < 0 || T < 0 || L < 0) return QAT_ERR_INVALID_ARG;
  const qat_status_t st = check_cache_sizes(H, D, num_pages, page_size, max_pages);
  if (st != QAT_OK) return st;
  if (T > qat::kTreeMaxTokens || L > T) return QAT_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * H > kMaxRows) return QAT_ERR_INVALID_ARG;
  if (B == 0) return QAT_OK;
  if (!cache_pointers_ok(k_codes, v_codes, k_scales, v_scales, block_table, seq_lens)) return QAT_ERR_INVALID_ARG;
  for (const int* p : {path_lens, static_cast<const int*>(new_lens)})
    if (p == nullptr || (reinterpret_cast<uintptr_t>(p) & 3u) != 0) return QAT_ERR_INVALID_ARG;
  if (L > 0 && (path == nullptr || (reinterpret_cast<uintptr_t>(path) & 3u) != 0)) return QAT_ERR_INVALID_ARG;
  if (new_lens == seq_lens || new_lens == path_lens) return QAT_ERR_INVALID_ARG;  // read by a sequence's other blocks
  qat::KvKeepArgs a = {};
  a.k_codes = static_cast<uint8_t*>(k_codes);
  a.v_codes = static_cast<uint8_t*>(v_codes);
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  a.table = block_table;
  a.seq_lens = seq_lens;
  a.path = path;
  a.path_lens = path_lens;
  a.new_lens = new_lens;
  a.B = B; a.H = H; a.T = T; a.L = L;
  a.num_pages = num_pages;
  a.page_shift = page_shift(page_size);
  a.max_pages = max_pages;
  int num_sms = 0;
  cudaError_t e = qat::device_context(&a.err, &num_sms);
  if (e == cudaSuccess) e = qat::launch_kv_keep(a, D, static_cast<cudaStream_t>(stream));
  return from_cuda(e);
}

qat_status_t qat_debug_quant_tiles(const float* p, int rows, int cols, float* deq, float* scales,
                                   unsigned char* codes, void* stream) {
  if (rows < 0 || cols < 0) return QAT_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return QAT_OK;
  if (p == nullptr || deq == nullptr || scales == nullptr || codes == nullptr)
    return QAT_ERR_INVALID_ARG;
  return from_cuda(qat::launch_debug_quant(p, rows, cols, deq, scales, codes,
                                           static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
