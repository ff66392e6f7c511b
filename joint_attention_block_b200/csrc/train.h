// Launchers of the training pass through the attention sublayer (gradients, and the forward forms
// that keep what the gradients need).  Declared apart from internal.h: the inference path does
// not use them.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "internal.h"

namespace jab {

// Device error codes of the waits in the gradient kernels (see internal.h).
enum : uint32_t {
  ERR_TIMEOUT_ABWD_PRODUCER = 0x121,
  ERR_TIMEOUT_ABWD_MMA = 0x122,
  ERR_TIMEOUT_ABWD_SOFTMAX = 0x123,
  ERR_TIMEOUT_ABWD_DRAIN = 0x124,
  ERR_TIMEOUT_QKBWD = 0x125,
  ERR_TIMEOUT_NORMBWD = 0x126,
};

// 16-bit [B, S, n_heads * head_dim] view: row stride ld elements, batch stride S * ld.
struct Rows {
  const void* p;
  int64_t ld;
};

// Joint attention of separate q, k, v with the log-sum-exp of every row (lse fp32 [B, H, S]).
// key_lens (device int32 [B] or NULL): tokens of each element that take part; rows at or beyond it
// get zero in out and lse.  workspace: attention_lse_workspace() bytes, used when key_lens is given.
size_t attention_lse_workspace(int batch, int seq, int n_heads, int head_dim);
cudaError_t launch_attention_lse(Rows q, Rows k, Rows v, void* out, float* lse, int fmt, int batch, int seq,
                                 int n_heads, int head_dim, const int32_t* key_lens, void* workspace,
                                 const KernelGuard& g, cudaStream_t s);

// The gradient of the above; dq, dk, dv in the inputs' format.
size_t attention_bwd_workspace(int batch, int seq, int n_heads, int head_dim);
cudaError_t launch_attention_bwd(Rows q, Rows k, Rows v, const void* out, const void* dout, const float* lse, Rows dq,
                                 Rows dk, Rows dv, int fmt, int batch, int seq, int n_heads, int head_dim,
                                 const int32_t* key_lens, void* workspace, const KernelGuard& g, cudaStream_t s);

// Per-head QK-RMSNorm + 3D M-RoPE of the raw q and k in the fused qkv buffer [B, S, 3d] into qk
// [B, S, 2d]; key_lens (optional, [B]) receives each element's token count.
cudaError_t launch_qknorm_mrope_out(const void* qkv, void* qk, int fmt, int batch, int seq, int n_heads, int head_dim,
                                    int n_text, int grid_w, int n_img, int t_img, const int32_t* pos,
                                    const int32_t* text_lens, int32_t* key_lens, const int32_t sections[3],
                                    float theta, const uint16_t* g_q, const uint16_t* g_k, float eps, cudaStream_t s);

// Its gradient: dqk ([B, S, >= 2d] rows) is the gradient of the rotated q and k, dx (same shape, may
// be dqk itself) receives that of the raw ones, dg_q / dg_k (fp32 [hd]) the gains'.
size_t qknorm_mrope_bwd_workspace(int64_t tokens, int n_heads, int head_dim);
cudaError_t launch_qknorm_mrope_bwd(const void* qkv, Rows dqk, Rows dx, float* dg_q, float* dg_k, int fmt, int batch,
                                    int seq, int n_heads, int head_dim, int n_text, int grid_w, int n_img, int t_img,
                                    const int32_t* pos, const int32_t* text_lens, const int32_t sections[3],
                                    float theta, const uint16_t* g_q, const uint16_t* g_k, float eps, void* workspace,
                                    const KernelGuard& guard, cudaStream_t s);

// The gradient of launch_rmsnorm: dx = (d/dx)(dy) + dres (dres NULL: none; same format as dx, may be
// dx itself), dg fp32 [cols].  cols % 8 == 0, cols <= 8192.
size_t rmsnorm_bwd_workspace(int64_t rows, int64_t cols);
cudaError_t launch_rmsnorm_bwd(const void* x, int x_fmt, const uint16_t* g, const void* dy, int dy_fmt,
                               const void* dres, void* dx, int dx_fmt, float* dg, int64_t rows, int64_t cols,
                               float eps, void* workspace, const KernelGuard& guard, cudaStream_t s);

// Let a kernel have `bytes` of dynamic shared memory, once per device and size: the call costs about a
// microsecond, which the smallest sizes notice.  The allowance only grows, under a lock, so that one thread
// cannot lower what another has just asked for.
template <auto Kernel>
cudaError_t allow_smem(int bytes) {
  constexpr int DEVICES = 64;
  static std::atomic<int> set[DEVICES];
  static std::mutex growing;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= DEVICES) return cudaErrorInvalidDevice;
  if (set[dev].load(std::memory_order_acquire) >= bytes) return cudaSuccess;
  const std::lock_guard<std::mutex> lock(growing);
  if (set[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) set[dev].store(bytes, std::memory_order_release);
  return e;
}

}  // namespace jab
