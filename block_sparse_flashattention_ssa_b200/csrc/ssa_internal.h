// Host-side helpers shared by the library's translation units (defined in
// ssa_kernel.cu). Not part of the C ABI.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

namespace ssa {
namespace internal {

// Records the error's text for ssa_last_cuda_error and returns SSA_ERR_CUDA.
int fail(cudaError_t e);
int fail(const char* text);

// SSA_OK when every non-null pointer is device (or managed) memory of the
// current device, else SSA_ERR_INVALID_ARG.
int device_pointers(std::initializer_list<const void*> ptrs);

// [total_tokens, H, D] bf16 as a (d, head, token) tensor map with boxes of
// 64 x 1 x 128 elements, 128-byte swizzle; rows past total_tokens read as zero.
bool bf16_tensor_map(CUtensorMap* map, const void* base, int total_tokens, int H, int D);

// Device address of the current device's status word (read by ssa_get_error).
int status_word(int** ptr);

// Arguments of a backward pass, as in ssa_bwd.
struct Backward {
  const void *dout, *q, *k, *v, *out;
  const float* lse;
  const int32_t* cu_seqlens;
  int batch, total_tokens, max_seqlen, num_heads, num_kv_heads, head_dim;
  float softmax_scale;
  const uint32_t* decision_bitmap;
  int num_qblocks;
  void *dq, *dk, *dv, *workspace;
  int64_t workspace_bytes;
};

// Every host-side check of ssa_bwd; nothing is launched.
int check_backward(const Backward& a);

// Enqueues the backward pass on arguments that passed the check.
int launch_backward(const Backward& a, cudaStream_t stream);

}  // namespace internal

// Bits of the status word.
constexpr int kStatusTimeout = 1;
constexpr int kStatusDeviceArg = 2;

// Limit of every device-side wait.
constexpr unsigned long long kWaitLimitNs = 2000000000ull;

}  // namespace ssa
