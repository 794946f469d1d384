// Activations saved in 8 bits for the backward pass, for B200 (sm_100a).
//
// x [tokens, H, D] is stored as E4M3 codes and one scale per 128 tokens and
// head: s = 2^e, the smallest power of two with max |x| <= 448 s, and
// code = E4M3(x / s), nearest even. A power of two costs nothing in relative
// precision (E4M3 has exponents to spare) and makes both directions exact but
// for that one rounding: x / s is exact, and s times an E4M3 value (4
// significant bits) is exact in bf16. At the largest scale, 2^120, the code
// stops at 240: the next one, 256, would restore to 2^128, past bf16. A value
// that is not finite gets the NaN code and does not count towards the scale, so
// an overflow in the forward still shows in the gradients.
//
// Saving is one pass: a CTA holds the 128 x D tile of its head (of two heads
// with D = 64) in registers between the maximum and the conversion. Bound by
// HBM: 3 bytes per element each way; at 75,600 x 40 x 128, 199 us to save (5.8
// TB/s) and 203 us to restore (5.7 TB/s).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "sm100.cuh"
#include "ssa.h"
#include "ssa_internal.h"

namespace ssa {
namespace {

constexpr int kT = SSA_TILE;
constexpr int kThreads = 256;
constexpr int kMinExponent = -100;  // of the scale: its reciprocal and its products stay normal
constexpr int kMaxExponent = 120;   // of the scale: that of the largest bf16 values

// Finite values only: what is not finite stays so.
__device__ __forceinline__ float up_to_240(float y) { return fabsf(y) > 240.f && !isinf(y) ? copysignf(240.f, y) : y; }

// blockIdx.x: block of 128 tokens; blockIdx.y: 128 / D heads.
template <int D>
__global__ void __launch_bounds__(kThreads) save_kernel(const __nv_bfloat16* __restrict__ x,
                                                        uint8_t* __restrict__ codes, float* __restrict__ scales,
                                                        int tokens, int heads) {
  constexpr int kHeads = 128 / D;  // of the CTA: 16 lanes take a row of 128 elements, half of them each head of two
  constexpr int kRowsAtOnce = kThreads / 16, kSteps = kT / kRowsAtOnce;
  __shared__ uint32_t warp_max[kHeads][kThreads / 32];
  const int part = threadIdx.x % 16, r0 = threadIdx.x / 16;
  const int which = part / (D / 8), head = blockIdx.y * kHeads + which;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kT;
  const int64_t base = (t0 * heads + blockIdx.y * kHeads) * D + part * 8;
  const int rows = head < heads ? static_cast<int>(min(static_cast<int64_t>(kT), tokens - t0)) : 0;
  uint4 v[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int r = r0 + i * kRowsAtOnce;
    v[i] = r < rows ? __ldcs(reinterpret_cast<const uint4*>(x + base + static_cast<int64_t>(r) * heads * D))
                    : make_uint4(0, 0, 0, 0);
  }
  // Largest |x|, two at a time; the packed maximum passes over NaN, not over
  // infinities, which are rare enough for a second look.
  __nv_bfloat162 top2 = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t a = w[k] & 0x7FFF7FFFu;
      top2 = __hmax2(top2, *reinterpret_cast<const __nv_bfloat162*>(&a));
    }
  }
  auto widest = [&](uint32_t t) -> uint32_t {  // over the head, as fp32 bits (which order like the values)
    const uint32_t other = kHeads == 2 ? __reduce_max_sync(0xFFFFFFFFu, which ? t : 0u) : 0u;
    const uint32_t first = __reduce_max_sync(0xFFFFFFFFu, which ? 0u : t);
    if ((threadIdx.x & 31) == 0) {
      warp_max[0][threadIdx.x >> 5] = first;
      if (kHeads == 2) warp_max[kHeads - 1][threadIdx.x >> 5] = other;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) t = max(t, warp_max[which][i]);
    return t;
  };
  const uint32_t pair = *reinterpret_cast<const uint32_t*>(&top2);
  uint32_t top = widest(max(pair << 16, pair & 0xFFFF0000u));
  const bool infinite = top >= 0x7F800000u;
  if (__syncthreads_or(infinite)) {
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t lo = (w[k] << 16) & 0x7FFF0000u, hi = w[k] & 0x7FFF0000u;
        t = max(t, max(lo < 0x7F800000u ? lo : 0u, hi < 0x7F800000u ? hi : 0u));
      }
    }
    __syncthreads();
    t = widest(t);
    if (infinite) top = t;
  }
  // |x| = m 2^k with 1 <= m < 2 is at most 448 s = 1.75 2^8 s when s = 2^(k-8)
  // and m <= 1.75, else s = 2^(k-7). Subnormal maxima fall below the least scale.
  int e = static_cast<int>(top >> 23) - 127 - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  if (top == 0) e = 0;
  e = max(e, kMinExponent);
  const float scale = __int_as_float((e + 127) << 23), inv = __int_as_float((127 - e) << 23);
  if (r0 == 0 && part % (D / 8) == 0 && rows > 0) scales[static_cast<int64_t>(blockIdx.x) * heads + head] = scale;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int r = r0 + i * kRowsAtOnce;
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    uint32_t o[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float lo = __uint_as_float(w[k] << 16) * inv, hi = __uint_as_float(w[k] & 0xFFFF0000u) * inv;
      if (e == kMaxExponent) {
        lo = up_to_240(lo);
        hi = up_to_240(hi);
      }
      if (infinite) {
        if (isinf(lo)) lo = __int_as_float(0x7FC00000);
        if (isinf(hi)) hi = __int_as_float(0x7FC00000);
      }
      o[k >> 1] |= sm100::pack_e4m3x2(lo, hi) << ((k & 1) * 16);
    }
    if (r < rows)
      *reinterpret_cast<uint2*>(codes + base + static_cast<int64_t>(r) * heads * D) = make_uint2(o[0], o[1]);
  }
}

// Two E4M3 codes (low byte first) to fp32, exactly: fp16 holds every E4M3 value.
__device__ __forceinline__ float2 decode2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<unsigned short>(two)));
  float2 f;
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

struct Restore {
  const uint8_t* codes[3];
  const float* scales[3];
  __nv_bfloat16* x[3];
  int heads[3];
  int tokens;
};

constexpr int kPieces = 8;  // 8-element pieces per thread: loads of all of them go out first

// blockIdx.x: block of 128 tokens; blockIdx.y: kThreads * kPieces of its
// 8-element pieces; blockIdx.z: the tensor.
template <int D>
__global__ void __launch_bounds__(kThreads) restore_kernel(const __grid_constant__ Restore p) {
  const int z = blockIdx.z;
  const int heads = p.heads[z], per_row = heads * (D / 8);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kT;
  const int n = static_cast<int>(min(static_cast<int64_t>(kT), p.tokens - t0)) * per_row;  // pieces of the block
  const int first = static_cast<int>(blockIdx.y) * (kThreads * kPieces) + static_cast<int>(threadIdx.x);
  if (first >= n) return;
  const uint2* codes = reinterpret_cast<const uint2*>(p.codes[z]) + t0 * per_row + first;
  uint4* x = reinterpret_cast<uint4*>(p.x[z]) + t0 * per_row + first;
  const float* scales = p.scales[z] + static_cast<int64_t>(blockIdx.x) * heads;
  uint2 v[kPieces];
  float s[kPieces];
  int col = first % per_row;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    if (first + i * kThreads < n) {
      v[i] = __ldcs(codes + i * kThreads);
      s[i] = scales[col / (D / 8)];
    }
    col += kThreads;
    while (col >= per_row) col -= per_row;
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    if (first + i * kThreads >= n) break;
    const float2 a = decode2(v[i].x & 0xFFFFu), b = decode2(v[i].x >> 16);
    const float2 c = decode2(v[i].y & 0xFFFFu), d = decode2(v[i].y >> 16);
    x[i * kThreads] = make_uint4(sm100::pack_bf16x2(a.x * s[i], a.y * s[i]), sm100::pack_bf16x2(b.x * s[i], b.y * s[i]),
                                 sm100::pack_bf16x2(c.x * s[i], c.y * s[i]), sm100::pack_bf16x2(d.x * s[i], d.y * s[i]));
  }
}

int check(const void* codes, const float* scales, const void* x, int tokens, int heads, int dim) {
  if (tokens < 0 || heads < 1 || heads > 65535) return SSA_ERR_INVALID_ARG;
  if (dim != 64 && dim != 128) return SSA_ERR_UNSUPPORTED;
  if (tokens == 0) return SSA_OK;
  if (!codes || !scales || !x) return SSA_ERR_INVALID_ARG;
  if (((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(codes)) & 15u) ||
      (reinterpret_cast<uintptr_t>(scales) & 3u))
    return SSA_ERR_UNSUPPORTED;
  return internal::device_pointers({codes, scales, x});
}

int launch_restore(const Restore& p, int tensors, int dim, cudaStream_t stream) {
  int heads = 0;
  for (int i = 0; i < tensors; ++i) heads = p.heads[i] > heads ? p.heads[i] : heads;
  const int rows = p.tokens < kT ? p.tokens : kT;
  const int64_t pieces = static_cast<int64_t>(rows) * heads * (dim / 8);
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(p.tokens) + kT - 1) / kT),
                  static_cast<unsigned>((pieces + kThreads * kPieces - 1) / (kThreads * kPieces)), tensors);
  if (dim == 64)
    restore_kernel<64><<<grid, kThreads, 0, stream>>>(p);
  else
    restore_kernel<128><<<grid, kThreads, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SSA_OK : internal::fail(e);
}

}  // namespace
}  // namespace ssa

using namespace ssa;

extern "C" int ssa_save_fp8(const void* x, void* codes, float* scales, int total_tokens, int num_heads, int head_dim,
                            void* stream) {
  if (const int rc = check(codes, scales, x, total_tokens, num_heads, head_dim); rc != SSA_OK) return rc;
  if (total_tokens == 0) return SSA_OK;
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(total_tokens) + kT - 1) / kT),
                  static_cast<unsigned>((num_heads + 128 / head_dim - 1) / (128 / head_dim)));
  auto kernel = head_dim == 64 ? save_kernel<64> : save_kernel<128>;
  kernel<<<grid, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const __nv_bfloat16*>(x), static_cast<uint8_t*>(codes), scales, total_tokens, num_heads);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SSA_OK : internal::fail(e);
}

extern "C" int ssa_restore_fp8(const void* codes, const float* scales, void* x, int total_tokens, int num_heads,
                               int head_dim, void* stream) {
  if (const int rc = check(codes, scales, x, total_tokens, num_heads, head_dim); rc != SSA_OK) return rc;
  if (total_tokens == 0) return SSA_OK;
  Restore p{};
  p.codes[0] = static_cast<const uint8_t*>(codes);
  p.scales[0] = scales;
  p.x[0] = static_cast<__nv_bfloat16*>(x);
  p.heads[0] = num_heads;
  p.tokens = total_tokens;
  return launch_restore(p, 1, head_dim, static_cast<cudaStream_t>(stream));
}

// The restored tensors stand at the end of the workspace, the row values of
// ssa_bwd before them; both parts are multiples of 16 bytes.
extern "C" int64_t ssa_bwd_fp8_workspace_bytes(int total_tokens, int batch, int num_heads, int num_kv_heads,
                                               int head_dim) {
  const int64_t rows = ssa_bwd_workspace_bytes(total_tokens, batch, num_heads);
  if (rows < 0 || num_kv_heads < 1 || head_dim < 1) return SSA_ERR_INVALID_ARG;
  return rows + static_cast<int64_t>(total_tokens) * (num_heads + 2 * static_cast<int64_t>(num_kv_heads)) * head_dim * 2;
}

extern "C" int ssa_bwd_fp8(const void* dout, const void* q, const float* q_scales, const void* k,
                           const float* k_scales, const void* v, const float* v_scales, const void* out,
                           const float* lse, const int32_t* cu_seqlens, int batch, int total_tokens, int max_seqlen,
                           int num_heads, int num_kv_heads, int head_dim, float softmax_scale,
                           const uint32_t* decision_bitmap, int num_qblocks, void* dq, void* dk, void* dv,
                           void* workspace, int64_t workspace_bytes, void* stream) {
  if (num_kv_heads < 1 || num_heads < 1 || batch < 1) return SSA_ERR_INVALID_ARG;
  int rc = check(q, q_scales, workspace, total_tokens, num_heads, head_dim);
  if (rc == SSA_OK) rc = check(k, k_scales, workspace, total_tokens, num_kv_heads, head_dim);
  if (rc == SSA_OK) rc = check(v, v_scales, workspace, total_tokens, num_kv_heads, head_dim);
  if (rc != SSA_OK) return rc;
  const int64_t rows = ssa_bwd_workspace_bytes(total_tokens, batch, num_heads);
  if (total_tokens > 0 &&
      workspace_bytes < ssa_bwd_fp8_workspace_bytes(total_tokens, batch, num_heads, num_kv_heads, head_dim))
    return SSA_ERR_INVALID_ARG;
  uint8_t* at = static_cast<uint8_t*>(workspace) + rows;
  Restore p{};
  const void* codes[3] = {q, k, v};
  const float* scales[3] = {q_scales, k_scales, v_scales};
  for (int i = 0; i < 3; ++i) {
    p.codes[i] = static_cast<const uint8_t*>(codes[i]);
    p.scales[i] = scales[i];
    p.heads[i] = i ? num_kv_heads : num_heads;
    p.x[i] = reinterpret_cast<__nv_bfloat16*>(at);
    at += static_cast<int64_t>(total_tokens) * p.heads[i] * head_dim * 2;
  }
  p.tokens = total_tokens;
  const internal::Backward a{dout, p.x[0], p.x[1], p.x[2], out, lse, cu_seqlens, batch, total_tokens, max_seqlen,
                             num_heads, num_kv_heads, head_dim, softmax_scale, decision_bitmap, num_qblocks, dq, dk,
                             dv, workspace, rows};
  if ((rc = internal::check_backward(a)) != SSA_OK || total_tokens == 0) return rc;
  if ((rc = launch_restore(p, 3, head_dim, static_cast<cudaStream_t>(stream))) != SSA_OK) return rc;
  return internal::launch_backward(a, static_cast<cudaStream_t>(stream));
}
