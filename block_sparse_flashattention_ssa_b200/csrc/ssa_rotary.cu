// Rotary positions on packed Q and K for B200 (sm_100a): pair i of a token's
// head is turned by the angle t = pos * inv_freq[i],
//   (a, b) -> scale (a cos t - b sin t, a sin t + b cos t),
// or by -t for the adjoint (the gradient). Elements past the rotated part of
// the head are copied.
//
// The angle is formed in double as a fraction of a turn, pos * inv_freq / 2 pi
// less its nearest integer, and only that remainder is rounded to fp32: in
// fp32 the product alone would be off by pos * 2^-24 radians, a whole degree
// at position 300,000. One CTA holds a few tokens: its threads first fill a
// table of (cos, sin) in shared memory, each angle computed once for all heads
// of Q and K, then stream the heads. Bound by HBM: 2 bytes in and 2 out per
// element of Q and K.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "ssa.h"
#include "ssa_internal.h"

namespace ssa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxDim = 256;
constexpr int kMaxAxes = 4;

struct Params {
  const __nv_bfloat16* x[2];  // q, k
  __nv_bfloat16* y[2];
  int64_t xs[2], ys[2];  // elements from one token to the next
  int heads[2];
  const int32_t* positions;  // [tokens][axes]
  const double* inv_freq;    // [rot / 2]
  int tokens, axes, dim, rot;
  int axis_end[kMaxAxes];  // pairs before axis_end[a] (and from axis_end[a - 1]) turn with axis a
  float scale, sign;
};

__device__ __forceinline__ void turn_pair(float a, float b, float2 cs, float& lo, float& hi) {
  lo = fmaf(a, cs.x, __fmul_rn(-b, cs.y));  // spelled out, so that every variant rounds alike
  hi = fmaf(a, cs.y, __fmul_rn(b, cs.x));
}

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// VEC: the heads are made of 16-byte pieces and, in the half layout, so is half
// the rotated part, so that a thread turns 8 elements (interleaved) or 8 pairs
// (half) with 16-byte accesses; otherwise one element or pair at a time.
template <bool INTERLEAVED, bool VEC>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ Params p, int tokens_per_cta) {
  extern __shared__ float2 table[];  // [tokens_per_cta][rot / 2]
  const int pairs = p.rot / 2;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens_per_cta;
  const int nt = static_cast<int>(min(static_cast<int64_t>(tokens_per_cta), p.tokens - t0));
  for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
    const int t = i / pairs, j = i - t * pairs;
    int axis = 0;
    while (axis < p.axes - 1 && j >= p.axis_end[axis]) ++axis;
    const double pos = static_cast<double>(p.positions[(t0 + t) * p.axes + axis]);
    const double turns = pos * (p.inv_freq[j] * 0.15915494309189533577);  // 1 / 2 pi
    float s, c;
    sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &c);
    table[i] = make_float2(c * p.scale, s * p.scale * p.sign);
  }
  __syncthreads();

  // A piece is what one thread turns at a time; a head has `turned` of them
  // and then `rest` copied ones.
  const int step = VEC ? 8 : 1;
  const int turned = INTERLEAVED ? (VEC ? p.rot / 8 : pairs) : pairs / step;
  const int rest = (p.dim - p.rot) / step;
  const int pieces = turned + rest;
  const int per_token = (p.heads[0] + p.heads[1]) * pieces;
  for (int i = threadIdx.x; i < nt * per_token; i += kThreads) {
    const int t = i / per_token;
    int r = i - t * per_token;
    const int head_all = r / pieces, piece = r - head_all * pieces;
    const int which = head_all >= p.heads[0] ? 1 : 0;
    const int head = head_all - (which ? p.heads[0] : 0);
    const __nv_bfloat16* x = p.x[which] + (t0 + t) * p.xs[which] + static_cast<int64_t>(head) * p.dim;
    __nv_bfloat16* y = p.y[which] + (t0 + t) * p.ys[which] + static_cast<int64_t>(head) * p.dim;
    const float2* cs = table + t * pairs;
    if (piece >= turned) {
      const int at = p.rot + (piece - turned) * step;
      if (VEC)
        *reinterpret_cast<uint4*>(y + at) = *reinterpret_cast<const uint4*>(x + at);
      else
        y[at] = x[at];
    } else if (INTERLEAVED) {
      if (VEC) {
        const uint4 v = *reinterpret_cast<const uint4*>(x + piece * 8);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float a, b;
          turn_pair(low(w[k]), high(w[k]), cs[piece * 4 + k], a, b);
          o[k] = pack(a, b);
        }
        *reinterpret_cast<uint4*>(y + piece * 8) = make_uint4(o[0], o[1], o[2], o[3]);
      } else {
        float a, b;
        turn_pair(__bfloat162float(x[2 * piece]), __bfloat162float(x[2 * piece + 1]), cs[piece], a, b);
        y[2 * piece] = __float2bfloat16_rn(a);
        y[2 * piece + 1] = __float2bfloat16_rn(b);
      }
    } else if (VEC) {
      const uint4 va = *reinterpret_cast<const uint4*>(x + piece * 8);
      const uint4 vb = *reinterpret_cast<const uint4*>(x + pairs + piece * 8);
      const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
      uint32_t oa[4], ob[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float a0, b0, a1, b1;
        turn_pair(low(wa[k]), low(wb[k]), cs[piece * 8 + 2 * k], a0, b0);
        turn_pair(high(wa[k]), high(wb[k]), cs[piece * 8 + 2 * k + 1], a1, b1);
        oa[k] = pack(a0, a1);
        ob[k] = pack(b0, b1);
      }
      *reinterpret_cast<uint4*>(y + piece * 8) = make_uint4(oa[0], oa[1], oa[2], oa[3]);
      *reinterpret_cast<uint4*>(y + pairs + piece * 8) = make_uint4(ob[0], ob[1], ob[2], ob[3]);
    } else {
      float a, b;
      turn_pair(__bfloat162float(x[piece]), __bfloat162float(x[pairs + piece]), cs[piece], a, b);
      y[piece] = __float2bfloat16_rn(a);
      y[pairs + piece] = __float2bfloat16_rn(b);
    }
  }
}

template <bool INTERLEAVED>
int launch(const Params& p, bool vec, cudaStream_t stream) {
  // Enough tokens per CTA that its threads have about four pieces each.
  const int per_token = (p.heads[0] + p.heads[1]) * (p.dim / 8);
  int n = (4 * kThreads + per_token - 1) / per_token;
  n = n < 1 ? 1 : (n > 16 ? 16 : n);
  const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(p.tokens) + n - 1) / n);
  const size_t smem = static_cast<size_t>(n) * (p.rot / 2) * sizeof(float2);
  if (vec)
    rotary_kernel<INTERLEAVED, true><<<blocks, kThreads, smem, stream>>>(p, n);
  else
    rotary_kernel<INTERLEAVED, false><<<blocks, kThreads, smem, stream>>>(p, n);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SSA_OK : internal::fail(e);
}

}  // namespace
}  // namespace ssa

using namespace ssa;

extern "C" int ssa_rotary(const void* q, const void* k, void* q_out, void* k_out, int64_t q_stride, int64_t k_stride,
                          int64_t q_out_stride, int64_t k_out_stride, int total_tokens, int num_heads,
                          int num_kv_heads, int head_dim, const int32_t* positions, int num_axes,
                          const int32_t* sections, const double* inv_freq, int rotary_dim, int interleaved,
                          float scale, int transpose, void* stream) {
  if (total_tokens < 0 || num_heads < 1 || num_heads > 65535 || num_kv_heads < 0 || num_kv_heads > 65535 || head_dim < 1 || rotary_dim < 0 ||
      rotary_dim > head_dim || rotary_dim % 2 != 0 || num_axes < 1 || num_axes > kMaxAxes || !sections ||
      !std::isfinite(scale))
    return SSA_ERR_INVALID_ARG;
  if (head_dim % 8 != 0 || head_dim > kMaxDim) return SSA_ERR_UNSUPPORTED;
  Params p{};
  int64_t pairs = 0;
  for (int a = 0; a < num_axes; ++a) {
    if (sections[a] < 0) return SSA_ERR_INVALID_ARG;
    pairs += sections[a];
    if (pairs > rotary_dim / 2) return SSA_ERR_INVALID_ARG;
    p.axis_end[a] = static_cast<int>(pairs);
  }
  if (pairs != rotary_dim / 2) return SSA_ERR_INVALID_ARG;
  // Tokens must not overlap.
  const int64_t row_q = static_cast<int64_t>(num_heads) * head_dim, row_k = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (total_tokens > 1 && (q_stride < row_q || q_out_stride < row_q ||
                           (num_kv_heads > 0 && (k_stride < row_k || k_out_stride < row_k))))
    return SSA_ERR_INVALID_ARG;
  if (total_tokens == 0) return SSA_OK;
  if (!q || !q_out || !positions || (rotary_dim > 0 && !inv_freq) || (num_kv_heads > 0 && (!k || !k_out)))
    return SSA_ERR_INVALID_ARG;
  const int n = num_kv_heads > 0 ? 2 : 1;
  const void* in[2] = {q, k};
  void* out[2] = {q_out, k_out};
  const int64_t xs[2] = {q_stride, k_stride}, ys[2] = {q_out_stride, k_out_stride};
  bool vec = interleaved ? rotary_dim % 8 == 0 : (rotary_dim / 2) % 8 == 0;
  for (int i = 0; i < n; ++i) {
    if ((reinterpret_cast<uintptr_t>(in[i]) | reinterpret_cast<uintptr_t>(out[i])) & 1u) return SSA_ERR_UNSUPPORTED;
    if (((reinterpret_cast<uintptr_t>(in[i]) | reinterpret_cast<uintptr_t>(out[i])) & 15u) || xs[i] % 8 != 0 ||
        ys[i] % 8 != 0)
      vec = false;
    p.x[i] = static_cast<const __nv_bfloat16*>(in[i]);
    p.y[i] = static_cast<__nv_bfloat16*>(out[i]);
    p.xs[i] = xs[i];
    p.ys[i] = ys[i];
    p.heads[i] = i ? num_kv_heads : num_heads;
  }
  if (const int rc = internal::device_pointers({q, q_out, positions, rotary_dim > 0 ? inv_freq : nullptr,
                                                n == 2 ? k : nullptr, n == 2 ? k_out : nullptr});
      rc != SSA_OK)
    return rc;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.tokens = total_tokens;
  p.axes = num_axes;
  p.dim = head_dim;
  p.rot = rotary_dim;
  p.scale = scale;
  p.sign = transpose ? -1.f : 1.f;
  return interleaved ? launch<true>(p, vec, static_cast<cudaStream_t>(stream))
                     : launch<false>(p, vec, static_cast<cudaStream_t>(stream));
}
