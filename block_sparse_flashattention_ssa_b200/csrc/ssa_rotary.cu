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
// element of Q and K (75,600 x 40 + 40 x 128 behind an L2 flush: 490 us adjacent,
// 473 us half, 6.3 and 6.5 TB/s; 8192 x 24 + 24: 44 and 42 us, 39 and 37 back to
// back).
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
  bool copies;  // false when every output is its input: the elements past the rotated part stay where they are
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

// (cos, sin) of pair j at a token, with the scale and the direction.
__device__ __forceinline__ float2 table_entry(const Params& p, int64_t token, int j) {
  int axis = 0;
  while (axis < p.axes - 1 && j >= p.axis_end[axis]) ++axis;
  const double pos = static_cast<double>(p.positions[token * p.axes + axis]);
  const double turns = pos * (p.inv_freq[j] * 0.15915494309189533577);  // 1 / 2 pi
  float s, c;
  sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &c);
  return make_float2(c * p.scale, s * p.scale * p.sign);
}

// N consecutive elements of a head, moved with one access of 2 N bytes.
template <int N>
struct Piece;
template <>
struct Piece<8> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* x) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(x));
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
  __device__ __forceinline__ void store(__nv_bfloat16* y) const {
    __stcs(reinterpret_cast<uint4*>(y), make_uint4(w[0], w[1], w[2], w[3]));
  }
};
template <>
struct Piece<4> {
  uint32_t w[2];
  __device__ __forceinline__ void load(const __nv_bfloat16* x) {
    const uint2 v = __ldcs(reinterpret_cast<const uint2*>(x));
    w[0] = v.x, w[1] = v.y;
  }
  __device__ __forceinline__ void store(__nv_bfloat16* y) const { __stcs(reinterpret_cast<uint2*>(y), make_uint2(w[0], w[1])); }
};
template <>
struct Piece<2> {
  uint32_t w[1];
  __device__ __forceinline__ void load(const __nv_bfloat16* x) { w[0] = __ldcs(reinterpret_cast<const uint32_t*>(x)); }
  __device__ __forceinline__ void store(__nv_bfloat16* y) const { __stcs(reinterpret_cast<uint32_t*>(y), w[0]); }
};
template <>
struct Piece<1> {  // in the low half of the word
  uint32_t w[1];
  __device__ __forceinline__ void load(const __nv_bfloat16* x) { w[0] = __ldcs(reinterpret_cast<const unsigned short*>(x)); }
  __device__ __forceinline__ void store(__nv_bfloat16* y) const {
    __stcs(reinterpret_cast<unsigned short*>(y), static_cast<unsigned short>(w[0]));
  }
};

// A piece is what one thread takes of a head at a time:
//   interleaved  N = 8 elements (4 pairs; the last one may hold copied
//                elements as well), or one pair as two single elements when the
//                rows are not 16-byte aligned (N = 1);
//   half         N pairs, as two runs of N elements, or N copied elements; N is
//                the largest of 8, 4, 2, 1 that divides rot / 2 and suits the
//                rows' alignment.
// A thread keeps its piece and steps through the CTA's rows (token, head of Q
// then K) kBatch at a time, all loads of a batch first. The table of (cos,
// sin) holds two pairs to a float4, the k-th float4 of all pieces side by
// side, so that a warp reads it without bank conflicts.
template <bool INTERLEAVED, int N>
__global__ void __launch_bounds__(kThreads, 4) rotary_kernel(const __grid_constant__ Params p, int tokens_per_cta) {
  extern __shared__ __align__(16) float2 table[];  // [tokens_per_cta][turned * kPairs]
  constexpr int kPairs = INTERLEAVED ? (N == 8 ? 4 : 1) : N;  // pairs of a piece
  constexpr int kCopied = INTERLEAVED && N == 8 ? 8 : N;      // elements of a copied piece
  const int pairs = p.rot / 2;
  const int turned = (pairs + kPairs - 1) / kPairs, row_table = turned * kPairs;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens_per_cta;
  const int nt = static_cast<int>(min(static_cast<int64_t>(tokens_per_cta), p.tokens - t0));
  for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
    const int t = i / pairs, j = i - t * pairs;
    const int piece = j / kPairs, k = j % kPairs;
    const int at = kPairs == 1 ? j : ((k / 2) * turned + piece) * 2 + (k & 1);
    table[t * row_table + at] = table_entry(p, t0 + t, j);
  }
  __syncthreads();

  const int first_copied = INTERLEAVED && N == 8 ? turned * 8 : p.rot;
  const int pieces = turned + (p.copies ? (p.dim - first_copied) / kCopied : 0);  // 1 to 256
  const int stride = kThreads / pieces;                          // rows the CTA takes at once
  const int piece = static_cast<int>(threadIdx.x) % pieces;
  int row = static_cast<int>(threadIdx.x) / pieces;
  if (row >= stride) return;
  const int heads = p.heads[0] + p.heads[1];
  const bool copy = piece >= turned;
  const int at = copy ? first_copied + (piece - turned) * kCopied : (INTERLEAVED ? piece * 2 * kPairs : piece * N);
  const int at2 = INTERLEAVED ? at + 1 : at + pairs;  // the other elements of the pairs, where they stand apart
  constexpr bool kApart = !(INTERLEAVED && N == 8);
  constexpr int kBatch = N == 8 ? (INTERLEAVED ? 4 : 2) : 4;
  int token = row / heads, head = row - token * heads;
  while (token < nt) {
    __nv_bfloat16* y[kBatch];
    const float2* cs[kBatch];
    Piece<N> a[kBatch], b[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int which = head >= p.heads[0] ? 1 : 0;
      const int64_t h = static_cast<int64_t>(head - (which ? p.heads[0] : 0)) * p.dim;
      const __nv_bfloat16* x = p.x[which] + (t0 + token) * p.xs[which] + h;
      y[i] = token < nt ? p.y[which] + (t0 + token) * p.ys[which] + h : nullptr;
      cs[i] = table + token * row_table;
      if (token < nt) {
        a[i].load(x + at);
        if (kApart && !copy) b[i].load(x + at2);
      }
      head += stride;
      while (head >= heads) {
        head -= heads;
        ++token;
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (!y[i]) continue;
      if (!copy) {
        if (kPairs == 1) {
          float lo, hi;
          turn_pair(low(a[i].w[0]), low(b[i].w[0]), cs[i][piece], lo, hi);
          a[i].w[0] = pack(lo, 0.f);
          b[i].w[0] = pack(hi, 0.f);
        } else {
#pragma unroll
          for (int k = 0; k < kPairs; k += 2) {
            const float4 c2 = reinterpret_cast<const float4*>(cs[i])[(k / 2) * turned + piece];
            const float2 c0 = make_float2(c2.x, c2.y), c1 = make_float2(c2.z, c2.w);
            float l0, h0, l1, h1;
            if (kApart) {
              uint32_t &wa = a[i].w[k / 2], &wb = b[i].w[k / 2];
              turn_pair(low(wa), low(wb), c0, l0, h0);
              turn_pair(high(wa), high(wb), c1, l1, h1);
              wa = pack(l0, l1);
              wb = pack(h0, h1);
            } else {  // the piece across the end of the rotated part keeps its other elements
              uint32_t &w0 = a[i].w[k], &w1 = a[i].w[k + 1];
              turn_pair(low(w0), high(w0), c0, l0, h0);
              turn_pair(low(w1), high(w1), c1, l1, h1);
              if (piece * kPairs + k < pairs) w0 = pack(l0, h0);
              if (piece * kPairs + k + 1 < pairs) w1 = pack(l1, h1);
            }
          }
        }
        if (kApart) b[i].store(y[i] + at2);
      }
      a[i].store(y[i] + at);
    }
  }
}

// The half layout where rot / 2 is odd, so that the elements of pairs suit no
// access wider than one, but the rows are 16-byte aligned (DIM 64, 128 or 256):
// a warp brings whole heads into shared memory with 16-byte loads and turns
// them there, a 32-bit word (two elements, each with a partner rot / 2 away on
// one side or the other) per lane at a time. 20,000 x 16 + 16 x 128, rot 126:
// 98 us, element by element 169; with rot / 2 even, two elements at a time, the
// kernel above takes 88 and this one 98.
template <int DIM>
__global__ void __launch_bounds__(kThreads, 4) rotary_words_kernel(const __grid_constant__ Params p,
                                                                   int tokens_per_cta) {
  extern __shared__ __align__(16) float2 table[];  // [tokens_per_cta][pairs]
  constexpr int kPieces = DIM / 8, kHeads = 32 / kPieces;  // 16-byte pieces of a head, heads a warp takes at once
  constexpr int kBatch = 4, kWarps = kThreads / 32;
  __shared__ __align__(16) uint4 staged[kWarps][kBatch][32];
  const int pairs = p.rot / 2;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens_per_cta;
  const int nt = static_cast<int>(min(static_cast<int64_t>(tokens_per_cta), p.tokens - t0));
  for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
    const int t = i / pairs;
    table[i] = table_entry(p, t0 + t, i - t * pairs);
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = p.heads[0] + p.heads[1], rows = nt * heads;
  for (int first = warp * kHeads * kBatch; first < rows; first += kWarps * kHeads * kBatch) {
    uint4 v[kBatch];
    int token = (first + lane / kPieces) / heads, head = (first + lane / kPieces) - token * heads;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (token < nt) {
        const int which = head >= p.heads[0] ? 1 : 0;
        v[b] = __ldcs(reinterpret_cast<const uint4*>(p.x[which] + (t0 + token) * p.xs[which] +
                                                     static_cast<int64_t>(head - (which ? p.heads[0] : 0)) * DIM) +
                      lane % kPieces);
      }
      head += kHeads;
      while (head >= heads) {
        head -= heads;
        ++token;
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) staged[warp][b][lane] = v[b];
    __syncwarp();
    token = first / heads;
    head = first - token * heads;
#pragma unroll
    for (int r = 0; r < kBatch * kHeads; ++r) {  // the warp's heads in turn
      if (token < nt) {
        const int which = head >= p.heads[0] ? 1 : 0;
        uint32_t* y = reinterpret_cast<uint32_t*>(p.y[which] + (t0 + token) * p.ys[which] +
                                                  static_cast<int64_t>(head - (which ? p.heads[0] : 0)) * DIM);
        const unsigned short* x = reinterpret_cast<const unsigned short*>(&staged[warp][0][0]) + r * DIM;
        const float2* cs = table + token * pairs;
#pragma unroll
        for (int k = 0; k < DIM / 64; ++k) {
          const int word = lane + 32 * k, e = 2 * word;
          const uint32_t own = reinterpret_cast<const uint32_t*>(x)[word];
          uint32_t w = own;
          if (e < p.rot) {
            // Left elements of pairs have their partner to the right, and the
            // other way round; the two elements of a word may differ in that.
            const bool l0 = e < pairs, l1 = e + 1 < pairs;
            const float o0 = low(x[l0 ? e + pairs : e - pairs]), o1 = low(x[l1 ? e + 1 + pairs : e + 1 - pairs]);
            const float2 c0 = cs[l0 ? e : e - pairs], c1 = cs[l1 ? e + 1 : e + 1 - pairs];
            float a0, b0, a1, b1;
            turn_pair(l0 ? low(own) : o0, l0 ? o0 : low(own), c0, a0, b0);
            turn_pair(l1 ? high(own) : o1, l1 ? o1 : high(own), c1, a1, b1);
            w = pack(l0 ? a0 : b0, l1 ? a1 : b1);
          }
          __stcs(y + word, w);
        }
      }
      if (++head == heads) {
        head = 0;
        ++token;
      }
    }
    __syncwarp();
  }
}

// Tokens per CTA: a thread gets two batches of 16-byte pieces, or four where
// that still makes 16 CTAs per SM (75,600 x 40 + 40 x 128 interleaved 497 / 465
// us, with one batch 579; 8192 x 24 + 24 39.5 / 40.0).
int tokens_of_cta(const Params& p) {
  const int per_token = (p.heads[0] + p.heads[1]) * (p.dim / 8);
  int n = (16 * kThreads + per_token - 1) / per_token;
  if (p.tokens / n < 148 * 16) n = (8 * kThreads + per_token - 1) / per_token;
  return n < 1 ? 1 : (n > 16 ? 16 : n);
}

template <int DIM>
int launch_words(const Params& p, cudaStream_t stream) {
  const int n = tokens_of_cta(p);
  const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(p.tokens) + n - 1) / n);
  rotary_words_kernel<DIM><<<blocks, kThreads, static_cast<size_t>(n) * (p.rot / 2) * sizeof(float2), stream>>>(p, n);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SSA_OK : internal::fail(e);
}

template <bool INTERLEAVED, int N>
int launch(const Params& p, cudaStream_t stream) {
  const int n = tokens_of_cta(p);
  const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(p.tokens) + n - 1) / n);
  const size_t smem = static_cast<size_t>(n) * (p.rot / 2 + 3) * sizeof(float2);  // + 3: the last piece's unused pairs
  rotary_kernel<INTERLEAVED, N><<<blocks, kThreads, smem, stream>>>(p, n);
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
  // Largest run of elements, up to 8, that suits every address and stride and,
  // in the half layout, the distance between the elements of a pair.
  uint64_t aligned = 0;
  p.copies = false;
  for (int i = 0; i < n; ++i) {
    const uintptr_t both = reinterpret_cast<uintptr_t>(in[i]) | reinterpret_cast<uintptr_t>(out[i]);
    if (both & 1u) return SSA_ERR_UNSUPPORTED;
    aligned |= both / 2 | static_cast<uint64_t>(xs[i]) | static_cast<uint64_t>(ys[i]);
    p.x[i] = static_cast<const __nv_bfloat16*>(in[i]);
    p.y[i] = static_cast<__nv_bfloat16*>(out[i]);
    p.xs[i] = xs[i];
    p.ys[i] = ys[i];
    p.heads[i] = i ? num_kv_heads : num_heads;
    if (in[i] != out[i] || (xs[i] != ys[i] && total_tokens > 1)) p.copies = true;
  }
  uint64_t steps = 8 | aligned | (interleaved ? 0 : static_cast<uint64_t>(rotary_dim / 2));
  steps &= ~steps + 1;  // its lowest set bit
  if (const int rc = internal::device_pointers({q, q_out, positions, rotary_dim > 0 ? inv_freq : nullptr,
                                                n == 2 ? k : nullptr, n == 2 ? k_out : nullptr});
      rc != SSA_OK)
    return rc;
  if (rotary_dim == 0 && !p.copies) return SSA_OK;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.tokens = total_tokens;
  p.axes = num_axes;
  p.dim = head_dim;
  p.rot = rotary_dim;
  p.scale = scale;
  p.sign = transpose ? -1.f : 1.f;
  const cudaStream_t on = static_cast<cudaStream_t>(stream);
  if (interleaved) return steps == 8 ? launch<true, 8>(p, on) : launch<true, 1>(p, on);
  if (aligned % 8 == 0 && steps == 1) {
    if (head_dim == 64) return launch_words<64>(p, on);
    if (head_dim == 128) return launch_words<128>(p, on);
    if (head_dim == 256) return launch_words<256>(p, on);
  }
  switch (steps) {
    case 8: return launch<false, 8>(p, on);
    case 4: return launch<false, 4>(p, on);
    case 2: return launch<false, 2>(p, on);
    default: return launch<false, 1>(p, on);
  }
}
