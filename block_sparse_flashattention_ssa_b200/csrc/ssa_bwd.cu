// Backward pass of the (skip-softmax) attention forward for B200 (sm_100a).
//
// With c the softmax scale, L_r the row log-sum-exp the forward wrote and the
// sums taken over the KV tiles the forward kept:
//   P_rj  = exp(c q_r.k_j - L_r)              (recomputed)
//   D_r   = sum_d dO_rd O_rd
//   dV_j  = sum_r P_rj dO_r
//   dS_rj = P_rj (dO_r.v_j - D_r)
//   dQ_r  = c sum_j dS_rj k_j,  dK_j = c sum_r dS_rj q_r
// The forward's decisions are constants: no gradient flows through them.
//
// P and dS are rounded to bf16 for the products of dV and dK, the precision the
// tensor core takes Q, K and dO in; sums, statistics and D stay in fp32. Because
// sum_j dS_rj is nearly zero, what the keys have in common cancels in dQ, but
// not in the rounding errors of a row's dS: rounded once, they put dQ off by
// 0.0026 to 0.0039 of its norm in 64-bit comparisons, against 0.0017 that
// rounding the result costs. The q role therefore takes dS in two bf16 parts,
// dS = hi + lo with lo the rounding error of hi, and two products: dQ is off by
// no more than 0.0017. Each part of dS_rj meets key j alone, so a key without
// probability leaves no trace (times, rounded once / in two parts: 8192 x 24 x
// 128 2.49 / 2.73 ms, D = 64 1.74 / 1.90 ms).
//
// A first kernel forms D and -L log2 e per row, padded to whole query blocks
// (rows past a sequence end get -inf, as rows whose L is -inf do). The
// main kernel's CTAs each own 128 output rows and walk the other side's tiles:
//   kv role: 128 rows of K, V of one K/V head against every query block of the
//            sequence and every query head of its group that kept the tile;
//            S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q;
//   q role:  128 query rows against the KV tiles they kept;
//            S = Q K^T, dP = dO V^T, dQ += dS K.
// When there are too few rows for the SMs, the CTAs of a cluster share one
// block's tiles between them and add their accumulators up over distributed
// shared memory, in the order of their ranks.
// Both roles are one pipeline with the operands exchanged ("fixed" tiles A, B
// loaded once; "ring" tiles A, B streamed): S = fixA ringA^T, dP = fixB
// ringB^T, accA += dS ringA, and in the kv role accB += P ringB. S and dP are
// formed twice and dQ's product has two parts (8 products instead of 5); in
// exchange every output row has one owner: no atomics, no fp32 dQ in memory,
// and results that do not depend on the order in which CTAs run.
//
// Warp 0: TMA producer; warps 1-3: one tcgen05 issuing thread each, for S, for
// dP and for the accumulating products; warps 4-11: element-wise work, 64
// columns of one of the 128 TMEM lanes per thread. With one issuer for all of them
// its waits (110-300 cycles each while its own MMAs run, four or five per tile)
// drained the tensor pipe: 3280 and 2976 cycles per tile in the kv and q role.
// TMEM (512 columns): two score regions X [0,128) and Y [128,256), accA
// [256,256+D), and
//   kv role, D = 128: accB [384,512). Tile j has S in one score region and dP
//            in the other; P and dS, as bf16 pairs, replace S once it is in
//            registers (P in the first 32 of each 64 columns, dS in the
//            second). S of the next tile takes the place of dP as soon as that
//            has been read, and dP of the next tile that of P and dS once the
//            products that read them are complete: the regions change places
//            with every tile.
//   q role, and kv role with D = 64 (accB [320,384)): S in X and Z [384,512) by
//            turns, dP in Y; P and dS, or in the q role dS's two parts, replace
//            S in the same places. S of a tile is formed as soon as those of
//            the tile before last are used, dP as soon as the last tile's has
//            been read.
//
// Bound by the board's power in long runs (75,600 tokens of 5 heads of 128, dense:
// 47.3 ms, 773 TFLOP/s of the five products, 1237 of the eight formed here; 8192
// x 24 x 128 2.78 ms), by the element-wise warps at D = 64 (8192 x 24: 1.90 ms),
// by the length of the walks and the launches in small batches (1024 x 2 x 64:
// 13 to 17 us).
//
// Every wait is bounded in time; one that runs out records SSA_ERR_TIMEOUT in
// the status word, the other roles leave at their next wait, in-flight loads
// and MMAs are drained and TMEM is released.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "sm100.cuh"
#include "ssa.h"
#include "ssa_internal.h"

namespace ssa {
namespace {

using namespace sm100;

constexpr int kT = SSA_TILE;  // rows of every tile
// The issuers come first: a warp scheduler prefers the older of its warps, and
// an issuer behind two element-wise warps in their arithmetic woke 300-500
// cycles late.
constexpr int kTmaWarp = 0;
constexpr int kSWarp = 1, kDPWarp = 2, kAccWarp = 3;  // issuers
constexpr int kEwWarp = 4;                            // first of eight element-wise warps
constexpr int kEwThreads = 256;
constexpr int kThreads = 32 * kEwWarp + kEwThreads;
constexpr int kAStages = 3;  // ring A lives from its S to its dS product, longer than ring B
constexpr int kBStages = 2;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColX = 0, kColY = 128, kColAccA = 256, kColZ = 384;  // accB: behind accA's D columns
constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int kSMs = 148;
constexpr float kLog2e = 1.44269504088896340736f;

struct Params {
  const int32_t* cu_seqlens;
  const uint32_t* bitmap;  // forward's skip decisions, or NULL: every tile is kept
  __nv_bfloat16 *dq, *dk, *dv;
  const __nv_bfloat16 *out, *dout, *v;
  const float* lse;
  float* rows;  // [num_heads][units][2][128]: -L log2 e, then -D, per query block
  int* status;
  int batch, total_tokens, max_seqlen, num_heads, num_kv_heads, bitmap_words, max_tiles;
  int units;     // bound on the query blocks of the batch: ceil(total / 128) + batch
  int nq_check;  // query blocks the bitmap was sized for, or -1
  int split[2];  // CTAs that share a block's tiles: kv role, q role (1, or the cluster's size: a power of two)
  float scale;   // c
  float c2;      // fp32(c log2 e), the forward's score factor
};

struct Unit {
  int seq, block, S, start, gqb0, nq_total;  // block: 128-row block inside the sequence; gqb0: the sequence's first
};

struct Ctl {
  uint64_t fix_full;
  uint64_t a_full[kAStages], a_empty[kAStages];
  uint64_t b_full[kBStages], b_empty[kBStages];  // b_empty: q role (kv role: a_empty says it)
  // MMA results ready: S of even and odd tiles, dP; element-wise warps: dP in
  // registers; P (kv role) or dS's upper part (q role), and dS or its lower part,
  // of even and odd tiles stored. Two barriers
  // where the side that completes them may be a tile ahead of the side that
  // looks (the S issuer of the element-wise warps with three score regions,
  // these of the accumulating issuer): a single one would have gone round.
  uint64_t s_full[2], dp_full, dp_done, p_full[2], ds_full[2];
  uint64_t acc_full, drain[3];
  uint32_t tmem_base;
  int abort_flag;
  int info[kAStages];  // rows of the ring tile inside the sequence (128 but for the last), or -1: no more tiles
  Unit u;
};

template <int D>
struct Layout {
  static constexpr int kChunks = D / 64;  // 64 bf16 = 128 B per swizzled row
  static constexpr int kChunkBytes = kT * 128;
  static constexpr int kTileBytes = kT * D * 2;
  static constexpr int kRowBytes = 2 * kT * 4;  // -L log2 e and -D of one query block
  static constexpr int kFixA = 0;
  static constexpr int kFixB = kTileBytes;
  static constexpr int kRingA = 2 * kTileBytes;
  static constexpr int kRingB = kRingA + kAStages * kTileBytes;
  static constexpr int kRows = kRingB + kBStages * kTileBytes;  // kv role only
  static constexpr int kCtl = kRows + kBStages * kRowBytes;
  // No slack to align the base: the kernel declares it 1024-byte aligned (128-byte swizzle atoms).
  static constexpr int kAlloc = kCtl + static_cast<int>(sizeof(Ctl));
  static_assert(kAlloc <= 232448, "shared memory beyond the 227 KB a CTA may use");
};

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 31u) == 0) {
      if (*abort_flag) return false;
      if (globaltimer_ns() - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        atomicOr(status, kStatusTimeout);
        return false;
      }
    }
  }
}

__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, int* status) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      atomicOr(status, kStatusTimeout);
      return;
    }
  }
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
  return __all_sync(kFull, wait_bar(bar, parity, abort_flag, status));
}

// warp_wait for a barrier that was looked at before (`seen`, per lane): a wait
// that is already over costs a warp 110 cycles, nearly all of it latency that a
// look some work ahead hides.
__device__ __forceinline__ bool warp_wait_seen(bool seen, uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                               int* status) {
  return __all_sync(kFull, seen) || warp_wait(bar, parity, abort_flag, status);
}

__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// Finds the 128-row block number x of the batch (whole warp) and checks
// cu_seqlens: u.seq < 0 when there is no such block or the input is
// inconsistent (negative, decreasing or past total_tokens; with a bitmap, a
// sequence longer than max_seqlen or another number of query blocks than the
// bitmap was sized for), which is reported in the status word. Up to 32
// sequences are numbered longest first, so the longest walks start first;
// longer batches keep their order. Units are indexed in sequence order.
//
// A CTA runs this and the other code outside its walk once, on a cold
// instruction cache: short code (one sequence apart, loops left rolled) takes
// 1000 cycles here where unrolled code took 3800.
__device__ void locate(const Params& p, int x, int lane, bool report, Unit& u) {
  if (p.batch == 1) {
    if (lane == 0) {
      const int lo = p.cu_seqlens[0], hi = p.cu_seqlens[1];
      const bool in = lo >= 0 && hi >= lo && hi <= p.total_tokens;  // before the difference, which may pass 32 bits
      const int len = in ? hi - lo : 0, nq = (len + kT - 1) / kT;
      const bool bad = !in || (p.bitmap && nq > p.max_tiles) || (p.nq_check >= 0 && nq != p.nq_check);
      if (bad && report) atomicOr(p.status, kStatusDeviceArg);
      u = Unit{!bad && x < nq ? 0 : -1, x, len, lo, 0, nq};
    }
    return;
  }
  int seq = -1, block = 0, S = 0, start = 0, gqb0 = 0, bad = 0, total = 0, seen = 0;
  for (int base = 0; base < p.batch; base += 32) {
    const int b = base + lane;
    int lo = 0, len = 0, nq = 0;
    if (b < p.batch) {
      lo = p.cu_seqlens[b];
      const int hi = p.cu_seqlens[b + 1];
      const bool in = lo >= 0 && hi >= lo && hi <= p.total_tokens;
      if (!in) bad = 1;
      len = in ? hi - lo : 0;
      nq = (len + kT - 1) / kT;
      if (p.bitmap && nq > p.max_tiles) bad = 1;
    }
    int off = nq;  // inclusive prefix sum in sequence order
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(kFull, off, o);
      if (lane >= o) off += t;
    }
    const int sum = __shfl_sync(kFull, off, 31);
    off -= nq;
    int first = seen + off;  // number of this sequence's first block in the order of work
    if (p.batch <= 32) {
      first = 0;
#pragma unroll 1
      for (int o = 0; o < p.batch; ++o) {
        const int len_o = __shfl_sync(kFull, len, o), nq_o = __shfl_sync(kFull, nq, o);
        if (len_o > len || (len_o == len && o < b)) first += nq_o;
      }
    }
    const unsigned who = __ballot_sync(kFull, b < p.batch && x >= first && x < first + nq);
    if (who) {
      const int src = __ffs(static_cast<int>(who)) - 1;
      seq = base + src;
      block = __shfl_sync(kFull, x - first, src);
      S = __shfl_sync(kFull, len, src);
      start = __shfl_sync(kFull, lo, src);
      gqb0 = __shfl_sync(kFull, total + off, src);
    }
    total += sum;
    seen += sum;
  }
  bad = __any_sync(kFull, bad) ? 1 : 0;
  if (p.nq_check >= 0 && total != p.nq_check) bad = 1;
  if (lane == 0) {
    if (bad) {
      if (report) atomicOr(p.status, kStatusDeviceArg);
      seq = -1;
    }
    u = Unit{seq, block, S, start, gqb0, total};
  }
}

// A small main kernel is launched while rows_kernel still runs (programmatic
// dependent launch, see launch()) and waits for it only where it reads the row
// values: its prologue, first loads and S overlap with it.
__device__ __forceinline__ void next_kernel_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_rows() {
  // The fence: the kv role reads the row values by bulk copies.
  asm volatile("griddepcontrol.wait;\n fence.proxy.async.global;" ::: "memory");
}

// A row whose bias -L log2 e is -inf takes no part: one that saw nothing, or one
// past the sequence end. What its q, dO and O hold may be anything, so the main
// kernel's kv role sets its elements aside (a zero probability times NaN is NaN).
// To look for such rows only where there are some inside the sequence, the lowest
// bit of the bias of a block's first row says so (and costs that row at most
// 2^-23 of its bias, like a rounding).
__device__ __forceinline__ bool takes_no_part(float bias) { return bias == -INFINITY; }
__device__ __forceinline__ bool some_take_no_part(float first_bias) {
  return takes_no_part(first_bias) || (__float_as_uint(first_bias) & 1u);
}

// -D_r = -dO_r.O_r and -L_r log2 e of one query block and head; D / 8 lanes per
// row, 16 bytes of dO and O each. Bound by the read of dO and O. The one row of
// a sequence of length one gets dP - D = dO.(v - O) in place of -D: the forward
// wrote O = v there, and the difference of two rounded dot products would be
// all that is left of a gradient that is zero.
template <int D>
__global__ void __launch_bounds__(256) rows_kernel(const __grid_constant__ Params p) {
  __shared__ Unit u;
  next_kernel_may_start();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, head = blockIdx.y;
  if (warp == 0) locate(p, static_cast<int>(blockIdx.x), lane, blockIdx.x == 0 && head == 0, u);
  __syncthreads();
  if (u.seq < 0) return;
  constexpr int kLanes = D / 8, kRowsAtOnce = 256 / kLanes, kSteps = kT / kRowsAtOnce;
  const int part = threadIdx.x % kLanes, r0 = threadIdx.x / kLanes;
  const int rows = min(kT, u.S - u.block * kT);
  float* dst = p.rows + (static_cast<int64_t>(head) * p.units + u.gqb0 + u.block) * (2 * kT);
  const int64_t base = (static_cast<int64_t>(u.start + u.block * kT) * p.num_heads + head) * D + part * 8;
  uint4 a[kSteps], b[kSteps];
  float bias[kSteps];
  bool none = false;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int r = r0 + i * kRowsAtOnce;
    a[i] = b[i] = make_uint4(0, 0, 0, 0);
    bias[i] = -INFINITY;
    if (r < rows) {
      const int64_t at = base + static_cast<int64_t>(r) * p.num_heads * D;
      a[i] = *reinterpret_cast<const uint4*>(p.dout + at);
      b[i] = *reinterpret_cast<const uint4*>(p.out + at);
      bias[i] = -p.lse[static_cast<int64_t>(head) * p.total_tokens + u.start + u.block * kT + r] * kLog2e;
    }
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {  // an lse of -inf has no reciprocal sum; one of +inf no probability
    if (isinf(bias[i])) bias[i] = -INFINITY;
    none = none || (r0 + i * kRowsAtOnce < rows && takes_no_part(bias[i]));
  }
  const uint32_t some = __syncthreads_or(none) ? 1u : 0u;
  if (r0 == 0 && !takes_no_part(bias[0])) bias[0] = __uint_as_float((__float_as_uint(bias[0]) & ~1u) | some);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int r = r0 + i * kRowsAtOnce;
    const uint32_t x[4] = {a[i].x, a[i].y, a[i].z, a[i].w}, y[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
    uint4 v4 = make_uint4(0, 0, 0, 0);
    if (u.S == 1 && r == 0)
      v4 = *reinterpret_cast<const uint4*>(
          p.v + (static_cast<int64_t>(u.start) * p.num_kv_heads + head / (p.num_heads / p.num_kv_heads)) * D + part * 8);
    const uint32_t z[4] = {v4.x, v4.y, v4.z, v4.w};
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 g = unpack_bf16x2(x[k]), o = unpack_bf16x2(y[k]), v = unpack_bf16x2(z[k]);
      sum = fmaf(g.x, o.x - v.x, sum);
      sum = fmaf(g.y, o.y - v.y, sum);
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if (part == 0) {
      dst[r] = bias[i];
      dst[kT + r] = takes_no_part(bias[i]) ? 0.f : -sum;
    }
  }
}

// One 1-D bulk copy global -> shared, counted on `bar` (16-byte aligned).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
      : "memory");
}

// All threads of the cluster; orders shared-memory accesses before it against
// those after it. (Every path to it is bounded in time.)
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}

// 16 bytes at this CTA's shared-memory address `addr` in the CTA of rank `rank`.
__device__ __forceinline__ float4 ld_cluster(uint32_t addr, int rank) {
  float4 v;
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %4, %5;\n ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}

template <int D, bool Q>
__device__ __forceinline__ void run_role(const CUtensorMap* tmFixA, const CUtensorMap* tmFixB,
                                         const CUtensorMap* tmRingA, const CUtensorMap* tmRingB, const Params& p,
                                         uint8_t* smem, int head, int rank) {
  using L = Layout<D>;
  constexpr int kAccs = Q ? 1 : 2;
  constexpr bool kThree = Q || D == 64;           // three score regions; else two, which change places
  constexpr uint32_t kColAccB = kColAccA + D;     // kv role
  constexpr int kPartRow = D + 4;         // floats; the pad spreads the rows over the banks
  constexpr int kStageRow = 2 * D + 16;  // bytes, likewise
  static_assert(2 * kT * kPartRow * 4 <= L::kRows, "the results are staged in the tiles' shared memory");
  Ctl& ctl = *reinterpret_cast<Ctl*>(smem + L::kCtl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Unit u = ctl.u;
  const int nt = (u.S + kT - 1) / kT;  // tiles of the sequence
  const int group = p.num_heads / p.num_kv_heads;
  const int split = p.split[Q ? 1 : 0];
  volatile int* abort_flag = &ctl.abort_flag;
  const uint32_t tmem = ctl.tmem_base;
  auto a_full = [&](int i) { return smem_u32(&ctl.a_full[i]); };
  auto a_empty = [&](int i) { return smem_u32(&ctl.a_empty[i]); };
  auto b_full = [&](int i) { return smem_u32(&ctl.b_full[i]); };
  auto b_empty = [&](int i) { return smem_u32(&ctl.b_empty[i]); };
  const uint32_t dp_full = smem_u32(&ctl.dp_full), dp_done = smem_u32(&ctl.dp_done);
  auto s_full = [&](int j) { return smem_u32(&ctl.s_full[j & 1]); };    // phase j >> 1
  auto p_full = [&](int j) { return smem_u32(&ctl.p_full[j & 1]); };    // phase j >> 1
  auto ds_full = [&](int j) { return smem_u32(&ctl.ds_full[j & 1]); };  // phase j >> 1
  const uint32_t fix_full = smem_u32(&ctl.fix_full), acc_full = smem_u32(&ctl.acc_full);
  // Tile j's ring A stage is free, which also says that the products that read
  // its P and dS (or dS's parts), and (kv role) its ring B stage and row values, are complete.
  auto acc_done = [&](int j) { return smem_u32(&ctl.a_empty[j % kAStages]); };  // phase j / kAStages
  // The region of S of tile j, then of its P and dS or of dS's parts; and that of dP.
  auto col_s = [&](int j) { return j & 1 ? (kThree ? kColZ : kColY) : kColX; };
  auto col_dp = [&](int j) { return kThree || !(j & 1) ? kColY : kColX; };

  if (warp == kTmaWarp) {
    // ------------------------------------------------------------ producer
    int it = 0, b_issued = 0;  // ring tiles issued
    bool ok = true;
    if (lane == 0) {
      mbar_arrive_expect_tx(fix_full, 2 * L::kTileBytes);
      for (int ch = 0; ch < L::kChunks; ++ch) {
        tma_load_3d(smem_u32(smem + L::kFixA + ch * L::kChunkBytes), tmFixA, fix_full, ch * 64, head,
                    u.start + u.block * kT);
        tma_load_3d(smem_u32(smem + L::kFixB + ch * L::kChunkBytes), tmFixB, fix_full, ch * 64, head,
                    u.start + u.block * kT);
      }
    }
    if (!Q) wait_for_rows();  // the ring brings the row values as well
    const int ring_heads = Q ? 1 : group;
    const int chunks = (nt + 31) / 32;
    // Bits of the tiles base .. base+31 that this CTA's block skips.
    auto skipped = [&](int step) -> uint32_t {
      const int g = step / chunks, base = (step % chunks) * 32;
      if (!p.bitmap || step >= ring_heads * chunks) return 0u;
      if (Q) {
        const int64_t unit = static_cast<int64_t>(head) * u.nq_total + u.gqb0 + u.block;
        return p.bitmap[unit * p.bitmap_words + base / 32];
      }
      const int i = base + lane;
      const int64_t unit = static_cast<int64_t>(head * group + g) * u.nq_total + u.gqb0 + i;
      const uint32_t w = i < nt ? p.bitmap[unit * p.bitmap_words + u.block / 32] : 0u;
      return __ballot_sync(kFull, (w >> (u.block & 31)) & 1u);
    };
    uint32_t next = skipped(0);
    for (int step = 0; step < ring_heads * chunks; ++step) {
      const int base = (step % chunks) * 32;
      const int ring_head = Q ? head / group : head * group + step / chunks;
      uint32_t keep = ~next;
      if (nt - base < 32) keep &= (1u << (nt - base)) - 1u;
      if (split > 1) {  // this rank's tiles: every split-th of the block's walk
        const uint32_t every = split == 2 ? 0x55555555u : (split == 4 ? 0x11111111u : 0x01010101u);
        keep &= every << ((rank - ((step / chunks) * nt + base)) & (split - 1));
      }
      next = skipped(step + 1);
      if (lane == 0) {
        for (; keep && ok; keep &= keep - 1) {
          const int t = base + __ffs(static_cast<int>(keep)) - 1;
          const int sa = it % kAStages, sb = it % kBStages;
          if (it >= kAStages && !(ok = wait_bar(a_empty(sa), ((it / kAStages) - 1) & 1, abort_flag, p.status))) break;
          ctl.info[sa] = min(kT, u.S - t * kT);
          mbar_arrive_expect_tx(a_full(sa), L::kTileBytes);
          for (int ch = 0; ch < L::kChunks; ++ch)
            tma_load_3d(smem_u32(smem + L::kRingA + sa * L::kTileBytes + ch * L::kChunkBytes), tmRingA, a_full(sa),
                        ch * 64, ring_head, u.start + t * kT);
          const int n = it++;
          if (n >= kBStages) {
            const int old = n - kBStages;  // the tile that had this ring B stage (kv role: and row values)
            if (!(ok = Q ? wait_bar(b_empty(sb), (old / kBStages) & 1, abort_flag, p.status)
                         : wait_bar(acc_done(old), (old / kAStages) & 1, abort_flag, p.status)))
              break;
          }
          mbar_arrive_expect_tx(b_full(sb), L::kTileBytes + (Q ? 0 : L::kRowBytes));
          if (!Q)
            bulk_load(smem_u32(smem + L::kRows + sb * L::kRowBytes),
                      p.rows + (static_cast<int64_t>(ring_head) * p.units + u.gqb0 + t) * (2 * kT), L::kRowBytes,
                      b_full(sb));
          for (int ch = 0; ch < L::kChunks; ++ch)
            tma_load_3d(smem_u32(smem + L::kRingB + sb * L::kTileBytes + ch * L::kChunkBytes), tmRingB, b_full(sb),
                        ch * 64, ring_head, u.start + t * kT);
          ++b_issued;
        }
      }
      ok = __shfl_sync(kFull, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
    }
    if (lane == 0) {
      if (ok) {  // say that there are no more tiles
        const int sa = it % kAStages;
        if (it < kAStages || (ok = wait_bar(a_empty(sa), ((it / kAStages) - 1) & 1, abort_flag, p.status))) {
          ctl.info[sa] = -1;
          mbar_arrive(a_full(sa));
        }
      }
      if (!ok) {  // drain the loads still in flight before shared memory goes away
        drain_wait(fix_full, 0, p.status);
        for (int i = 0; i < kAStages; ++i)
          if (it > i) drain_wait(a_full(i), ((it - 1 - i) / kAStages) & 1, p.status);
        for (int i = 0; i < kBStages; ++i)
          if (b_issued > i) drain_wait(b_full(i), ((b_issued - 1 - i) / kBStages) & 1, p.status);
      }
    }
  } else if (warp < kEwWarp) {
    // ------------------------------------------------------ tcgen05 issuers
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_bf16_f32(kT, kT, false);
      constexpr uint32_t idesc_acc = idesc_bf16_f32(kT, D, true);
      // dst = fix ring^T, both K-major with 128-byte swizzle: 32 B of d per MMA.
      auto product = [&](uint32_t dst, int fix, int ring) {
        const uint64_t da = smem_desc_sw128(smem_u32(smem + fix), 16, 1024);
        const uint64_t db = smem_desc_sw128(smem_u32(smem + ring), 16, 1024);
        const uint32_t a_lo = static_cast<uint32_t>(da), b_lo = static_cast<uint32_t>(db);
        const uint64_t a_hi = da & 0xFFFFFFFF00000000ull, b_hi = db & 0xFFFFFFFF00000000ull;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = ((ks >> 2) * L::kChunkBytes + (ks & 3) * 32) >> 4;
          mma_ss(tmem + dst, a_hi | (a_lo + off), b_hi | (b_lo + off), idesc_s, ks > 0 ? 1u : 0u);
        }
      };
      // acc += E ring with E (bf16 pairs, 128 x 128) in TMEM and the ring tile
      // MN-major (d contiguous), 16 of its rows per MMA; the two halves of E
      // are 64 columns apart.
      auto accumulate = [&](uint32_t acc, uint32_t e, int ring, bool more) {
        const uint64_t db = smem_desc_sw128(smem_u32(smem + ring), L::kChunkBytes, 1024);
        const uint32_t b_lo = static_cast<uint32_t>(db);
        const uint64_t b_hi = db & 0xFFFFFFFF00000000ull;
#pragma unroll
        for (int ks = 0; ks < kT / 16; ++ks)
          mma_ts(tmem + acc, tmem + e + ks * 8 + (ks >= 4 ? 32 : 0), b_hi | (b_lo + (ks * 16 * 128 >> 4)), idesc_acc,
                 (more || ks > 0) ? 1u : 0u);
      };
      auto wait = [&](uint32_t bar, int parity) { return wait_bar(bar, parity, abort_flag, p.status); };
      auto ring_a = [&](int j) { return L::kRingA + (j % kAStages) * L::kTileBytes; };
      auto ring_b = [&](int j) { return L::kRingB + (j % kBStages) * L::kTileBytes; };
      // True when tile j exists; its A tile has landed then.
      bool ok = true;
      auto has = [&](int j) {
        ok = wait(a_full(j % kAStages), (j / kAStages) & 1);
        return ok && *static_cast<volatile int*>(&ctl.info[j % kAStages]) >= 0;
      };
      if (warp == kSWarp) {
        // S(j), once P and dS of tile j-2 are used (three regions) or dP(j-1) has been read (two).
        ok = wait(fix_full, 0);
        for (int j = 0; ok && has(j); ++j) {
          if (kThree ? j > 1 && !(ok = wait(acc_done(j - 2), ((j - 2) / kAStages) & 1))
                     : j > 0 && !(ok = wait(dp_done, (j - 1) & 1)))
            break;
          tc_fence_after();
          product(col_s(j), L::kFixA, ring_a(j));
          tc_commit(s_full(j));
        }
      } else if (warp == kDPWarp) {
        // dP(j), once dP(j-1) has been read (three regions), or P and dS of tile j-1 used (two).
        ok = wait(fix_full, 0);
        for (int j = 0; ok && has(j); ++j) {
          if (!(ok = wait(b_full(j % kBStages), (j / kBStages) & 1))) break;
          if (j > 0 && !(ok = kThree ? wait(dp_done, (j - 1) & 1) : wait(acc_done(j - 1), ((j - 1) / kAStages) & 1)))
            break;
          tc_fence_after();
          product(col_dp(j), L::kFixB, ring_b(j));
          tc_commit(dp_full);
          if (Q) tc_commit(b_empty(j % kBStages));
        }
      } else {  // kAccWarp
        // q role: dQ += hi(j) K_j, dQ += lo(j) K_j. kv role: dV += P(j)^T dO_j, dK += dS(j)^T Q_j.
        for (int j = 0; ok && has(j); ++j) {
          if (!(ok = wait(p_full(j), (j >> 1) & 1))) break;
          tc_fence_after();
          accumulate(Q ? kColAccA : kColAccB, col_s(j), Q ? ring_a(j) : ring_b(j), j > 0);
          if (!(ok = wait(ds_full(j), (j >> 1) & 1))) break;
          tc_fence_after();
          accumulate(kColAccA, col_s(j) + 32, ring_a(j), Q || j > 0);
          tc_commit(acc_done(j));
        }
        if (ok) tc_commit(acc_full);
      }
      if (!ok) {  // let every MMA issued so far finish before TMEM is released
        const uint32_t drain = smem_u32(&ctl.drain[warp - kSWarp]);
        tc_commit(drain);
        drain_wait(drain, 0, p.status);
      }
    }
  } else {
    // -------------------------------------------------------- element-wise
    const int half = (warp - kEwWarp) >> 2;  // columns [64 half, 64 half + 64)
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    float row_bias = 0.f, row_ndelta = 0.f;  // q role: this thread's row
    if (Q) {
      wait_for_rows();
      const float* r = p.rows + (static_cast<int64_t>(head) * p.units + u.gqb0 + u.block) * (2 * kT);
      row_bias = r[row];
      row_ndelta = r[kT + row];
    }
    const float2 c2 = make_float2(p.c2, p.c2), minus_one = make_float2(-1.f, -1.f);
    // Waits are looked at ahead of their time, over work that does not need
    // them. The check right behind the arrival on dp_done also keeps the
    // compiler from moving that arrival behind the arithmetic that follows it.
    bool ok = warp_wait(a_full(0), 0, abort_flag, p.status);
    int j = 0, valid = ok ? *static_cast<volatile int*>(&ctl.info[0]) : -1;
    bool s_seen = false, rows_seen = false;
    int sa = 0, a_phase = 0;  // j % kAStages, (j / kAStages) & 1
    for (; ok && valid >= 0; ++j) {
      const int sa_next = sa + 1 == kAStages ? 0 : sa + 1, a_phase_next = a_phase ^ (sa_next == 0 ? 1 : 0);
      const float* tile_rows = reinterpret_cast<const float*>(smem + L::kRows + (j % kBStages) * L::kRowBytes);
      const float* rows = tile_rows + half * 64;
      if (!Q && !(ok = warp_wait_seen(rows_seen, b_full(j % kBStages), (j / kBStages) & 1, abort_flag, p.status))) break;
      const float first_bias = Q ? 0.f : tile_rows[0];
      if (!(ok = warp_wait_seen(s_seen, s_full(j), (j >> 1) & 1, abort_flag, p.status))) break;
      tc_fence_after();
      uint32_t s[64];
      tmem_ld_x64_async(lanes + col_s(j) + half * 64, s);
      const bool a_seen = mbar_test_wait(a_full(sa_next), a_phase_next);
      const bool gaps = !Q && some_take_no_part(first_bias), masked = gaps || valid < kT;
      if (masked) {
        // The tile ends past the sequence, or (kv role) rows of it take no part.
        // Those are summation rows of the accumulating products: they must be
        // zeros, not whatever memory holds (NaN times a zero probability is NaN).
        const int first = gaps ? 0 : valid;
        const int words = (kT - first) * 8;  // 16-byte words of a chunk's rows from there on
        for (int i = threadIdx.x - 32 * kEwWarp; i < L::kChunks * words; i += kEwThreads) {
          const int at = (i / words) * L::kChunkBytes + first * 128 + (i % words) * 16;
          if (!Q && !takes_no_part(tile_rows[first + i % words / 8])) continue;
          *reinterpret_cast<uint4*>(smem + L::kRingA + sa * L::kTileBytes + at) = make_uint4(0, 0, 0, 0);
          if (!Q)
            *reinterpret_cast<uint4*>(smem + L::kRingB + (j % kBStages) * L::kTileBytes + at) = make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      tmem_wait_ld_tied(s);
      if (masked) {  // no probability there, whatever stands there
#pragma unroll
        for (int i = 0; i < 64; ++i)
          if (Q ? half * 64 + i >= valid : takes_no_part(rows[i])) s[i] = __float_as_uint(-INFINITY);
      }
      const bool dp_seen = mbar_test_wait(dp_full, j & 1);
      // P = 2^(c2 S - L log2 e)
      uint32_t pk[32];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float4 b4 = Q ? make_float4(row_bias, row_bias, row_bias, row_bias) : reinterpret_cast<const float4*>(rows)[i];
        const float2 e0 = ffma2(make_float2(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1])), c2,
                                make_float2(b4.x, b4.y));
        const float2 e1 = ffma2(make_float2(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])), c2,
                                make_float2(b4.z, b4.w));
        const float2 p0 = make_float2(ex2_approx(e0.x), ex2_approx(e0.y));
        const float2 p1 = make_float2(ex2_approx(e1.x), ex2_approx(e1.y));
        s[4 * i] = __float_as_uint(p0.x);
        s[4 * i + 1] = __float_as_uint(p0.y);
        s[4 * i + 2] = __float_as_uint(p1.x);
        s[4 * i + 3] = __float_as_uint(p1.y);
        if (!Q) {
          pk[2 * i] = pack_bf16x2(p0.x, p0.y);
          pk[2 * i + 1] = pack_bf16x2(p1.x, p1.y);
        }
      }
      if (!Q) {
        tmem_st_x32(lanes + col_s(j) + half * 64, pk);
        warp_arrive(p_full(j), lane);
      }
      if (!(ok = warp_wait_seen(dp_seen, dp_full, j & 1, abort_flag, p.status))) break;
      tc_fence_after();
      uint32_t d[64];
      tmem_ld_x64_async(lanes + col_dp(j) + half * 64, d);
      tmem_wait_ld_tied(d);
      warp_arrive(dp_done, lane);
      if (!(ok = warp_wait_seen(a_seen, a_full(sa_next), a_phase_next, abort_flag, p.status))) break;
      const int valid_next = *static_cast<volatile int*>(&ctl.info[sa_next]);
      if (kThree) s_seen = mbar_test_wait(s_full(j + 1), ((j + 1) >> 1) & 1);
      if (!Q)
        rows_seen = mbar_test_wait(b_full((j + 1) % kBStages), ((j + 1) / kBStages) & 1);
      if (masked) {
#pragma unroll
        for (int i = 0; i < 64; ++i)
          if (Q ? half * 64 + i >= valid : takes_no_part(rows[i])) d[i] = 0u;
        if (u.S == 1) d[0] = half == 0 ? 0u : d[0];  // -D holds dP - D (see rows_kernel)
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float4 n4 = Q ? make_float4(row_ndelta, row_ndelta, row_ndelta, row_ndelta)
                            : reinterpret_cast<const float4*>(rows + kT)[i];
        const float2 x = fmul2(make_float2(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1])),
                               fadd2(make_float2(__uint_as_float(d[4 * i]), __uint_as_float(d[4 * i + 1])),
                                     make_float2(n4.x, n4.y)));
        const float2 y = fmul2(make_float2(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])),
                               fadd2(make_float2(__uint_as_float(d[4 * i + 2]), __uint_as_float(d[4 * i + 3])),
                                     make_float2(n4.z, n4.w)));
        pk[2 * i] = pack_bf16x2(x.x, x.y);
        pk[2 * i + 1] = pack_bf16x2(y.x, y.y);
        if (Q) {
          s[4 * i] = __float_as_uint(x.x);
          s[4 * i + 1] = __float_as_uint(x.y);
          s[4 * i + 2] = __float_as_uint(y.x);
          s[4 * i + 3] = __float_as_uint(y.y);
        }
      }
      if (Q) {
        tmem_st_x32(lanes + col_s(j) + half * 64, pk);
        warp_arrive(p_full(j), lane);
#pragma unroll
        for (int i = 0; i < 32; ++i) {  // what rounding left of dS, exact in fp32
          const float2 l = ffma2(unpack_bf16x2(pk[i]), minus_one,
                                 make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])));
          pk[i] = pack_bf16x2(l.x, l.y);
        }
      }
      tmem_st_x32(lanes + col_s(j) + half * 64 + 32, pk);
      warp_arrive(ds_full(j), lane);
      valid = valid_next;
      sa = sa_next;
      a_phase = a_phase_next;
    }

    // Epilogue: this thread's row and half of the D columns of each accumulator.
    const bool any = j > 0;  // no tile was kept: the gradients are zero
    const bool part = any && !(Q && takes_no_part(row_bias));  // nor has a row that takes no part one
    if (ok) ok = warp_wait(acc_full, 0, abort_flag, p.status);
    // Results are staged over the tiles: all loads must have landed. Where tiles
    // were walked the accumulators say so; where none was, the fixed tiles may
    // still be on their way.
    if (ok && !any) ok = warp_wait(fix_full, 0, abort_flag, p.status);
    if (ok) {
      tc_fence_after();
#pragma unroll 1
      for (int a = 0; a < kAccs; ++a) {
        const float f = a ? 1.f : p.scale;
#pragma unroll 1
        for (int ch = 0; ch < D / 64; ++ch) {
          uint32_t o[32];
          tmem_ld_x32(lanes + (a ? kColAccB : kColAccA) + half * (D / 2) + ch * 32, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = part ? o[i] : 0u;
          if (split > 1) {
            uint4* part = reinterpret_cast<uint4*>(smem + ((a * kT + row) * kPartRow + half * (D / 2) + ch * 32) * 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) part[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          } else {
            uint4* part = reinterpret_cast<uint4*>(smem + (a * kT + row) * kStageRow + (half * (D / 2) + ch * 32) * 2);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w[k] = pack_bf16x2(__uint_as_float(o[8 * i + 2 * k]) * f, __uint_as_float(o[8 * i + 2 * k + 1]) * f);
              part[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
      }
    }
    if (split == 1) {  // whole rows of 128 or 256 bytes to memory, not 16 bytes of 32 rows at a time
      named_barrier_sync(1, kEwThreads);  // every element-wise warp comes here, with or without an error
      if (ok) {
        const int heads = Q ? p.num_heads : p.num_kv_heads;
        constexpr int kWords = D / 8;  // 16-byte words of a row
        const int rows = min(kT, u.S - u.block * kT);
        const int64_t base = (static_cast<int64_t>(u.start + u.block * kT) * heads + head) * D;
#pragma unroll 1
        for (int a = 0; a < kAccs; ++a) {
          __nv_bfloat16* dst = (Q ? p.dq : (a ? p.dv : p.dk)) + base;
#pragma unroll 4
          for (int i = threadIdx.x - 32 * kEwWarp; i < rows * kWords; i += kEwThreads)
            *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(i / kWords) * heads * D + i % kWords * 8) =
                *reinterpret_cast<const uint4*>(smem + (a * kT + i / kWords) * kStageRow + i % kWords * 16);
        }
      }
    }
  }

  if (split > 1) {  // the cluster's CTAs each add up a share of the rows
    __syncwarp();
    cluster_sync();
    if (warp >= kEwWarp) {
      const int heads = Q ? p.num_heads : p.num_kv_heads;
      const int r0 = rank * (kT / split);
      constexpr int kWords = D / 4;  // float4 per row
      // Two words at a time, the loads of all ranks before their sums: a remote
      // load takes hundreds of cycles.
      const int words = kAccs * (kT / split) * kWords;
      for (int i0 = threadIdx.x - 32 * kEwWarp; i0 < words; i0 += 2 * kEwThreads) {
        float4 v[2][8];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int i = min(i0 + n * kEwThreads, words - 1);
          const int word = i % kWords, a = i / kWords / (kT / split), row = r0 + i / kWords % (kT / split);
          const uint32_t part = smem_u32(smem + ((a * kT + row) * kPartRow + word * 4) * 4);
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (c < split) v[n][c] = ld_cluster(part, c);
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int i = i0 + n * kEwThreads;
          const int word = i % kWords, a = i / kWords / (kT / split), row = r0 + i / kWords % (kT / split);
          float4 sum = v[n][0];
#pragma unroll
          for (int c = 1; c < 8; ++c)
            if (c < split) sum.x += v[n][c].x, sum.y += v[n][c].y, sum.z += v[n][c].z, sum.w += v[n][c].w;
          if (i < words && u.block * kT + row < u.S) {
            const float f = a ? 1.f : p.scale;
            __nv_bfloat16* dst = (Q ? p.dq : (a ? p.dv : p.dk)) +
                                 (static_cast<int64_t>(u.start + u.block * kT + row) * heads + head) * D + word * 4;
            *reinterpret_cast<uint2*>(dst) =
                make_uint2(pack_bf16x2(sum.x * f, sum.y * f), pack_bf16x2(sum.z * f, sum.w * f));
          }
        }
      }
    }
    cluster_sync();  // no CTA leaves while another still reads its shared memory
  }
}

// blockIdx.x: 128-row block of the batch; blockIdx.y: the K/V heads (kv role,
// the longer one, first), then the query heads (q role), each as often as the
// role is split. A cluster spans blockIdx.y.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
               const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO,
               const __grid_constant__ Params p) {
  using L = Layout<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Ctl& ctl = *reinterpret_cast<Ctl*>(smem + L::kCtl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int y = static_cast<int>(blockIdx.y);
  if (warp == 0) {
    locate(p, static_cast<int>(blockIdx.x), lane, blockIdx.x == 0 && y == 0, ctl.u);
  } else if (warp == kSWarp) {
    tmem_alloc(smem_u32(&ctl.tmem_base), kTmemCols);
    tmem_relinquish();
  } else if (warp == kDPWarp && lane == 0) {
    mbar_init(smem_u32(&ctl.fix_full), 1);
    for (int i = 0; i < kAStages; ++i) {
      mbar_init(smem_u32(&ctl.a_full[i]), 1);
      mbar_init(smem_u32(&ctl.a_empty[i]), 1);
    }
    for (int i = 0; i < kBStages; ++i) {
      mbar_init(smem_u32(&ctl.b_full[i]), 1);
      mbar_init(smem_u32(&ctl.b_empty[i]), 1);
    }
    mbar_init(smem_u32(&ctl.dp_full), 1);
    mbar_init(smem_u32(&ctl.dp_done), 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ctl.s_full[i]), 1);
      mbar_init(smem_u32(&ctl.p_full[i]), 8);
      mbar_init(smem_u32(&ctl.ds_full[i]), 8);
    }
    mbar_init(smem_u32(&ctl.acc_full), 1);
    for (int i = 0; i < 3; ++i) mbar_init(smem_u32(&ctl.drain[i]), 1);
    ctl.abort_flag = 0;
    fence_mbar_init();
  } else if (warp == kAccWarp && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
    prefetch_tmap(&tmdO);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (ctl.u.seq < 0) {  // uniform
    if (threadIdx.x == 0) wait_for_rows();  // no CTA, and so not this kernel, ends before rows_kernel has
    if (warp == kSWarp) tmem_dealloc(ctl.tmem_base, kTmemCols);
    return;
  }

  const int kv_ctas = p.num_kv_heads * p.split[0];
  if (y < kv_ctas)
    run_role<D, false>(&tmK, &tmV, &tmQ, &tmdO, p, smem, y / p.split[0], y % p.split[0]);
  else
    run_role<D, true>(&tmQ, &tmdO, &tmK, &tmV, p, smem, (y - kv_ctas) / p.split[1], (y - kv_ctas) % p.split[1]);

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kSWarp) {
    tc_fence_after();
    tmem_dealloc(ctl.tmem_base, kTmemCols);
  }
}

// ----------------------------------------------------------------- host side

int64_t bound_units(int total_tokens, int batch) { return (static_cast<int64_t>(total_tokens) + kT - 1) / kT + batch; }

template <int D>
int launch(Params p, const void* q, const void* k, const void* v, cudaStream_t stream) {
  CUtensorMap tq, tk, tv, tdo;
  if (!internal::bf16_tensor_map(&tq, q, p.total_tokens, p.num_heads, D) ||
      !internal::bf16_tensor_map(&tk, k, p.total_tokens, p.num_kv_heads, D) ||
      !internal::bf16_tensor_map(&tv, v, p.total_tokens, p.num_kv_heads, D) ||
      !internal::bf16_tensor_map(&tdo, p.dout, p.total_tokens, p.num_heads, D))
    return internal::fail("cuTensorMapEncodeTiled failed or the driver entry point is unavailable");
  constexpr int smem = Layout<D>::kAlloc;
  cudaError_t e = cudaFuncSetAttribute(bwd_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return internal::fail(e);
  // Blocks are split as long as all CTAs still run at once (us, D = 128 unless
  // said, unsplit / split: 1024 tokens of 2 heads, D = 64, 21.3 / 15.5 in 4;
  // 1024 tokens of 8 query heads over 2 K/V heads 66.1 / 30.8 in 4, over one
  // 117.4 / 37.7 in 8). Beyond that a split costs (2048 tokens of 8 heads 69.1 / 80.6 in
  // 2), except where several query heads to a K/V head make the kv role's walk
  // longer than a fair share of the work: then that role alone is split.
  int split = 1, q_split = 1;
  const int64_t kv_blocks = static_cast<int64_t>(p.units) * p.num_kv_heads;
  const int64_t q_blocks = static_cast<int64_t>(p.units) * p.num_heads;
  const int64_t group = p.num_heads / p.num_kv_heads;
  const int64_t tiles = (static_cast<int64_t>(p.max_seqlen) + kT - 1) / kT;
  // Per tile the kv role takes about 7/5 of the q role's time.
  const bool long_walk = 7 * group * tiles * kSMs > (7 * group * kv_blocks + 5 * q_blocks) * tiles;
  for (int s = 2; s <= 8 && s <= group * tiles; s *= 2) {
    const bool heads_fill = p.num_heads % s == 0;  // clusters of whole q role blocks
    if ((kv_blocks + q_blocks) * s <= kSMs) {
      split = q_split = s;
    } else if (heads_fill && (kv_blocks * s + q_blocks <= kSMs ||
                              (s <= group && long_walk && 4 * kv_blocks * s <= 5 * kSMs))) {
      split = s;
      q_split = 1;
    } else {
      break;
    }
  }
  p.split[0] = split;
  p.split[1] = q_split;
  const unsigned units = static_cast<unsigned>(p.units);
  rows_kernel<D><<<dim3(units, static_cast<unsigned>(p.num_heads)), 256, 0, stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return internal::fail(e);
  cudaLaunchConfig_t config{};
  config.gridDim = dim3(units, static_cast<unsigned>(p.num_kv_heads * p.split[0] + p.num_heads * p.split[1]));
  config.blockDim = dim3(kThreads);
  config.dynamicSmemBytes = smem;
  config.stream = stream;
  // An early start gains 3 to 5 us in batches that leave SMs free or are split
  // (128 x 1 x 128 16.5 / 12.8 us, 512 x 4 20.9 / 16.9), and costs as much when
  // long unsplit walks take nearly every SM (1000 x 8 28.3 / 31.3, 1700 x 5 39.5 /
  // 47.3): a CTA takes a whole SM, and those that find rows_kernel on theirs wait.
  const bool early = split > 1 || 2 * static_cast<int64_t>(config.gridDim.x) * config.gridDim.y <= kSMs;
  cudaLaunchAttribute attrs[2]{};
  attrs[0].id = cudaLaunchAttributeClusterDimension;
  attrs[0].val.clusterDim.x = 1;
  attrs[0].val.clusterDim.y = static_cast<unsigned>(split);
  attrs[0].val.clusterDim.z = 1;
  attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[1].val.programmaticStreamSerializationAllowed = early ? 1 : 0;
  config.attrs = attrs;
  config.numAttrs = early ? 2 : 0;  // neither split nor early: a plain launch
  e = cudaLaunchKernelEx(&config, bwd_kernel<D>, tq, tk, tv, tdo, p);
  return e == cudaSuccess ? SSA_OK : internal::fail(e);
}

}  // namespace
}  // namespace ssa

using namespace ssa;

extern "C" int64_t ssa_bwd_workspace_bytes(int total_tokens, int batch, int num_heads) {
  if (total_tokens < 0 || batch < 1 || num_heads < 1) return SSA_ERR_INVALID_ARG;
  return bound_units(total_tokens, batch) * num_heads * (2 * kT * static_cast<int64_t>(sizeof(float)));
}

int internal::check_backward(const Backward& a) {
  if (!a.cu_seqlens || a.batch < 1 || a.total_tokens < 0 || a.max_seqlen < 0 || a.num_kv_heads < 1 ||
      a.num_heads < 1 || a.num_heads % a.num_kv_heads != 0 || a.num_heads > 65535 - a.num_kv_heads)
    return SSA_ERR_INVALID_ARG;
  if (std::isnan(a.softmax_scale) || std::isinf(a.softmax_scale)) return SSA_ERR_INVALID_ARG;
  if (a.head_dim != 64 && a.head_dim != 128) return SSA_ERR_UNSUPPORTED;
  if (a.decision_bitmap && (a.num_qblocks < 0 || a.max_seqlen < 1)) return SSA_ERR_INVALID_ARG;
  if (a.total_tokens == 0) return SSA_OK;
  if (bound_units(a.total_tokens, a.batch) > 0x7FFFFFFF) return SSA_ERR_INVALID_ARG;
  if (a.workspace_bytes < ssa_bwd_workspace_bytes(a.total_tokens, a.batch, a.num_heads)) return SSA_ERR_INVALID_ARG;
  for (const void* ptr : {a.dout, a.q, a.k, a.v, a.out, static_cast<const void*>(a.dq), static_cast<const void*>(a.dk),
                          static_cast<const void*>(a.dv), static_cast<const void*>(a.workspace)}) {
    if (!ptr) return SSA_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(ptr) & 15u) return SSA_ERR_UNSUPPORTED;
  }
  if (!a.lse) return SSA_ERR_INVALID_ARG;
  return device_pointers({a.dout, a.q, a.k, a.v, a.out, a.lse, a.cu_seqlens, a.decision_bitmap, a.dq, a.dk, a.dv,
                          a.workspace});
}

int internal::launch_backward(const Backward& a, cudaStream_t stream) {
  Params p{};
  if (const int rc = status_word(&p.status); rc != SSA_OK) return rc;
  p.cu_seqlens = a.cu_seqlens;
  p.bitmap = a.decision_bitmap;
  p.dq = static_cast<__nv_bfloat16*>(a.dq);
  p.dk = static_cast<__nv_bfloat16*>(a.dk);
  p.dv = static_cast<__nv_bfloat16*>(a.dv);
  p.out = static_cast<const __nv_bfloat16*>(a.out);
  p.dout = static_cast<const __nv_bfloat16*>(a.dout);
  p.v = static_cast<const __nv_bfloat16*>(a.v);
  p.lse = a.lse;
  p.rows = static_cast<float*>(a.workspace);
  p.batch = a.batch;
  p.total_tokens = a.total_tokens;
  p.max_seqlen = a.max_seqlen;
  p.num_heads = a.num_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.max_tiles = static_cast<int>((static_cast<int64_t>(a.max_seqlen) + kT - 1) / kT);
  p.bitmap_words = (p.max_tiles + 31) / 32;
  p.units = static_cast<int>(bound_units(a.total_tokens, a.batch));
  p.nq_check = a.decision_bitmap ? a.num_qblocks : -1;
  const double c =
      a.softmax_scale > 0.f ? static_cast<double>(a.softmax_scale) : 1.0 / std::sqrt(static_cast<double>(a.head_dim));
  p.scale = static_cast<float>(c);
  p.c2 = static_cast<float>(c * 1.4426950408889634073599246810019);
  return a.head_dim == 64 ? launch<64>(p, a.q, a.k, a.v, stream) : launch<128>(p, a.q, a.k, a.v, stream);
}

extern "C" int ssa_bwd(const void* dout, const void* q, const void* k, const void* v, const void* out,
                       const float* lse, const int32_t* cu_seqlens, int batch, int total_tokens, int max_seqlen,
                       int num_heads, int num_kv_heads, int head_dim, float softmax_scale,
                       const uint32_t* decision_bitmap, int num_qblocks, void* dq, void* dk, void* dv,
                       void* workspace, int64_t workspace_bytes, void* stream) {
  const internal::Backward a{dout, q, k, v, out, lse, cu_seqlens, batch, total_tokens, max_seqlen, num_heads,
                             num_kv_heads, head_dim, softmax_scale, decision_bitmap, num_qblocks, dq, dk, dv,
                             workspace, workspace_bytes};
  if (const int rc = internal::check_backward(a); rc != SSA_OK || total_tokens == 0) return rc;
  return internal::launch_backward(a, static_cast<cudaStream_t>(stream));
}
