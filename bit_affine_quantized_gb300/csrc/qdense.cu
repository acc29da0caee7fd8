// Dense projection of 8-bit rows with an 8-bit matrix, a scale per row and per
// output channel (moe_qdense_forward):
//
//   y[t, n] = cap(xs[t] * ws[n] * sum_k x[t, k] w[n, k]),  cap(z) = c tanh(z / c) or z
//
// qdense_rows_kernel: one or two rows, and 3 to 8 rows wider than 12272, for whose
// widened codes the next kernel has no room.  A warp takes kR channels; each lane loads 16 bytes of every
// channel's row (one 512-byte run per warp and channel) and multiplies them
// with the rows' codes in shared memory by dp4a, so the sums are exact 32-bit
// integers (at most 128 * 128 * 16384 = 2^28 in magnitude).  HBM bound: 1 x
// 262144 x 2816 in 107 us, 6.9 TB/s of codes; 1 x 4096 x 2816 in 3.3 us; 3 and 8 x
// 65536 x 12288 in 119 and 133 us, 6.8 and 6.1 TB/s.
//
// qdense_few_kernel: 3 to 8 rows, mma.sync with the codes widened to fp16 in
// registers on their way from global memory; the fp32 sums go to integers
// every 1024 of K, so they stay exact.  HBM bound (8 x 262144 x 2816: 119 us;
// dp4a took 186).  Rows wider than 8192 leave it less and less of that rate (8 x
// 65536 x 8192 91 us, 5.9 TB/s; x 10240 146; x 12272 379, 2.1 TB/s).  From 9 rows
// on mma.sync's rate bounds it (16 rows: 155 us against 122 in the next kernel).
//
// qdense_mma_kernel: more rows, on the 5th-generation tensor cores.  sm_103a
// has no 8-bit integer form of tcgen05.mma; 8-bit codes are exact in fp16, so
// the products run as fp16 with fp32 sums (exact while the partial sums stay
// below 2^24).  The rows are widened to fp16 once per call by
// qdense_widen_kernel, or, where every block has one tile or less, by each
// block; the matrix, the larger operand, is read as 8-bit codes
// and widened on its way into the tensor cores:
//   weights warp   TMA: 128 channels x 128 codes per stage
//   rows warp      TMA: up to 128 rows x 128 fp16 per stage and block
//   8 widen warps  four to a stage, a channel per thread: 128 codes from shared
//                  memory to fp16 pairs in registers to the A operand in
//                  tensor memory
//   MMA warp       tcgen05.mma, M = 128 channels (A in tensor memory),
//                  N = rows (B in shared memory), fp32 sums in tensor memory
//   8 finish warps the sums times both scales, the softcap, the store
// A in tensor memory keeps the widened codes out of shared memory, whose
// bandwidth is what a 128 x 256 fp16 tile asks most of.  Up to 64 rows HBM
// bounds it (24 x 262144 x 2816: 123 us with a bf16 output, 6.0 TB/s of
// codes; 14 rounds of tiles for 13.5 rounds of work are 4 of it, the stores of
// the outputs 5).
// More rows: a pair of blocks on a tile of 256 channels, each with 128 of them in
// its tensor memory and half of the rows in its shared memory, which both read
// (cta_group::2).  A 256-row stage brings 48 KB into an SM's shared memory, 768
// clocks at 64 bytes each; single blocks would bring 80 KB, 1280 clocks, more
// than the stage's MMAs (1024), and took 4 to 9 % longer.  Of 4096 x 4096 x
// 2816's 60 us (1570 TFLOP/s; a library product of fp16 operands takes 53 us on
// such integers, 60 us on random values) the widening of the rows is 6, the
// stores of the outputs 6, and the rest runs at the rate that a library product
// reaches.
// Few tiles: the blocks of a cluster share a tile, each takes a part of K, and
// the parts are added through distributed shared memory in rank order.
#include <cuda.h>
#include <math.h>
#include <string.h>

#include "dense.cuh"
#include "fused.cuh"
#include "kernels.h"
#include "tma_maps.h"

namespace moe {

namespace {
constexpr int kQdWarps = 8;
constexpr int kQdThreads = kQdWarps * 32;
constexpr int kQdRowsMax = 8;  // rows that the dp4a and mma.sync kernels take

__device__ __forceinline__ int4 qd_stream(const int8_t *p) {
  int4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ float qd_value(const QdenseArgs &a, float acc, float xs, float ws) {
  const float v = __fmul_rn(__fmul_rn(acc, xs), ws);
  return a.softcap > 0.f ? a.softcap * tanhf(v / a.softcap) : v;
}
__device__ __forceinline__ void qd_put(const QdenseArgs &a, int t, int n, float acc, float xs, float ws) {
  const float v = qd_value(a, acc, xs, ws);
  const size_t o = (size_t)t * a.N + n;
  if (a.y32) a.y32[o] = v;
  if (a.y) a.y[o] = float_to_bf16_bits(v);
}
// The same of an integer sum.
__device__ __forceinline__ void qd_store(const QdenseArgs &a, int t, int n, int acc, float xs, float ws) {
  qd_put(a, t, n, (float)acc, xs, ws);
}

// kT rows, kR channels per warp; kAhead 16-byte pieces of each channel's row
// are requested before the first is used (those of a warp's first channels
// before the rows' codes have arrived).
template <int kT, int kR, int kAhead>
__global__ void __launch_bounds__(kQdThreads) qdense_rows_kernel(const QdenseArgs a) {
  extern __shared__ __align__(16) int4 qsm[];  // [kT][K / 16]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int K = a.K, nck = K / 16, nt = min(kT, a.T);
  const bool tracer = blockIdx.x == 0 && tid == 0;
  if (tracer) trace_min(a.trace, kTrEntry);
  pdl_wait();
  pdl_launch_dependents();
  if (tracer) trace_min(a.trace, kTrWaited);
  const int units = (a.N + kR - 1) / kR;
  int u = blockIdx.x * kQdWarps + warp;
  int4 w[kR][kAhead];
  auto request = [&](int n0, int c0) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int c = c0 + 32 * j + lane;
#pragma unroll
      for (int r = 0; r < kR; ++r)  // channels past N: discarded below
        w[r][j] = c < nck ? qd_stream(a.w + (size_t)min(n0 + r, a.N - 1) * K + 16 * c) : make_int4(0, 0, 0, 0);
    }
  };
  if (u < units) request(u * kR, 0);
  const int4 *x4 = reinterpret_cast<const int4 *>(a.x);
  for (int i = tid; i < kT * nck; i += kQdThreads) qsm[i] = i < nt * nck ? __ldcg(x4 + i) : make_int4(0, 0, 0, 0);
  __syncthreads();
  for (bool first = true; u < units; u += gridDim.x * kQdWarps, first = false) {
    const int n0 = u * kR;
    if (!first) request(n0, 0);
    int acc[kR][kT];
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
      for (int t = 0; t < kT; ++t) acc[r][t] = 0;
    for (int c0 = 0; c0 < nck; c0 += 32 * kAhead) {
      if (c0 > 0) request(n0, c0);
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int c = min(c0 + 32 * j + lane, nck - 1);  // past the row: the weights are zero
#pragma unroll
        for (int t = 0; t < kT; ++t) {
          const int4 x = qsm[t * nck + c];
#pragma unroll
          for (int r = 0; r < kR; ++r)
            acc[r][t] = __dp4a(w[r][j].w, x.w,
                               __dp4a(w[r][j].z, x.z, __dp4a(w[r][j].y, x.y, __dp4a(w[r][j].x, x.x, acc[r][t]))));
        }
      }
    }
    // lane r * kT + t ends with sum (r, t)
    int mine = 0;
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
      for (int t = 0; t < kT; ++t) {
        const int s = __reduce_add_sync(0xffffffffu, acc[r][t]);
        if (lane == r * kT + t) mine = s;
      }
    const int r = lane / kT, t = lane % kT;
    if (r < kR && t < nt && n0 + r < a.N) qd_store(a, t, n0 + r, mine, __ldcg(a.xs + t), __ldg(a.ws + n0 + r));
  }
  if (tid == 0) trace_max(a.trace, kTrExit);
}

template <int kT, int kR, int kAhead>
cudaError_t launch_rows(const QdenseArgs &a, int n_sm, cudaStream_t st, bool pdl) {
  const size_t smem = (size_t)kT * a.K;
  int per_sm = 0;
  cudaError_t e =
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, qdense_rows_kernel<kT, kR, kAhead>, kQdThreads, smem);
  if (e != cudaSuccess) return e;
  if (per_sm < 1) return cudaErrorInvalidConfiguration;
  const int units = (a.N + kR - 1) / kR, blocks = (units + kQdWarps - 1) / kQdWarps;
  const int most = n_sm * per_sm;
  return launch_k(qdense_rows_kernel<kT, kR, kAhead>, dim3(blocks < most ? blocks : most), dim3(kQdThreads), smem, st,
                  pdl, a);
}

template <int kT>
cudaError_t launch_rows_t(const QdenseArgs &a, int n_sm, cudaStream_t st, bool pdl) {
  if (a.N >= 4 * kQdWarps * 4 * n_sm) return launch_rows<kT, 4, 3>(a, n_sm, st, pdl);
  return launch_rows<kT, 1, 6>(a, n_sm, st, pdl);
}

template <int kT>
cudaError_t set_rows_attr() {
  cudaError_t e = cudaFuncSetAttribute(qdense_rows_kernel<kT, 4, 3>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kT * kQdenseMaxK);
  if (e) return e;
  return cudaFuncSetAttribute(qdense_rows_kernel<kT, 1, 6>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kT * kQdenseMaxK);
}

// Four 8-bit codes as two exact fp16 pairs: the code + 128 goes under the
// exponent of 1024 (1024 + c is exact for c < 1024), then 1152 is subtracted.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi) {
  const uint32_t u = w ^ 0x80808080u;
  const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
}

// ------------------------------------------------------------------ few rows, mma.sync
constexpr int kQfWarps = 16;
constexpr int kQfThreads = kQfWarps * 32;
constexpr int kQfAhead = 4;          // 64-wide K blocks whose codes a warp has in flight
constexpr int kQfFlush = 1024 / 64;  // blocks after which the fp32 sums go to integers: 128 * 128 * 1024 = 2^24
constexpr size_t kQfSmemMax = 200 * 1024;
__host__ __device__ constexpr int qf_pitch(int K) { return 2 * K + 16; }  // bytes of a row: consecutive rows 4 banks apart

// Up to 8 rows (those past T: zero).  A warp takes a tile of 16 channels (or, where tiles
// are few, a part of a tile's K: split parts by neighbouring warps).  K comes
// in 64-wide blocks; lane (r, c) = (lane / 4, lane % 4) loads the codes 16 c
// .. 16 c + 15 of channels r and r + 8, and multiplication j of a block takes
// codes 4 j .. 4 j + 3 of those for the k positions that mma.m16n8k16 gives
// the lane; the rows, widened to fp16 in shared memory, follow the same order.
__global__ void __launch_bounds__(kQfThreads, 1) qdense_few_kernel(const QdenseArgs a, const int split) {
  extern __shared__ __align__(16) uint8_t fsm[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, c = lane & 3;
  const int K = a.K, nb = (K + 63) / 64, pitch = qf_pitch(K);
  const bool tracer = blockIdx.x == 0 && tid == 0;
  if (tracer) trace_min(a.trace, kTrEntry);
  pdl_wait();
  pdl_launch_dependents();
  if (tracer) trace_min(a.trace, kTrWaited);

  const int tiles = (a.N + 15) / 16, per_block = kQfWarps / split;
  const int part = warp % split;
  const int b0 = nb * part / split, b1 = nb * (part + 1) / split;  // this warp's blocks
  int tile = blockIdx.x * per_block + warp / split;
  int4 w0[kQfAhead], w1[kQfAhead];
  auto request = [&](int n0, int b) {
    const int8_t *p0 = a.w + (size_t)min(n0 + r, a.N - 1) * K + 16 * c;  // channels past N: discarded below
    const int8_t *p1 = a.w + (size_t)min(n0 + r + 8, a.N - 1) * K + 16 * c;
#pragma unroll
    for (int j = 0; j < kQfAhead; ++j) {
      const bool there = b + j < b1 && 64 * (b + j) + 16 * c < K;
      w0[j] = there ? qd_stream(p0 + 64 * (b + j)) : make_int4(0, 0, 0, 0);
      w1[j] = there ? qd_stream(p1 + 64 * (b + j)) : make_int4(0, 0, 0, 0);
    }
  };
  if (tile < tiles) request(tile * 16, b0);
  // the rows, widened (those past T: zero)
  const int nck = K / 16;
  for (int i = tid; i < 8 * nck; i += kQfThreads) {
    const int t = i / nck, k = i - t * nck;
    const uint4 v = t < a.T ? __ldcg(reinterpret_cast<const uint4 *>(a.x + (size_t)t * K) + k) : make_uint4(0u, 0u, 0u, 0u);
    uint4 o0, o1;
    widen4(v.x, o0.x, o0.y);
    widen4(v.y, o0.z, o0.w);
    widen4(v.z, o1.x, o1.y);
    widen4(v.w, o1.z, o1.w);
    uint4 *dst = reinterpret_cast<uint4 *>(fsm + (size_t)t * pitch + 32 * k);
    dst[0] = o0;
    dst[1] = o1;
  }
  __syncthreads();
  int *parts = reinterpret_cast<int *>(fsm + (size_t)8 * pitch);  // [warp][4][32], split > 1
  // (every warp of a block makes the same number of rounds: barriers below)
  const int rounds = (tiles + gridDim.x * per_block - 1) / (gridDim.x * per_block);
  for (int round = 0; round < rounds; ++round, tile += gridDim.x * per_block) {
    const int n0 = tile * 16;
    int sum[4] = {0, 0, 0, 0};
    if (tile < tiles) {
      if (round > 0) request(n0, b0);
      for (int f = b0; f < b1; f += kQfFlush) {  // exact in fp32
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        const int fe = min(b1, f + kQfFlush);
        for (int b = f; b < fe; b += kQfAhead) {
          int4 x0[kQfAhead], x1[kQfAhead];
#pragma unroll
          for (int j = 0; j < kQfAhead; ++j) {
            x0[j] = w0[j];
            x1[j] = w1[j];
          }
          request(n0, b + kQfAhead);
          __syncwarp();  // (mma.sync wants the warp together, and the loads depend on the lane)
#pragma unroll
          for (int j = 0; j < kQfAhead; ++j) {
            if (b + j >= fe) break;  // (warp-uniform)
            const int k = min(64 * (b + j) + 16 * c, K - 16);  // past the row: the weights are zero
            const uint32_t *q0 = reinterpret_cast<const uint32_t *>(&x0[j]), *q1 = reinterpret_cast<const uint32_t *>(&x1[j]);
            uint32_t A[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              widen4(q0[i], A[i][0], A[i][2]);
              widen4(q1[i], A[i][1], A[i][3]);
            }
            const uint4 *bx = reinterpret_cast<const uint4 *>(fsm + (size_t)r * pitch + 2 * k);
            const uint4 v0 = bx[0], v1 = bx[1];
            mma_f16(acc, A[0], v0.x, v0.y);
            mma_f16(acc, A[1], v0.z, v0.w);
            mma_f16(acc, A[2], v1.x, v1.y);
            mma_f16(acc, A[3], v1.z, v1.w);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] += __float2int_rn(acc[i]);
      }
    }
    if (split > 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) parts[(warp * 4 + i) * 32 + lane] = sum[i];
      __syncthreads();
      if (part == 0) {
        for (int p = 1; p < split; ++p)
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[i] += parts[((warp + p) * 4 + i) * 32 + lane];
      }
      __syncthreads();
    }
    if (part == 0 && tile < tiles) {
      // sum[i]: channel n0 + r + 8 (i / 2), row 2 c + i % 2
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ch = n0 + r + 8 * (i >> 1);
        const int t = 2 * c + (i & 1);
        if (t < a.T && ch < a.N) qd_store(a, t, ch, sum[i], __ldcg(a.xs + t), __ldg(a.ws + ch));
      }
    }
  }
  if (tid == 0) trace_max(a.trace, kTrExit);
}

size_t few_smem(int K) { return (size_t)8 * qf_pitch(K) + (size_t)kQfWarps * 4 * 32 * 4; }

// Whether the rows, widened, fit a block's shared memory.
bool few_fits(int T, int K) { return T <= kQdRowsMax && few_smem(K) <= kQfSmemMax; }

cudaError_t launch_few(const QdenseArgs &a, int n_sm, cudaStream_t st, bool pdl) {
  const int tiles = (a.N + 15) / 16, nb = (a.K + 63) / 64;
  // parts of K per tile while whole tiles would leave warps without work
  int split = 1;
  while (split < kQfWarps && 2 * split * tiles <= n_sm * kQfWarps && 2 * split <= nb) split *= 2;
  const int per_block = kQfWarps / split, blocks = (tiles + per_block - 1) / per_block;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks < n_sm ? blocks : n_sm);
  cfg.blockDim = dim3(kQfThreads);
  cfg.dynamicSmemBytes = few_smem(a.K);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, qdense_few_kernel, a, split);
}

// ------------------------------------------------------------------ rows to fp16
constexpr int kWidenThreads = 256;
constexpr int kWidenAhead = 2;  // loads of a thread in flight

// (16 bytes per thread and store, whole lines per warp: from 16 codes per
// thread, in two stores, 4096 x 2816 took 1.5 us longer)
__global__ void __launch_bounds__(kWidenThreads) qdense_widen_kernel(const QdenseArgs a) {
  if (blockIdx.x == 0 && threadIdx.x == 0) trace_min(a.trace, kTrEntry);
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) trace_min(a.trace, kTrWaited);
  const size_t n = (size_t)a.T * (a.K / 8);
  const uint2 *src = reinterpret_cast<const uint2 *>(a.x);
  uint4 *dst = reinterpret_cast<uint4 *>(a.work);
  const size_t step = (size_t)gridDim.x * kWidenThreads;
  for (size_t i = (size_t)blockIdx.x * kWidenThreads + threadIdx.x; i < n; i += kWidenAhead * step) {
    uint2 v[kWidenAhead];
#pragma unroll
    for (int j = 0; j < kWidenAhead; ++j)
      if (i + j * step < n) v[j] = __ldcs(src + i + j * step);
#pragma unroll
    for (int j = 0; j < kWidenAhead; ++j) {
      if (i + j * step >= n) break;
      uint4 o;
      widen4(v[j].x, o.x, o.y);
      widen4(v[j].y, o.z, o.w);
      dst[i + j * step] = o;
    }
  }
  if (threadIdx.x == 0) trace_max(a.trace, kTrExit);
}

// ------------------------------------------------------------------ tensor cores
constexpr int kMmM = 128;                  // channels per tile
constexpr int kMmWiden = 8;                // widen warps
constexpr int kMmFin0 = kMmWiden;
constexpr int kMmFin = 8;                  // finish warps
constexpr int kMmWts = kMmFin0 + kMmFin;   // weights warp
constexpr int kMmRows = kMmWts + 1;        // rows warp
constexpr int kMmMma = kMmRows + 1;        // MMA warp
constexpr int kMmThreads = (kMmMma + 1) * 32;
constexpr int kMmK = 128;                  // K of a stage
constexpr int kMmABufs = 4;                // A tiles in tensor memory (64 columns: 128 x 128 fp16)
constexpr uint32_t kMmACol = 256;          // first column of the A tiles; the sums lie below
constexpr int kMmWStage = kMmM * kMmK;     // bytes of a weight stage
constexpr int kMmMaxN = 256;
constexpr int kMmSplitN = 128;             // rows per tile, at most, where blocks have one tile or a part of one
constexpr int kMmMaxSplit = kQdenseMaxCluster;
constexpr int kMmWst = 6;                  // weight stages, at least
static_assert(kMmWst * kMmWStage >= kMmSplitN * kMmM * 4, "a block's part of the sums lies over them");
constexpr int kMmBarBytes = 512;
// Waits for the other warps' last words, at most, where a wait ran out (a warp
// leaves its loop once one of its own, of a stage's two or three, has run out).
constexpr int kMmLastWaits = 4;
constexpr int kMmSmemMax = 227 * 1024;
constexpr int kMmXsBytes = kMmMaxN * 4;

// kOne: tiles of up to 128 rows or parts of them; the rows widened by a launch
// before.  kPair: wider tiles, whole, a pair of blocks on each.  kFew: as kOne, one
// tile or part of a tile per block; the rows come as 8-bit codes, and the finish
// warps, idle until the sums are there, widen them.
enum { kOne, kPair, kFew };

struct MmPlan {
  int n;            // rows per tile (the MMA N): a multiple of 16
  int wst, rst;     // stages of weights and of rows, 128 of K each
  int xst;          // kFew: stages of the rows' codes
  int dbufs;        // sets of sums in tensor memory
  int split;        // blocks of a cluster that share a tile along K
  int ntile, ttile; // tiles of channels, of rows
  int whole, units; // units of work: `whole` tiles, then halves of tiles (by rows)
  int form;
  int nload;        // rows that a block loads of a tile: n, or n / 2 in pairs
  int smem;
};

struct MmParams {
  CUtensorMap w;     // 8-bit codes {K, N}, box {128, 128}, 128-byte swizzle
  CUtensorMap x[2];  // fp16 rows {K, T}, box {64, nload} and {64, nload / 2}, 128-byte swizzle; kFew: codes, box {128, n}
  QdenseArgs a;
  MmPlan p;
};

// A unit's place: first channel, first row, rows (the MMA N) and how many of
// them there are.
struct MmUnit {
  int n0, t0, n, cnt, half;
};
template <int kForm>
__device__ __forceinline__ MmUnit mm_unit(const MmPlan &p, int T, int u, int rank) {
  MmUnit q;
  q.half = u >= p.whole ? 1 : 0;
  const int tile = q.half ? p.whole + (u - p.whole) / 2 : u;
  q.n = q.half ? p.n / 2 : p.n;
  q.n0 = (kForm == kPair ? tile / p.ttile * 2 + rank : tile / p.ttile) * kMmM;
  q.t0 = tile % p.ttile * p.n + (q.half ? ((u - p.whole) & 1) * q.n : 0);
  q.cnt = min(q.n, T - q.t0);  // none: a half past the last row, which every warp passes over
  return q;
}

// Bounded wait that suspends in hardware; the timer is read only once a wait
// is not over at its first look (reading it costs more than most waits).
// What it orders, by who arrives: kBlock threads and copies of this block;
// kClusterAcquire copies of the pair's other block too; kClusterRelaxed the
// tensor cores or threads of the other block, for accesses of tensor memory (the
// tcgen05 fences on either side order those) and for places that are free again.
enum { kBlock, kClusterAcquire, kClusterRelaxed };
template <int kOrder>
__device__ __forceinline__ bool mm_try(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  if (kOrder == kClusterAcquire)
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, "
        "0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity), "r"(1000000u)
        : "memory");
  else if (kOrder == kClusterRelaxed)
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, "
        "0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity), "r"(1000000u)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity), "r"(1000000u)
        : "memory");
  return ok != 0;
}
template <int kOrder = kBlock>
__device__ __forceinline__ bool mm_wait(uint64_t *bar, uint32_t parity) {
  if (mm_try<kOrder>(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
  for (;;) {
    if (mm_try<kOrder>(bar, parity)) return true;
    if (global_ns() - t0 > kWaitLimitNs) return false;
  }
}
// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred P;\n elect.sync _|P, 0xffffffff;\n selp.u32 %0, 1, 0, P;\n}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void mm_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// D (tensor memory) += A (tensor memory, 128 x 16) * B (shared memory, n x 16)^T;
// kPair: A is 256 x 16 and B n x 16, a half of each in either block's memory.
template <int kForm>
__device__ __forceinline__ void mm_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if (kForm == kPair)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(
            d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(
            d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// Arrives on `bar` (kPair: in both blocks) once the MMAs issued before are complete.
template <int kForm>
__device__ __forceinline__ void mm_commit(uint64_t *bar) {
  if (kForm == kPair)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"((uint16_t)3)
        : "memory");
  else
    dense::tc_commit(bar);
}
// The instructions below with .aligned (and bar.sync) have to be executed by a
// warp's lanes together.  Lanes come apart wherever a branch depends on the lane
// (one lane's arrival, channels past the last), and what brings them together for
// certain is a warp barrier alone: each of these functions begins with one.
template <int kForm>
__device__ __forceinline__ void mm_alloc(uint32_t *dst) {
  __syncwarp();
  if (kForm == kPair) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    dense::tc_alloc(dst, 512);
  }
}
template <int kForm>
__device__ __forceinline__ void mm_dealloc(uint32_t tmem) {
  __syncwarp();
  if (kForm == kPair)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  else
    dense::tc_dealloc(tmem, 512);
}

// 32 registers of each lane to 32 tensor-memory columns of the warp's lanes
// (complete after mm_st_wait).
__device__ __forceinline__ void mm_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  __syncwarp();
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void mm_st_wait() {
  __syncwarp();
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// 32 tensor-memory columns of the warp's lanes.
__device__ __forceinline__ void mm_ld32(uint32_t taddr, float (&v)[32]) {
  __syncwarp();
  dense::tc_ld32(taddr, v);
}
// Barrier of the finish warps.
__device__ __forceinline__ void mm_fin_sync() {
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(kMmFin * 32) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of this block's shared memory `addr` in block `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
  return at;
}
// An arrival on a barrier of another block of the cluster.  No thread of a pair
// reads memory that a thread of the other block writes: what the arrivals pass on
// are A tiles and sums in tensor memory, ordered by the tcgen05 fences before the
// arrival and after the wait, so the arrival itself need not order anything (a
// release at cluster scope, which waits for the warp's own stores too, nearly
// doubles the time: 128 x 65536 x 2816 78 us against 42).
__device__ __forceinline__ void cluster_arrive(uint32_t addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// A block's rows of a pair's tile; their bytes count on the barrier at `bar`, which
// may be the other block's.  A copy's completion is a release at cluster scope.
__device__ __forceinline__ void mm_load_pair(void *dst, const CUtensorMap *map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ float4 cluster_ld4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// Rows of a shared tile that one block of the cluster adds up.
__host__ __device__ inline int mm_quota(const MmPlan &p) { return (p.n + p.split - 1) / p.split; }

template <int kForm>
__global__ void __launch_bounds__(kMmThreads, 1) qdense_mma_kernel(const __grid_constant__ MmParams prm) {
  extern __shared__ __align__(1024) uint8_t msm[];
  const QdenseArgs &a = prm.a;
  const MmPlan &P = prm.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t *base = msm + ((1024u - (smem_addr(msm) & 1023u)) & 1023u);
  const int rstep = P.nload * 128, rstage = 2 * rstep;  // a rows stage: two steps of 64 of K
  uint8_t *wbuf = base, *rbuf = base + P.wst * kMmWStage, *xbuf = rbuf + P.rst * rstage;
  const int xstage = P.n * 128;  // kFew
  uint64_t *bar = reinterpret_cast<uint64_t *>(xbuf + P.xst * xstage);
  uint64_t *wfull = bar, *wempty = wfull + P.wst, *rfull = wempty + P.wst, *rempty = rfull + P.rst;
  uint64_t *afull = rempty + P.rst, *aempty = afull + kMmABufs, *dfull = aempty + kMmABufs, *dempty = dfull + 2;
  uint64_t *tready = dempty + 2, *tdone = tready + 1, *xfull = tdone + 1, *xempty = xfull + P.xst;
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(xempty + P.xst);
  float *s_xs = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(bar) + kMmBarBytes);  // [n] row scales
  float *s_part = reinterpret_cast<float *>(base);  // [n][128] this block's part of the sums, over the stages
  constexpr bool kPairs = kForm == kPair, kOwn = kForm == kFew;
  constexpr int kTc = kPairs ? kClusterRelaxed : kBlock;  // waits on barriers that pass on tensor memory, or the MMAs' words
  const bool tracer = blockIdx.x == 0 && tid == 0;
  const int split = kPairs ? 1 : P.split;
  const int rank = kPairs || split > 1 ? (int)cluster_rank() : 0;
  const int part = kPairs ? 0 : rank;  // this block's part of K
  const bool leader = !kPairs || rank == 0;

  if (tid < 2 * P.wst + 2 * P.rst + 2 * P.xst + 2 * kMmABufs + 6) {
    // arrivals per phase.  The leader of a pair hears of both blocks' A tiles, rows
    // (one arrival, for the bytes of both) and finish warps.
    uint64_t *b = bar + tid;
    int n = 1;
    if ((b >= wempty && b < rfull) || (b >= afull && b < aempty)) n = kMmWiden / 2;
    if (b >= dempty && b < tready) n = kMmFin;
    if (b == tdone) n = kMmWiden + kMmFin;
    if (b >= xempty || (kOwn && b >= rfull && b < rempty)) n = kMmFin / 2;
    if (kPairs && leader && ((b >= afull && b < aempty) || (b >= dempty && b < tready)))
      n *= 2;
    mbar_init(b, n);
    fence_mbar_init();
  }
  __syncthreads();
  if (tracer) trace_min(a.trace, kTrEntry);
  if (!kOwn) pdl_launch_dependents();  // (the launch before has waited for those before it)

  if (kPairs) cluster_sync_all();  // the other block runs, its barriers are set
  const int csize = kPairs ? 2 : split;
  const int first = blockIdx.x / csize, stride = gridDim.x / csize;  // units of this block
  const int units = P.units;
  const int nst = (a.K + kMmK - 1) / kMmK, st0 = nst * part / split, st1 = nst * (part + 1) / split;  // its part of K
  const int g0 = 2 * st0, g1 = min(2 * st1, (a.K + 63) / 64);  // the same in steps of 64

  if (warp == kMmWts) {
    // ============================================================ weights
    // Nothing that an earlier launch still writes is read here: the launch
    // before this one (the widening of the rows) waited for those, or this does.
    if (kOwn) {
      pdl_wait();
      pdl_launch_dependents();
    }
    if (lane == 0) {
      fused::fence_proxy_async_global();
      bool ok = true;
      int st = 0, ph = 0, issued = 0;
      for (int u = first; u < units && ok; u += stride) {
        const MmUnit q = mm_unit<kForm>(P, a.T, u, rank);
        if (q.cnt <= 0) continue;
        for (int s = st0; s < st1; ++s, ++issued) {
          if (issued >= P.wst && !(ok = mm_wait(&wempty[st], ph ^ 1))) break;
          mbar_arrive_expect_tx(&wfull[st], kMmWStage);
          dense::tma_load_2d(wbuf + st * kMmWStage, &prm.w, kMmK * s, q.n0, &wfull[st]);
          if (++st == P.wst) {
            st = 0;
            ph ^= 1;
          }
        }
      }
      if (!ok) set_error(a.err, kErrTimeout);
      // copies in flight land before the block's shared memory is released
      for (int j = max(0, issued - P.wst); j < issued; ++j) mm_wait(&wfull[j % P.wst], (j / P.wst) & 1);
    }
  } else if (warp == kMmRows) {
    // ============================================================ rows
    pdl_wait();  // the widened rows
    if (lane == 0) {
      if (blockIdx.x == 0) trace_min(a.trace, kTrWaited);
      fused::fence_proxy_async_global();
      bool ok = true;
      int st = 0, ph = 0, issued = 0;
      if (kOwn) {
        const MmUnit q = mm_unit<kForm>(P, a.T, first, rank);
        for (int s = st0; s < st1; ++s, ++issued) {
          if (issued >= P.xst && !(ok = mm_wait(&xempty[st], ph ^ 1))) break;
          mbar_arrive_expect_tx(&xfull[st], (uint32_t)xstage);
          dense::tma_load_2d(xbuf + st * xstage, &prm.x[0], kMmK * s, q.t0, &xfull[st]);
          if (++st == P.xst) {
            st = 0;
            ph ^= 1;
          }
        }
        for (int j = max(0, issued - P.xst); j < issued; ++j) mm_wait(&xfull[j % P.xst], (j / P.xst) & 1);
      }
      for (int u = first; !kOwn && u < units && ok; u += stride) {
        const MmUnit q = mm_unit<kForm>(P, a.T, u, rank);
        if (q.cnt <= 0) continue;
        const int rows = kPairs ? q.n / 2 : q.n, t0 = q.t0 + (kPairs ? rank * rows : 0);
        for (int g = g0; g < g1; g += 2, ++issued) {
          if (issued >= P.rst && !(ok = mm_wait<kTc>(&rempty[st], ph ^ 1))) break;
          const int h = min(2, g1 - g);
          if (leader) mbar_arrive_expect_tx(&rfull[st], (uint32_t)((kPairs ? 2 : 1) * h * rows * 128));
          for (int i = 0; i < h; ++i) {
            if (kPairs)  // (rempty is passed, so the MMAs have used the place's last rows and the leader's rfull is in this phase)
              mm_load_pair(rbuf + st * rstage + i * rstep, &prm.x[q.half], 64 * (g + i), t0,
                           cluster_map(smem_addr(&rfull[st]), 0));
            else
              dense::tma_load_2d(rbuf + st * rstage + i * rstep, &prm.x[q.half], 64 * (g + i), t0, &rfull[st]);
          }
          if (++st == P.rst) {
            st = 0;
            ph ^= 1;
          }
        }
      }
      if (!ok) set_error(a.err, kErrTimeout);
      for (int j = max(0, issued - P.rst); !kOwn && j < issued; ++j) {
        if (leader)
          mm_wait<kPairs ? kClusterAcquire : kBlock>(&rfull[j % P.rst], (j / P.rst) & 1);
        else  // its copies count on the leader's barrier: they have landed once the MMAs have read them
          mm_wait<kTc>(&rempty[j % P.rst], (j / P.rst) & 1);
      }
    }
  } else if (warp == kMmMma) {
    // ============================================================ MMA
    mm_alloc<kForm>(s_tmem);
    dense::tc_fence_before();
    __syncwarp();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(s_tmem);
    // The whole warp runs the loop and one lane issues: with the loop in one
    // lane's branch the descriptors have to be moved to uniform registers for
    // every MMA, and an MMA of few rows takes three times as long (24 x 262144
    // x 2816: 186 us against 129).
    if (lane == 0) mm_arrive(tready);
    const uint64_t bdesc0 = dense::sdesc(smem_addr(rbuf), 16, 1024, 2);
    bool ok = true;
    int gi = 0, du = 0, st = 0, ph = 0, ab = 0, aph = 0;
    for (int u = first; leader && u < units; u += stride) {
      const MmUnit q = mm_unit<kForm>(P, a.T, u, rank);
      if (q.cnt <= 0) continue;
      const uint32_t idesc = dense::idesc_f16(kPairs ? 2 * kMmM : kMmM, q.n);
      const int db = du % P.dbufs;
      if (du >= P.dbufs) ok = __all_sync(0xffffffffu, mm_wait<kTc>(&dempty[db], ((du / P.dbufs) - 1) & 1));
      if (!ok) break;
      ++du;
      const uint32_t acc = tmem + db * 128;
      for (int s = st0; s < st1; ++s, ++gi) {
        ok = __all_sync(0xffffffffu, mm_wait<kPairs ? kClusterAcquire : kBlock>(&rfull[st], ph) && mm_wait<kTc>(&afull[ab], aph));
        if (!ok) break;
        dense::tc_fence_after();
        const uint32_t ad = tmem + kMmACol + 64 * ab;
        uint64_t bd = bdesc0 + (uint64_t)((st * rstage) >> 4);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)  // K = 16 per MMA: 8 columns of A, 32 bytes of B's rows
          if (elect_one()) mm_mma<kForm>(acc, ad + 8 * ks, bd + 2 * ks, idesc, (s > st0 || ks > 0) ? 1u : 0u);
        if (2 * s + 1 < g1) {  // the stage's second half
          bd += (uint64_t)(rstep >> 4);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            if (elect_one()) mm_mma<kForm>(acc, ad + 32 + 8 * ks, bd + 2 * ks, idesc, 1u);
        }
        if (elect_one()) {
          mm_commit<kForm>(&rempty[st]);
          mm_commit<kForm>(&aempty[ab]);
          if (s == st1 - 1) mm_commit<kForm>(&dfull[db]);
        }
        __syncwarp();
        if (++st == P.rst) {
          st = 0;
          ph ^= 1;
        }
        if (++ab == kMmABufs) {
          ab = 0;
          aph ^= 1;
        }
      }
      if (!ok) break;
    }
    if (!ok && lane == 0) set_error(a.err, kErrTimeout);
    // The last MMAs are complete and the sums read before the tensor memory goes
    // back (bounded waits): every A tile was used and every set of sums handed back,
    // so no warp uses it any more.  Where one of the waits ran out the other warps
    // may still do so, and their last words are waited for.
    if (gi > 0) ok = mm_wait<kTc>(&aempty[(gi - 1) % kMmABufs], ((gi - 1) / kMmABufs) & 1) && ok;
    if (leader && du > 0) ok = mm_wait<kTc>(&dempty[(du - 1) % P.dbufs], ((du - 1) / P.dbufs) & 1) && ok;
    if (!kPairs) {
      if (!__all_sync(0xffffffffu, ok))
        for (int i = 0; i < kMmLastWaits && !__all_sync(0xffffffffu, mm_wait(tdone, 0)); ++i) {
        }
      dense::tc_fence_after();
      mm_dealloc<kForm>(tmem);
    }
  } else if (warp >= kMmFin0) {
    // ============================================================ finish
    // Warp w reads tensor-memory lanes 32 (w % 4) .. +31: channels n0 + rr; the
    // two warps of a lane quarter take turns at pieces of 32 columns.  A
    // register per lane and column: 32 neighbouring channels of one row are one
    // store instruction.
    bool ok = __all_sync(0xffffffffu, mm_wait(tready, 0));
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(s_tmem);
    const int rr = 32 * (warp & 3) + lane, ft = tid - kMmFin0 * 32, side = (warp - kMmFin0) >> 2;
    if (kOwn) {
      // First the rows of this block's stages, taken in turn by the two halves
      // of the warps.  (The rings' lengths are even, so each barrier belongs to
      // one half: a waiter that meets a barrier at every second phase only would
      // take the phase before last for the last.)  Eight lanes to a row, 16 codes each: 16-byte chunk j of a
      // row of codes (swizzled as the copy left it) becomes chunks 2 j, 2 j + 1
      // of the row's 256 bytes in two steps of 64; lanes 4 to 7 of the eight
      // store theirs in the other order, for 32 different banks.
      pdl_wait();
      const int j = lane & 7, r0 = 4 * (warp & 3) + (lane >> 3), c = 2 * (j & 3), odd = j >> 2;
      for (int i = side; i < st1 - st0 && ok; i += kMmFin / 4) {
        const int st = i % P.rst, xs = i % P.xst;
        ok = mm_wait(&xfull[xs], (i / P.xst) & 1);
        if (i >= P.rst) ok = ok && mm_wait(&rempty[st], ((i / P.rst) - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint8_t *const from = xbuf + xs * xstage;
        uint8_t *const to = rbuf + st * rstage + odd * rstep;
        uint4 v[kMmSplitN / 16];
#pragma unroll
        for (int k = 0; k < kMmSplitN / 16; ++k) {
          const int r = r0 + 16 * k;
          if (16 * k < P.n) v[k] = *reinterpret_cast<const uint4 *>(from + r * 128 + ((j ^ (r & 7)) << 4));
        }
#pragma unroll
        for (int k = 0; k < kMmSplitN / 16; ++k) {
          if (16 * k >= P.n) break;
          const int r = r0 + 16 * k;
          uint4 o[2];
          widen4(v[k].x, o[0].x, o[0].y);
          widen4(v[k].y, o[0].z, o[0].w);
          widen4(v[k].z, o[1].x, o[1].y);
          widen4(v[k].w, o[1].z, o[1].w);
          *reinterpret_cast<uint4 *>(to + r * 128 + (((c + odd) ^ (r & 7)) << 4)) = odd ? o[1] : o[0];
          *reinterpret_cast<uint4 *>(to + r * 128 + (((c + 1 - odd) ^ (r & 7)) << 4)) = odd ? o[0] : o[1];
        }
        dense::fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mm_arrive(&xempty[xs]);
          mm_arrive(&rfull[st]);
        }
      }
    }
    int du = 0;
    for (int u = first; u < units; u += stride) {
      const MmUnit q = mm_unit<kForm>(P, a.T, u, rank);
      if (q.cnt <= 0) continue;
      const int n = q.n0 + rr, t0 = q.t0, cnt = q.cnt;
      const int db = du % P.dbufs;
      float ws = 0.f;
      if (split == 1) {  // the tile's row scales to shared memory while its sums are made
        mm_fin_sync();  // every finish warp is done with the tile before
        for (int i = ft; i < q.n; i += kMmFin * 32) s_xs[i] = i < cnt ? __ldcg(a.xs + t0 + i) : 0.f;
        ws = n < a.N ? __ldg(a.ws + n) : 0.f;
        mm_fin_sync();
      }
      ok = __all_sync(0xffffffffu, ok && mm_wait<kTc>(&dfull[db], (du / P.dbufs) & 1));
      dense::tc_fence_after();
      const uint32_t ta = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + db * 128;
      if (split > 1) {
        // its part to shared memory, over the stages: their last MMA is complete
        for (int c0 = 32 * side; ok && c0 < cnt; c0 += 8 * kMmFin) {
          float v[32];
          mm_ld32(ta + c0, v);
          const int m = min(32, cnt - c0);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j < m) s_part[(c0 + j) * kMmM + rr] = v[j];
        }
      } else {
        for (int c0 = 32 * side; ok && c0 < cnt; c0 += 8 * kMmFin) {
          float v[32];
          mm_ld32(ta + c0, v);  // (columns past the tile's: not used)
          const int m = min(32, cnt - c0);
          if (n < a.N) {
            const size_t o = (size_t)(t0 + c0) * a.N + n;
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 xs = *reinterpret_cast<const float4 *>(s_xs + c0 + j);
              v[j] = __fmul_rn(__fmul_rn(v[j], xs.x), ws);
              v[j + 1] = __fmul_rn(__fmul_rn(v[j + 1], xs.y), ws);
              v[j + 2] = __fmul_rn(__fmul_rn(v[j + 2], xs.z), ws);
              v[j + 3] = __fmul_rn(__fmul_rn(v[j + 3], xs.w), ws);
            }
            if (a.softcap > 0.f) {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = a.softcap * tanhf(v[j] / a.softcap);
            }
            if (a.y32) {
              float *p = a.y32 + o;
#pragma unroll
              for (int j = 0; j < 32; ++j, p += a.N)
                if (j < m) *p = v[j];
            }
            if (a.y) {
              uint16_t *p = a.y + o;
#pragma unroll
              for (int j = 0; j < 32; ++j, p += a.N)
                if (j < m) *p = float_to_bf16_bits(v[j]);
            }
          }
        }
      }
      dense::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader)
          mm_arrive(&dempty[db]);
        else
          cluster_arrive(cluster_map(smem_addr(&dempty[db]), 0));
      }
      ++du;
    }
    if (!ok && lane == 0) set_error(a.err, kErrTimeout);
    if (!kPairs && lane == 0) mm_arrive(tdone);
  } else {
    // ============================================================ widen
    // Two halves of the warps take turns at the stages, so that one's waits and
    // loads pass while the other converts.  (The rings of weights and A tiles have
    // even lengths: each barrier belongs to one half.)  Thread: channel rr of the
    // tile, a stage's 128 codes in two pieces of 64.  Its 16-byte chunk j lies at
    // j ^ (rr % 8) of the row (128-byte swizzle).
    const int grp = warp >> 2, rr = 32 * (warp & 3) + lane, sw = rr & 7;
    bool ok = __all_sync(0xffffffffu, mm_wait(tready, 0));
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(s_tmem) + ((uint32_t)(32 * (warp & 3)) << 16) + kMmACol;
    int st = grp, ph = 0, gi = 0;
    for (int u = first; u < units && ok; u += stride) {
      if (mm_unit<kForm>(P, a.T, u, rank).cnt <= 0) continue;
      for (int s = st0; s < st1 && ok; ++s, ++gi) {
        if ((gi & 1) != grp) continue;
        const int ab = gi % kMmABufs;
        ok = mm_wait(&wfull[st], ph);
        const uint8_t *row = wbuf + st * kMmWStage + rr * 128;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint4 c[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) c[j] = *reinterpret_cast<const uint4 *>(row + (((4 * h + j) ^ sw) << 4));
          uint32_t o[32];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            widen4(c[j].x, o[8 * j], o[8 * j + 1]);
            widen4(c[j].y, o[8 * j + 2], o[8 * j + 3]);
            widen4(c[j].z, o[8 * j + 4], o[8 * j + 5]);
            widen4(c[j].w, o[8 * j + 6], o[8 * j + 7]);
          }
          if (h == 0) {
            if (gi >= kMmABufs) ok = ok && mm_wait<kTc>(&aempty[ab], ((gi / kMmABufs) - 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            dense::tc_fence_after();
          } else {
            __syncwarp();
            if (lane == 0) mm_arrive(&wempty[st]);
          }
          mm_st32(tmem + 64 * ab + 32 * h, o);
        }
        if (!ok) break;
        mm_st_wait();
        dense::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (leader)
            mm_arrive(&afull[ab]);
          else
            cluster_arrive(cluster_map(smem_addr(&afull[ab]), 0));
        }
        st += 2;
        if (st >= P.wst) {
          st -= P.wst;
          ph ^= 1;
        }
      }
    }
    if (!ok && lane == 0) set_error(a.err, kErrTimeout);
    if (!kPairs && lane == 0) mm_arrive(tdone);
  }

  if (kPairs) {
    // neither block leaves, or frees its tensor memory, while the other may
    // still arrive on its barriers or the leader's MMAs use it
    __syncwarp();
    dense::tc_fence_before();
    cluster_sync_all();
    dense::tc_fence_after();
    if (warp == kMmMma) mm_dealloc<kForm>(*reinterpret_cast<volatile uint32_t *>(s_tmem));
  }
  if (!kPairs && split > 1) {
    // One tile per cluster; this block adds the parts of its rows, a warp to a
    // row, four channels per lane, read from the other blocks' shared memory, 16
    // bytes a lane.  (Single floats pushed by the blocks that have them: 128 x
    // 2816 x 4096 11.4 us against 10.4, 128 x 704 x 2816 7.6 against 8.1.)
    __syncwarp();
    if (kOwn) pdl_wait();
    const MmUnit q = mm_unit<kForm>(P, a.T, first, rank);
    const int n0 = q.n0 + 4 * lane, t0 = q.t0, cnt = q.cnt;
    const int quota = mm_quota(P), r0 = part * quota, mine = min(quota, cnt - r0);
    float ws[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) ws[i] = n0 + i < a.N ? __ldg(a.ws + n0 + i) : 0.f;
    const float xl = lane < mine ? __ldcg(a.xs + t0 + r0 + lane) : 0.f;  // scales of rows lane, lane + 32
    const float xh = lane + 32 < mine ? __ldcg(a.xs + t0 + r0 + lane + 32) : 0.f;
    const bool quad = a.N % 4 == 0 && ((reinterpret_cast<uintptr_t>(a.y32) & 15) | (reinterpret_cast<uintptr_t>(a.y) & 7)) == 0;
    __syncwarp();
    cluster_sync_all();
    uint32_t from[kMmMaxSplit];
#pragma unroll
    for (int r = 0; r < kMmMaxSplit; ++r)
      from[r] = r < split ? cluster_map(smem_addr(s_part + (size_t)r0 * kMmM + 4 * lane), r) : 0u;
    for (int c = warp; c < mine; c += kMmThreads / 32) {
      const float xs = __shfl_sync(0xffffffffu, c < 32 ? xl : xh, c & 31);
      float4 v[kMmMaxSplit];
#pragma unroll
      for (int r = 0; r < kMmMaxSplit; ++r)
        if (r < split) v[r] = cluster_ld4(from[r] + (uint32_t)(c * kMmM) * 4u);
      float z[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int r = 1; r < kMmMaxSplit; ++r) {  // in rank order
        if (r >= split) break;
        z[0] += v[r].x;
        z[1] += v[r].y;
        z[2] += v[r].z;
        z[3] += v[r].w;
      }
      const int t = t0 + r0 + c;
      if (quad) {
        if (n0 < a.N) {
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] = qd_value(a, z[i], xs, ws[i]);
          const size_t o = (size_t)t * a.N + n0;
          if (a.y32) *reinterpret_cast<float4 *>(a.y32 + o) = make_float4(z[0], z[1], z[2], z[3]);
          if (a.y) {
            const uint32_t lo = float_to_bf16_bits(z[0]) | (uint32_t)float_to_bf16_bits(z[1]) << 16;
            const uint32_t hi = float_to_bf16_bits(z[2]) | (uint32_t)float_to_bf16_bits(z[3]) << 16;
            *reinterpret_cast<uint2 *>(a.y + o) = make_uint2(lo, hi);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n0 + i < a.N) qd_put(a, t, n0 + i, z[i], xs, ws[i]);
      }
    }
    cluster_sync_all();  // no block leaves while another reads its part
  }
  if (warp >= kMmFin0 && warp < kMmWts && lane == 0) trace_max(a.trace, kTrExit);  // the last warps at work
}

// Tiles of up to 256 rows where they fill the device, by pairs of blocks: a
// 128-wide K stage takes 0.45 us at 128 rows, 0.65 us at 256.
//
// Fewer of those than half the SMs: up to 128 rows per tile.  Where every block
// then has one tile or less, two choices by what they were measured to cost:
//   a cluster of s blocks per tile, each with a part of its stages, the parts
//   added up at 1.2 us + 7 ns per row of the tile + 6 ns per block (4 ns more per
//   row for clusters of over four; 0.6 us where there are several tiles of rows:
//   their norm's blocks leave a cluster's SMs late);
//   the rows widened by a launch before (1.45 us, then 0.35 us per stage) or by
//   the finish warps (0.37 us + 2 ns per row and stage).
// Measured, us, clusters of 1, 2, 3, 4, 6 (16 x 704 also 8):
//   16 x 704 x 2816    launch 11.2 8.8 7.8 7.3 6.6 6.3, finish warps 11.4 8.1 6.9 6.2 5.3 5.1
//   48 x 2816 x 2816   launch 11.5 9.5 8.4 7.8 7.4, finish warps 12.7 9.4 7.8 7.2 6.8
//   80 x 704 x 704     launch 6.3 7.2 7.0 7.1 6.7, finish warps 6.0 6.2 5.8 6.0 5.6
//   128 x 2816 x 4096  launch 16.1 12.7 11.3 10.4 10.4, finish warps 24.3 15.7 12.8 11.0 10.6
//   128 x 8192 x 1408  launch 8.8 9.3, finish warps 10.7 9.8
// clusters[s]: clusters of s blocks that the device holds at once (more than
// those would run in a second wave: 16 tiles in clusters of 8 took 15.7 us, in
// clusters of 4 10.4).
//
// Whole tiles of 48 rows and more go to pairs of blocks too, which halves what
// each takes of the rows (64 x 131072 x 2816 67.4 us by single blocks, 66.5 by
// pairs; 128 x 65536 x 2816 44.5, 41.6; 128 x 16384 x 16384 67.1, 60.4; 24 x
// 65536 x 2816 38.2, 38.5), unless they are soon done (48 x 65536 x 704, 6
// stages, 16.1, 16.4); of several tiles of rows from 112 (160 x 8192 x 2816,
// 80 each, 12.0, 12.7; 512 x 4096 x 8192 29.7, 27.2).
//
// The last round of tiles of more than 128 rows, if at most half the pairs have
// one: in halves.
MmPlan mm_plan(int T, int N, int K, int n_sm, const int *clusters) {
  MmPlan p;
  auto tiles = [&](int most) {
    p.ttile = (T + most - 1) / most;
    p.n = ((T + p.ttile - 1) / p.ttile + 15) / 16 * 16;
  };
  p.ntile = (N + kMmM - 1) / kMmM;
  p.split = 1;
  tiles(kMmMaxN);
  const int nst = (K + kMmK - 1) / kMmK;
  if (2 * p.ntile * p.ttile <= n_sm) tiles(kMmSplitN);
  p.form = p.n > kMmSplitN ? kPair : kOne;
  if (p.form == kOne && p.ntile * p.ttile <= n_sm) {
    const int count = p.ntile * p.ttile;
    double least = 0.0;
    for (int s = 1; s <= kMmMaxSplit && s <= nst; ++s) {
      if (s > 1 && count > clusters[s]) continue;
      const int stages = (nst + s - 1) / s;
      const double sum =
          s == 1 ? 0.0 : 1.2 + 0.007 * p.n + 0.006 * count * s + (s > 4 ? 0.004 * p.n : 0.0) + (p.ttile > 1 ? 0.6 : 0.0);
      const double one = 1.45 + 0.35 * stages, few = (0.37 + 0.002 * p.n) * stages;
      const double t = sum + (one < few ? one : few);
      if (s == 1 || t < least) {
        least = t;
        p.split = s;
        p.form = one < few ? kOne : kFew;
      }
    }
  }
  if (p.form == kOne && p.split == 1 && p.ntile > 1 && p.n >= (p.ttile == 1 ? 48 : 112) && nst * p.n >= 560)
    p.form = kPair;
  int room = n_sm;  // units at once
  if (p.form == kPair) {
    p.ntile = (p.ntile + 1) / 2;
    p.n = (p.n + 31) / 32 * 32;
    room = clusters[2];
  }
  p.whole = p.ntile * p.ttile;
  p.units = p.whole;
  const int rest = p.whole % room;
  if (p.n > 128 && p.whole > room && rest > 0 && 2 * rest <= room) {
    p.n = (p.n + 63) / 64 * 64;
    p.whole -= rest;
    p.units = p.whole + 2 * rest;
  }
  p.nload = p.form == kPair ? p.n / 2 : p.n;
  p.dbufs = p.n <= 128 ? 2 : 1;
  // Weight stages, an even number: whole tiles stream them from HBM (24 x 65536 x
  // 2816 with 6, 8, 10, 12: 39.0, 38.8, 39.5, 40.2 us; 24 x 262144 x 2816 124.3,
  // 124.3, 125.1, 125.0); the others need the room otherwise.
  p.wst = p.form != kFew && p.split == 1 && p.n <= 128 ? 8 : kMmWst;
  p.rst = p.form == kOne ? 3 : 4;
  p.xst = p.form == kFew ? 4 : 0;
  auto bytes = [&] {
    return p.wst * kMmWStage + p.rst * 2 * p.nload * 128 + p.xst * p.n * 128 + kMmBarBytes + kMmXsBytes + 1024;
  };
  if (bytes() > kMmSmemMax) p.rst = 2;  // (kFew, over 80 rows)
  p.smem = bytes();
  return p;
}

cudaError_t launch_mma(const QdenseArgs &a, int n_sm, const int *clusters, cudaStream_t st, bool pdl) {
  const EncodeTiledFn f = encode_tiled();
  if (!f) return cudaErrorNotSupported;
  MmParams prm;
  memset(&prm, 0, sizeof(prm));
  prm.a = a;
  const MmPlan &p = prm.p = mm_plan(a.T, a.N, a.K, n_sm, clusters);
  const cuuint64_t dw[2] = {(cuuint64_t)a.K, (cuuint64_t)a.N}, sw[1] = {(cuuint64_t)a.K};
  const cuuint64_t dx[2] = {(cuuint64_t)a.K, (cuuint64_t)a.T}, sx[1] = {(cuuint64_t)a.K * 2};
  const cuuint32_t bw[2] = {128, kMmM}, bx[2] = {64, (cuuint32_t)p.nload}, by[2] = {64, (cuuint32_t)p.nload / 2};
  const cuuint32_t bc[2] = {128, (cuuint32_t)p.n};
  constexpr CUtensorMapDataType k8 = CU_TENSOR_MAP_DATA_TYPE_UINT8, k16 = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  constexpr CUtensorMapSwizzle k128 = CU_TENSOR_MAP_SWIZZLE_128B;
  bool ok = encode_map(f, &prm.w, k8, 2, a.w, dw, sw, bw, k128);
  if (p.form == kFew)
    ok = ok && encode_map(f, &prm.x[0], k8, 2, a.x, dx, sw, bc, k128);
  else
    ok = ok && encode_map(f, &prm.x[0], k16, 2, a.work, dx, sx, bx, k128);
  if (p.units > p.whole) ok = ok && encode_map(f, &prm.x[1], k16, 2, a.work, dx, sx, by, k128);
  if (!ok) return cudaErrorInvalidValue;
  if (p.form != kFew) {
    const size_t pieces = (size_t)a.T * (a.K / 8), blocks = (pieces + kWidenThreads - 1) / kWidenThreads;
    const size_t most = (size_t)n_sm * 8;
    const cudaError_t e = launch_k(qdense_widen_kernel, dim3((unsigned)(blocks < most ? blocks : most)),
                                   dim3(kWidenThreads), 0, st, pdl, a);
    if (e != cudaSuccess) return e;
    if (prm.a.trace) prm.a.trace += 4;
  }
  const int units = p.units;
  cudaLaunchConfig_t cfg = {};
  const int room = p.form == kPair ? clusters[2] : n_sm;
  const int csize = p.form == kPair ? 2 : p.split;
  cfg.gridDim = dim3(p.split > 1 ? units * p.split : (units < room ? units : room) * csize);
  cfg.blockDim = dim3(kMmThreads);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (csize > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = csize;
    attr[n].val.clusterDim.y = 1;
    attr[n++].val.clusterDim.z = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, p.form == kPair ? qdense_mma_kernel<kPair> : p.form == kFew ? qdense_mma_kernel<kFew> : qdense_mma_kernel<kOne>,
                            prm);
}
}  // namespace

cudaError_t qdense_set_attributes(int *clusters) {
  cudaError_t e;
  if ((e = set_rows_attr<1>()) || (e = set_rows_attr<2>()) || (e = set_rows_attr<4>()) || (e = set_rows_attr<8>()) ||
      (e = cudaFuncSetAttribute(qdense_few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kQfSmemMax)) ||
      (e = cudaFuncSetAttribute(qdense_mma_kernel<kOne>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMmSmemMax)) ||
      (e = cudaFuncSetAttribute(qdense_mma_kernel<kPair>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMmSmemMax)) ||
      (e = cudaFuncSetAttribute(qdense_mma_kernel<kFew>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMmSmemMax)))
    return e;
  for (int s = 0; s <= kQdenseMaxCluster; ++s) {
    clusters[s] = 0;
    if (s < 2) continue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(s);
    cfg.blockDim = dim3(kMmThreads);
    cfg.dynamicSmemBytes = kMmSmemMax;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = s;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaOccupancyMaxActiveClusters(&clusters[s], qdense_mma_kernel<kFew>, &cfg)))
      return e;
  }
  if (clusters[2] < 1) return cudaErrorInvalidConfiguration;
  return cudaSuccess;
}

// The widened rows of the tensor-core path.
size_t qdense_ws_bytes(int T, int K) {
  return T <= kQdRowsMax ? 0 : ((size_t)T * K * 2 + 255) / 256 * 256;
}

int qdense_launches(int T, int N, int K, int n_sm, const int *clusters) {
  return T > kQdRowsMax && mm_plan(T, N, K, n_sm, clusters).form != kFew ? 2 : 1;
}

cudaError_t launch_qdense(const QdenseArgs &a, int n_sm, const int *clusters, cudaStream_t st, bool pdl) {
  if (a.T > 2 && few_fits(a.T, a.K)) return launch_few(a, n_sm, st, pdl);
  if (a.T <= 1) return launch_rows_t<1>(a, n_sm, st, pdl);
  if (a.T <= 2) return launch_rows_t<2>(a, n_sm, st, pdl);
  if (a.T <= 4) return launch_rows_t<4>(a, n_sm, st, pdl);
  if (a.T <= kQdRowsMax) return launch_rows_t<8>(a, n_sm, st, pdl);
  return launch_mma(a, n_sm, clusters, st, pdl);
}

}  // namespace moe
