// Dense projection of 8-bit rows with an 8-bit matrix, a scale per row and per
// output channel (moe_qdense_forward):
//
//   y[t, n] = cap(xs[t] * ws[n] * sum_k x[t, k] w[n, k]),  cap(z) = c tanh(z / c) or z
//
// qdense_rows_kernel: up to 8 rows per block row of the grid.  A warp takes
// kR channels; each lane loads 16 bytes of every channel's row (one 512-byte
// run per warp and channel) and multiplies them with the rows' codes in
// shared memory by dp4a, so the sums are exact 32-bit integers (at most
// 128 * 128 * 16384 = 2^28 in magnitude).
#include <math.h>

#include "kernels.h"

namespace moe {

namespace {
constexpr int kQdWarps = 8;
constexpr int kQdThreads = kQdWarps * 32;

__device__ __forceinline__ int4 qd_stream(const int8_t *p) {
  int4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ float qd_finish(int acc, float xs, float ws, float cap) {
  const float v = __fmul_rn(__fmul_rn((float)acc, xs), ws);
  return cap > 0.f ? cap * tanhf(v / cap) : v;
}

template <int kT, int kR>
__global__ void __launch_bounds__(kQdThreads) qdense_rows_kernel(const QdenseArgs a) {
  extern __shared__ __align__(16) int4 qsm[];  // [kT][K / 16]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int K = a.K, nck = K / 16, t0 = blockIdx.y * kT, nt = min(kT, a.T - t0);
  const bool tracer = blockIdx.x == 0 && blockIdx.y == 0 && tid == 0;
  if (tracer) trace_min(a.trace, kTrEntry);
  pdl_wait();
  pdl_launch_dependents();
  if (tracer) trace_min(a.trace, kTrWaited);
  const int4 *x4 = reinterpret_cast<const int4 *>(a.x + (size_t)t0 * K);
  for (int i = tid; i < kT * nck; i += kQdThreads) qsm[i] = i < nt * nck ? __ldcg(x4 + i) : make_int4(0, 0, 0, 0);
  __syncthreads();
  const int units = (a.N + kR - 1) / kR;
  for (int u = blockIdx.x * kQdWarps + warp; u < units; u += gridDim.x * kQdWarps) {
    const int n0 = u * kR;
    const int8_t *wr[kR];
#pragma unroll
    for (int r = 0; r < kR; ++r) wr[r] = a.w + (size_t)min(n0 + r, a.N - 1) * K;  // past N: discarded below
    int acc[kR][kT];
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
      for (int t = 0; t < kT; ++t) acc[r][t] = 0;
#pragma unroll 2
    for (int c = lane; c < nck; c += 32) {
      int4 w[kR];
#pragma unroll
      for (int r = 0; r < kR; ++r) w[r] = qd_stream(wr[r] + 16 * c);
#pragma unroll
      for (int t = 0; t < kT; ++t) {
        const int4 x = qsm[t * nck + c];
#pragma unroll
        for (int r = 0; r < kR; ++r)
          acc[r][t] = __dp4a(w[r].w, x.w, __dp4a(w[r].z, x.z, __dp4a(w[r].y, x.y, __dp4a(w[r].x, x.x, acc[r][t]))));
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
    if (r < kR && t < nt && n0 + r < a.N) {
      const float v = qd_finish(mine, __ldcg(a.xs + t0 + t), __ldg(a.ws + n0 + r), a.softcap);
      const size_t o = (size_t)(t0 + t) * a.N + n0 + r;
      if (a.y32) a.y32[o] = v;
      if (a.y) a.y[o] = float_to_bf16_bits(v);
    }
  }
  if (tracer) trace_max(a.trace, kTrExit);
}

template <int kT, int kR>
cudaError_t launch_rows(const QdenseArgs &a, int n_sm, cudaStream_t st, bool pdl) {
  const size_t smem = (size_t)kT * a.K;
  int per_sm = 0;
  cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, qdense_rows_kernel<kT, kR>, kQdThreads, smem);
  if (e != cudaSuccess) return e;
  if (per_sm < 1) return cudaErrorInvalidConfiguration;
  const int units = (a.N + kR - 1) / kR, blocks = (units + kQdWarps - 1) / kQdWarps;
  const int most = n_sm * per_sm;
  return launch_k(qdense_rows_kernel<kT, kR>, dim3(blocks < most ? blocks : most, (a.T + kT - 1) / kT),
                  dim3(kQdThreads), smem, st, pdl, a);
}

template <int kT>
cudaError_t launch_rows_t(const QdenseArgs &a, int n_sm, cudaStream_t st, bool pdl) {
  if (a.N >= 4 * kQdWarps * 4 * n_sm) return launch_rows<kT, 4>(a, n_sm, st, pdl);
  return launch_rows<kT, 1>(a, n_sm, st, pdl);
}

template <int kT>
cudaError_t set_rows_attr() {
  cudaError_t e = cudaFuncSetAttribute(qdense_rows_kernel<kT, 4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kT * kQdenseMaxK);
  if (e) return e;
  return cudaFuncSetAttribute(qdense_rows_kernel<kT, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kT * kQdenseMaxK);
}
}  // namespace

cudaError_t qdense_set_attributes() {
  cudaError_t e;
  if ((e = set_rows_attr<1>()) || (e = set_rows_attr<2>()) || (e = set_rows_attr<4>()) || (e = set_rows_attr<8>()))
    return e;
  return cudaSuccess;
}

size_t qdense_ws_bytes(int T, int K) {
  (void)T;
  (void)K;
  return 0;
}

cudaError_t launch_qdense(const QdenseArgs &a, int n_sm, cudaStream_t st, bool pdl) {
  if (a.T <= 1) return launch_rows_t<1>(a, n_sm, st, pdl);
  if (a.T <= 2) return launch_rows_t<2>(a, n_sm, st, pdl);
  if (a.T <= 4) return launch_rows_t<4>(a, n_sm, st, pdl);
  return launch_rows_t<8>(a, n_sm, st, pdl);
}

}  // namespace moe
