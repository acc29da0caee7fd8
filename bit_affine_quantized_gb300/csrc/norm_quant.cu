// Residual addition, root-mean-square norm and 8-bit rows with a scale each:
// what stands between a layer's output and the next 8-bit projection
// (moe_norm_quant).  Per row of width H:
//
//   s = bf16(h + y)                     (s = h without y)
//   u = s * g                           (u = s without a norm weight)
//   r = 1 / sqrt(mean(s^2) + eps),  m = max |u|
//   q = rint(127 u / m),  scale = m r / 127,  x = bf16(u r)
//
// The rows' common factor r cancels in the codes, so they need the maximum of
// u alone and one block reduction serves both statistics.  u is the product of
// two bf16 numbers, exact in fp32, and so is 127 u (8 + 8 + 7 bits); the
// quotient is rounded once, and no quotient of such numbers lies closer to a
// half integer than that rounding moves it: with B the 16-bit significand of
// m and 2^j <= |127 u / m| < 2^(j+1), a quotient that is no half integer is
// at least 2^(j-6) / (2 B) > 2^(j-23) away from one, and the rounding moves
// it by at most 2^(j-24).  The codes are therefore those of exact arithmetic,
// ties to even, whatever the order of the sums.
//
// One block per row: the row stays in registers between the statistics and
// the codes, so every byte moves once.
#include <math.h>

#include "kernels.h"

namespace moe {

namespace {
constexpr unsigned kInfBits = 0x7F800000u;

__device__ __forceinline__ float nq_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float nq_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t nq_pack(float lo, float hi) {
  return (uint32_t)float_to_bf16_bits(lo) | ((uint32_t)float_to_bf16_bits(hi) << 16);
}

// kVec: 8-element vectors of the row per thread (blockDim.x * kVec * 8 >= H)
template <int kVec>
__global__ void __launch_bounds__(1024) norm_quant_kernel(const NormQuantArgs a) {
  __shared__ float s_sum[32];
  __shared__ unsigned s_max[32];
  const int H = a.H, nvec = H / 8, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const size_t row = blockIdx.x;
  const bool tracer = blockIdx.x == 0 && tid == 0;
  if (tracer) trace_min(a.trace, kTrEntry);
  pdl_wait();
  pdl_launch_dependents();
  if (tracer) trace_min(a.trace, kTrWaited);

  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const uint4 *h4 = reinterpret_cast<const uint4 *>(a.h + row * H);
  uint4 hv[kVec], yv[kVec], gv[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int v = tid + i * blockDim.x;
    hv[i] = v < nvec ? __ldcs(h4 + v) : zero;
    yv[i] = a.y && v < nvec ? __ldcs(reinterpret_cast<const uint4 *>(a.y + row * H) + v) : zero;
    gv[i] = a.g && v < nvec ? __ldg(reinterpret_cast<const uint4 *>(a.g) + v) : zero;
  }
  float u[kVec][8];
  float ss = 0.f;
  unsigned mx = 0u;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int v = tid + i * blockDim.x;
    uint32_t hw[4] = {hv[i].x, hv[i].y, hv[i].z, hv[i].w};
    const uint32_t yw[4] = {yv[i].x, yv[i].y, yv[i].z, yv[i].w}, gw[4] = {gv[i].x, gv[i].y, gv[i].z, gv[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (a.y) hw[j] = nq_pack(nq_lo(hw[j]) + nq_lo(yw[j]), nq_hi(hw[j]) + nq_hi(yw[j]));
      const float s0 = nq_lo(hw[j]), s1 = nq_hi(hw[j]);
      ss = fmaf(s0, s0, fmaf(s1, s1, ss));
      u[i][2 * j] = a.g ? s0 * nq_lo(gw[j]) : s0;
      u[i][2 * j + 1] = a.g ? s1 * nq_hi(gw[j]) : s1;
      // as bit patterns: infinity and NaN compare above every finite value
      mx = max(mx, max(__float_as_uint(u[i][2 * j]) & 0x7FFFFFFFu, __float_as_uint(u[i][2 * j + 1]) & 0x7FFFFFFFu));
    }
    if (a.h_out && v < nvec)
      reinterpret_cast<uint4 *>(a.h_out + row * H)[v] = make_uint4(hw[0], hw[1], hw[2], hw[3]);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
  mx = __reduce_max_sync(0xffffffffu, mx);
  if (lane == 0) {
    s_sum[warp] = ss;
    s_max[warp] = mx;
  }
  __syncthreads();
  const int nw = blockDim.x >> 5;
  float tot = lane < nw ? s_sum[lane] : 0.f;
  unsigned m = lane < nw ? s_max[lane] : 0u;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, off);
  m = __reduce_max_sync(0xffffffffu, m);

  const bool bad = m >= kInfBits || !(tot < INFINITY);
  const float mf = __uint_as_float(m);
  const float r = 1.0f / sqrtf(tot / (float)H + a.eps);
  if (tid == 0) {
    if (bad) set_error(a.err, kErrNonFinite);
    a.scales[row] = bad ? NAN : mf * r / 127.0f;
  }
  // a power of two that keeps 127 u and the divisor in range (exact)
  const float pre = mf > 1.2676506e30f ? 0x1p-24f : mf < 0x1p-80f ? 0x1p40f : 1.0f;
  const float num = 127.0f * pre, den = mf * pre;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int v = tid + i * blockDim.x;
    if (v >= nvec) continue;
    uint32_t qw[2] = {0u, 0u};
    if (!bad && m != 0u) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        qw[j >> 2] |= (uint32_t)(__float2int_rn(__fdiv_rn(u[i][j] * num, den)) & 0xFF) << (8 * (j & 3));
    }
    reinterpret_cast<uint2 *>(a.q + row * H)[v] = make_uint2(qw[0], qw[1]);
    if (a.x_out) {
      uint32_t xw[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) xw[j] = bad ? 0x7FFF7FFFu : nq_pack(u[i][2 * j] * r, u[i][2 * j + 1] * r);
      reinterpret_cast<uint4 *>(a.x_out + row * H)[v] = make_uint4(xw[0], xw[1], xw[2], xw[3]);
    }
  }
  if (tracer) trace_max(a.trace, kTrExit);
}
}  // namespace

cudaError_t launch_norm_quant(const NormQuantArgs &a, cudaStream_t st, bool pdl) {
  if (a.T < 1 || a.H < 16 || a.H % 16 || a.H > kNormMaxWidth) return cudaErrorInvalidValue;
  const int nvec = a.H / 8;
  auto block = [&](int per) { return dim3((((nvec + per - 1) / per) + 31) / 32 * 32); };
  if (nvec <= 1024) return launch_k(norm_quant_kernel<1>, dim3(a.T), block(1), 0, st, pdl, a);
  return launch_k(norm_quant_kernel<2>, dim3(a.T), block(2), 0, st, pdl, a);
}

}  // namespace moe
