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
// ties to even, whatever the order of the sums.  (Products below fp32's normal
// range, 2^-126, round when they are formed.)
//
// The kernel multiplies by k = 127 / m and divides only the vectors that have a
// product within 2^-14 of a half integer: k is within 2 roundings of its value
// and the product adds one, so the product is within 3 * 2^-24 * 127 < 2^-15
// of the quotient and every other product rounds to the same code.  (Dividing
// throughout, the kernel was bound by its instructions: 18.2 us at 4096 x
// 2816 against 14.5.)
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
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
// The larger of two, NaN if one of them is (the sign of a zero does not matter here).
__device__ __forceinline__ float nq_max(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// kVec: 8-element vectors of the row per thread (blockDim.x * kVec * 8 >= H)
template <int kVec>
__global__ void __launch_bounds__(kVec <= 2 ? 1024 : 512) norm_quant_kernel(const NormQuantArgs a) {
  __shared__ float s_sum[32];
  __shared__ unsigned s_max[32];
  const int H = a.H, nvec = H / 8, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nw = blockDim.x >> 5;
  const size_t row = blockIdx.x, at = row * H;
  const bool leaver = a.trace && tid == 0, tracer = blockIdx.x == 0 && leaver;
  if (tracer) trace_min(a.trace, kTrEntry);
  pdl_wait();
  pdl_launch_dependents();
  if (tracer) trace_min(a.trace, kTrWaited);

  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  uint4 hv[kVec], yv[kVec], gv[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int v = tid + i * blockDim.x;
    hv[i] = v < nvec ? __ldcs(reinterpret_cast<const uint4 *>(a.h + at) + v) : zero;
    yv[i] = a.y && v < nvec ? __ldcs(reinterpret_cast<const uint4 *>(a.y + at) + v) : zero;
    gv[i] = a.g && v < nvec ? __ldg(reinterpret_cast<const uint4 *>(a.g) + v) : zero;
  }
  float u[kVec][8];
  // The squares of two vectors each: no chain of additions is longer than 16, so a
  // scale is within 20 * 2^-24 of its value (16 + 1 + 10 roundings of the sum, halved
  // by the square root, and 6 more operations).
  constexpr int kParts = (kVec + 1) / 2;
  float part[kParts], mx = 0.f;
#pragma unroll
  for (int p = 0; p < kParts; ++p) part[p] = 0.f;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int v = tid + i * blockDim.x;
    uint32_t h4[4] = {hv[i].x, hv[i].y, hv[i].z, hv[i].w};
    const uint32_t y4[4] = {yv[i].x, yv[i].y, yv[i].z, yv[i].w}, g4[4] = {gv[i].x, gv[i].y, gv[i].z, gv[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (a.y) h4[j] = nq_pack(nq_lo(h4[j]) + nq_lo(y4[j]), nq_hi(h4[j]) + nq_hi(y4[j]));
      const float s0 = nq_lo(h4[j]), s1 = nq_hi(h4[j]);
      part[i / 2] = fmaf(s0, s0, fmaf(s1, s1, part[i / 2]));
      u[i][2 * j] = a.g ? s0 * nq_lo(g4[j]) : s0;
      u[i][2 * j + 1] = a.g ? s1 * nq_hi(g4[j]) : s1;
      mx = nq_max(nq_max(mx, fabsf(u[i][2 * j])), fabsf(u[i][2 * j + 1]));
    }
    if (a.h_out && v < nvec) __stcs(reinterpret_cast<uint4 *>(a.h_out + at) + v, make_uint4(h4[0], h4[1], h4[2], h4[3]));
  }
  float ss = part[0];
#pragma unroll
  for (int p = 1; p < kParts; ++p) ss += part[p];
  // as bit patterns infinity and NaN compare above every finite value
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
  const unsigned mw = __reduce_max_sync(0xffffffffu, __float_as_uint(mx));
  float tot = ss;
  unsigned m = mw;
  if (nw > 1) {
    if (lane == 0) {
      s_sum[warp] = ss;
      s_max[warp] = mw;
    }
    __syncthreads();
    tot = lane < nw ? s_sum[lane] : 0.f;
    m = lane < nw ? s_max[lane] : 0u;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, off);
    m = __reduce_max_sync(0xffffffffu, m);
  }

  const float mf = __uint_as_float(m);
  // (a row of zeros: 0, where eps = 0 would make it infinite)
  const float r = m == 0u ? 0.0f : 1.0f / sqrtf(tot / (float)H + a.eps);
  const float mr = mf * r;  // the largest normalised value (infinite if r is)
  const bool bad = m >= kInfBits || !(tot < INFINITY) || !(mr < a.most);
  if (tid == 0) {
    if (bad) set_error(a.err, kErrNonFinite);
    a.scales[row] = bad ? NAN : mr / 127.0f;
  }
  // a power of two that keeps 127 u and the divisor in range (exact)
  const float pre = mf > 0x1p100f ? 0x1p-24f : mf < 0x1p-80f ? 0x1p40f : 1.0f;
  const float num = 127.0f * pre, den = mf * pre;
  const bool zeros = bad || m == 0u;
  const float k = num / den, kAdd = 12582912.0f;  // 3 * 2^22: adding it rounds to an integer, held in the low bits
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int v = tid + i * blockDim.x;
    if (v >= nvec) continue;
    uint32_t qw[2] = {0u, 0u};
    if (!zeros) {
      float far = mf < 0x1p-80f ? 1.f : 0.f, z[8];  // (k may be out of range there)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float c = u[i][j] * k;
        z[j] = c + kAdd;
        far = fmaxf(far, fabsf(c - (z[j] - kAdd)));
      }
      if (far > 0.5f - 0x1p-14f) {  // near a half integer: the quotient itself decides
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = __fdiv_rn(u[i][j] * num, den) + kAdd;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
        qw[j] = __byte_perm(__byte_perm(__float_as_uint(z[4 * j]), __float_as_uint(z[4 * j + 1]), 0x0040),
                            __byte_perm(__float_as_uint(z[4 * j + 2]), __float_as_uint(z[4 * j + 3]), 0x0040), 0x5410);
    }
    __stcs(reinterpret_cast<uint2 *>(a.q + at) + v, make_uint2(qw[0], qw[1]));
    if (a.x_out) {
      uint32_t xw[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) xw[j] = bad ? 0x7FFF7FFFu : nq_pack(u[i][2 * j] * r, u[i][2 * j + 1] * r);
      __stcs(reinterpret_cast<uint4 *>(a.x_out + at) + v, make_uint4(xw[0], xw[1], xw[2], xw[3]));
    }
  }
  if (leaver) trace_max(a.trace, kTrExit);
}

template <int kVec>
cudaError_t launch_rows(const NormQuantArgs &a, cudaStream_t st, bool pdl) {
  const int threads = ((a.H / 8 + kVec - 1) / kVec + 31) / 32 * 32;
  return launch_k(norm_quant_kernel<kVec>, dim3(a.T), dim3(threads), 0, st, pdl, a);
}
}  // namespace

// Vectors per thread: many rows go with few threads each, whose loads are all
// in flight (4096 x 2816 at kVec 1, 2, 4: 17.5, 16.2, 14.7 us, 81 MB at 5.5
// TB/s; 600 rows: 3.8, 3.8, 3.6); few rows finish sooner with more threads
// (128 rows: 2.12, 2.33, 2.80 us; one row 2.0, 2.05, 2.4).
cudaError_t launch_norm_quant(const NormQuantArgs &a0, int n_sm, cudaStream_t st, bool pdl) {
  NormQuantArgs a = a0;
  // past fp32's range the scale would be infinite, from 2^128 - 2^119 on its bf16 rounding
  a.most = a.x_out ? 0x1.FFp127f : INFINITY;
  if (a.T < 1 || a.H < 16 || a.H % 16 || a.H > kNormMaxWidth) return cudaErrorInvalidValue;
  if (a.T > 3 * n_sm) return launch_rows<4>(a, st, pdl);
  return a.H <= 8 * 1024 ? launch_rows<1>(a, st, pdl) : launch_rows<2>(a, st, pdl);
}

}  // namespace moe
