// Rotary positions on queries and keys, keys and values into a paged cache, in
// bf16 or as 8-bit rows with a scale each (moe_kv_append), and rows of the cache
// back as bf16 (moe_kv_read).
//
// A pair (x_j, x_{j + r/2}) of a head turns by the angle a = pos f_j.  In turns,
// pos f_j / (2 pi) in 64 bits less its nearest integer is exact to 2^-53 of the
// turns counted, so that a position of 2^30 still has its angle to 2^-22; the
// sine and cosine are then taken of the remainder in 32 bits.  A block works
// them out once per row, in shared memory, for all heads.
//
// An 8-bit row of a head is rint(127 x / m) with m its largest magnitude, and
// the scale m / 127: one rounding from the turned key, which is never rounded to
// bf16 on the way.  For a value's row 127 x is exact (8 + 7 bits) and the
// division is rounded once, so its codes are those of exact arithmetic, ties to
// even: with M the 8-bit significand of m and 2^j <= |127 x / m| < 2^(j+1), a
// quotient that is no half integer is at least 2^(j-6) / (2 M) > 2^(j-15) away
// from one, and the rounding moves it by at most 2^(j-24).
//
// A thread has two vectors of eight values that turn together: v and v + r/16 of
// the first r dimensions, or two neighbours behind them; D / 16 threads have a
// head's row, and its maximum goes round them by shuffles.
#include <math.h>

#include "kernels.h"

namespace moe {

namespace {
constexpr int kKvThreads = 256;

__device__ __forceinline__ float kv_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float kv_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t kv_pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ void kv_unpack(const uint4 w, float *f) {
  const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = kv_lo(a[j]);
    f[2 * j + 1] = kv_hi(a[j]);
  }
}
__device__ __forceinline__ uint4 kv_pack8(const float *f) {
  return make_uint4(kv_pack(f[0], f[1]), kv_pack(f[2], f[3]), kv_pack(f[4], f[5]), kv_pack(f[6], f[7]));
}
// The larger of two, NaN if one of them is.
__device__ __forceinline__ float kv_max(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <bool kBits8>
__global__ void __launch_bounds__(kKvThreads) kv_append_kernel(const KvAppendArgs a) {
  __shared__ float2 s_turn[128];  // cosine and sine of the row's angles
  const int tid = threadIdx.x, row = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
  const bool tracer = a.trace && blockIdx.x == 0 && tid == 0;
  if (tracer) trace_min(a.trace, kTrEntry);
  pdl_wait();
  pdl_launch_dependents();
  if (tracer) trace_min(a.trace, kTrWaited);
  const int pos = __ldg(a.pos + row);
  if (pos >= 0) {
    const long long at = kv_row(a.c, a.seq ? __ldg(a.seq + row) : row, pos);
    if (at < 0 && part == 0 && tid == 0) set_error(a.err, kErrBadId);
    if (tid < a.rot / 2) {
      const double turns = (double)pos * ((double)__ldg(a.freq + tid) * 0.15915494309189535);  // 1 / (2 pi)
      float s, c;
      sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
      s_turn[tid] = make_float2(c, s);
    }
    __syncthreads();

    const int D = a.c.D, pairs = D / 16, turned = a.rot / 16;
    const int lanes = pairs <= 1 ? 1 : 1 << (32 - __clz(pairs - 1));  // threads of a head's row: a power of two
    const int me = tid % lanes, per = kKvThreads / lanes;
    const int va = me < turned ? me : 2 * me, vb = me < turned ? me + turned : 2 * me + 1;  // my two vectors
    const int heads = a.Hq + 2 * a.c.heads;
    // (whole warps go round together: the shuffles below need every lane)
    for (int h0 = part * per; h0 < heads; h0 += a.parts * per) {
      const int h = h0 + tid / lanes;
      const bool is_q = h < a.Hq, is_k = !is_q && h < a.Hq + a.c.heads;
      const bool mine = h < heads && me < pairs && (is_q || at >= 0);
      const uint16_t *from = is_q   ? a.q + (size_t)row * a.ldq + (size_t)h * D
                             : is_k ? a.k + (size_t)row * a.ldk + (size_t)(h - a.Hq) * D
                                    : a.v + (size_t)row * a.ldv + (size_t)(h - a.Hq - a.c.heads) * D;
      float x[16];
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      kv_unpack(mine ? __ldg(reinterpret_cast<const uint4 *>(from) + va) : zero, x);
      kv_unpack(mine ? __ldg(reinterpret_cast<const uint4 *>(from) + vb) : zero, x + 8);
      if ((is_q || is_k) && me < turned) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 t = s_turn[8 * me + j];
          const float u = x[j], w = x[j + 8];
          x[j] = u * t.x - w * t.y;
          x[j + 8] = w * t.x + u * t.y;
        }
      }
      if (is_q) {
        if (mine) {
          uint4 *to = reinterpret_cast<uint4 *>(a.q_out + (size_t)row * a.ldo + (size_t)h * D);
          to[va] = kv_pack8(x);
          to[vb] = kv_pack8(x + 8);
        }
      }
      const int kv_head = is_q ? 0 : is_k ? h - a.Hq : h - a.Hq - a.c.heads;
      const size_t place = (size_t)(at + (long long)kv_head * a.c.rows);  // of the head's row in the pages
      if (!kBits8) {
        if (mine && !is_q) {
          uint4 *to = reinterpret_cast<uint4 *>((is_k ? a.c.k : a.c.v) + place * D * 2);
          to[va] = kv_pack8(x);
          to[vb] = kv_pack8(x + 8);
        }
        continue;
      }
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) m = kv_max(m, fabsf(x[j]));
      for (int off = lanes / 2; off > 0; off >>= 1) m = kv_max(m, __shfl_xor_sync(0xffffffffu, m, off));
      if (!mine || is_q) continue;
      const bool bad = !(m < INFINITY);
      // a power of two that keeps 127 x and the divisor in range (exact)
      const float pre = m > 0x1p100f ? 0x1p-24f : m < 0x1p-80f ? 0x1p40f : 1.0f;
      const float den = m * pre;
      uint32_t w[4] = {0u, 0u, 0u, 0u};
      if (!bad && m > 0.f) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int q = __float2int_rn(__fdiv_rn(x[j] * pre * 127.0f, den));
          w[j / 4] |= (uint32_t)(q & 255) << (8 * (j % 4));
        }
      }
      uint2 *to = reinterpret_cast<uint2 *>((is_k ? a.c.k : a.c.v) + place * D);
      to[va] = make_uint2(w[0], w[1]);
      to[vb] = make_uint2(w[2], w[3]);
      if (me == 0) (is_k ? a.c.ks : a.c.vs)[place] = bad ? NAN : m / 127.0f;
      if (me == 0 && bad) set_error(a.err, kErrNonFinite);
    }
  }
  if (a.trace && tid == 0) trace_max(a.trace, kTrExit);
}

// One row per block and turn: its place once, then a vector of 16 values per thread.
template <bool kBits8>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const KvReadArgs a) {
  const int tid = threadIdx.x;
  const bool tracer = a.trace && blockIdx.x == 0 && tid == 0;
  if (tracer) trace_min(a.trace, kTrEntry);
  pdl_wait();
  pdl_launch_dependents();
  if (tracer) trace_min(a.trace, kTrWaited);
  const int D = a.c.D, vecs = D / 16, n = a.c.heads * vecs;
  for (int r = blockIdx.x * a.per; r < min(a.T, (int)(blockIdx.x + 1) * a.per); ++r) {
    const int pos = __ldg(a.pos + r);
    if (pos < 0) continue;
    const long long at = kv_row(a.c, a.seq ? __ldg(a.seq + r) : r, pos);
    if (at < 0 && tid == 0) set_error(a.err, kErrBadId);
    for (int i = tid; i < 2 * n; i += kKvThreads) {
      const bool is_k = i < n;
      uint16_t *out = is_k ? a.k : a.v;
      if (!out) continue;
      const int e = is_k ? i : i - n, head = e / vecs, vec = e % vecs;
      uint4 *to = reinterpret_cast<uint4 *>(out + (size_t)r * (is_k ? a.ldk : a.ldv)) + 2 * e;
      uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
      if (at >= 0) {
        const size_t place = (size_t)(at + (long long)head * a.c.rows);
        const uint8_t *from = is_k ? a.c.k : a.c.v;
        if (kBits8) {
          const float s = __ldg((is_k ? a.c.ks : a.c.vs) + place);
          const uint4 w = __ldg(reinterpret_cast<const uint4 *>(from + place * D) + vec);
          const uint32_t c[4] = {w.x, w.y, w.z, w.w};
          float f[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) f[j] = (float)(int8_t)(c[j / 4] >> (8 * (j % 4))) * s;
          lo = kv_pack8(f);
          hi = kv_pack8(f + 8);
        } else {
          const uint4 *p = reinterpret_cast<const uint4 *>(from + place * D * 2) + 2 * vec;
          lo = __ldg(p);
          hi = __ldg(p + 1);
        }
      }
      to[0] = lo;
      to[1] = hi;
    }
  }
  if (a.trace && tid == 0) trace_max(a.trace, kTrExit);
}
}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs &a0, int n_sm, cudaStream_t st, bool pdl) {
  KvAppendArgs a = a0;
  a.parts = 1;
  return launch_k(a.c.ks ? kv_append_kernel<true> : kv_append_kernel<false>, dim3((unsigned)a.T * a.parts),
                  dim3(kKvThreads), 0, st, pdl, a);
}

cudaError_t launch_kv_read(const KvReadArgs &a0, int n_sm, cudaStream_t st, bool pdl) {
  KvReadArgs a = a0;
  a.per = 1;
  return launch_k(a.c.ks ? kv_read_kernel<true> : kv_read_kernel<false>, dim3((unsigned)((a.T + a.per - 1) / a.per)),
                  dim3(kKvThreads), 0, st, pdl, a);
}

}  // namespace moe
