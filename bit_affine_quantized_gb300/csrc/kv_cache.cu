// Rotary positions on queries and keys, keys and values into a paged cache, in
// bf16 or as 8-bit rows with a scale each (moe_kv_append), and rows of the cache
// back as bf16 (moe_kv_read).
//
// A pair (x_j, x_{j + r/2}) of a head turns by the angle a = pos f_j.  Angles count
// in turns modulo one: with w = f_j / (2 pi) as a 64-bit fraction, pos w modulo 2^64
// is one integer product, and its upper 32 bits are the angle to 2^-32 of a turn
// whatever the position: w, the product of f_j's 24 bits and 1 / (2 pi) to 64 bits,
// is good to 2^-64 for f up to 1, pos w to 2^-34 at position 2^30.  Sine and cosine
// are then taken in 32 bits, once per row for all heads, in shared memory, in the
// order in which the threads of a head read them.  No 64-bit floating point: this
// chip has little of it.
//
// An 8-bit row of a head is rint(127 x / m) with m its largest magnitude, and
// the scale m / 127: one rounding from the turned key, which is never rounded to
// bf16 on the way.  For a value's row 127 x is exact (8 + 7 bits) and the
// division is rounded once, so its codes are those of exact arithmetic, ties to
// even: with M the 8-bit significand of m and 2^j <= |127 x / m| < 2^(j+1), a
// quotient that is no half integer is at least 2^(j-6) / (2 M) > 2^(j-15) away
// from one, and the rounding moves it by at most 2^(j-24).  The kernel multiplies
// by 127 / m (with its errors within 6 * 2^-24 * 127 < 2^-14 of the quotient) and
// divides the eights that have a product within 2^-14 of a half integer.
//
// A thread has two vectors of eight values that turn together: v and v + r/16 of
// the first r dimensions, or two neighbours behind them; D / 16 threads have a
// head's row, and its maximum goes round them by shuffles.  All loads of a
// thread's two units are on their way before the first is used.
//
// 4096 rows of 16 query and 2 x 8 key and value heads of 256, turned: 23.7 us in
// bf16 (134 MB, 5.7 TB/s), 28 in 8 bits (117 MB, 4.2 TB/s: the issue slots are 72 %
// used, 346 instructions a unit and warp); 31 and 25 with four units a thread, 32 and
// 27 with one.  The angles' table read across its banks and 64-bit floating point per
// row cost 10 us of it.
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

constexpr int kKvUnits = 2;  // of a thread, whose loads go together
constexpr int kKvMaxBlockRows = 8;

// f / (2 pi) in turns modulo one, times 2^64.
__device__ __forceinline__ unsigned long long kv_turns(float f) {
  constexpr unsigned long long kTurn = 0x28BE60DB9391054Aull;  // 2^64 / (2 pi)
  const unsigned b = __float_as_uint(f), e = b >> 23 & 255u;
  const unsigned long long m = e ? (b & 0x7FFFFFu) | 0x800000u : b & 0x7FFFFFu;  // |f| = m 2^-down
  const int down = 150 - (int)max(e, 1u);
  const unsigned long long lo = m * kTurn, hi = __umul64hi(m, kTurn);
  const unsigned long long w = down >= 128 ? 0 : down >= 64 ? hi >> (down - 64)
                               : down > 0 ? hi << (64 - down) | lo >> down : down > -64 ? lo << -down : 0;
  return b >> 31 ? 0 - w : w;
}

// 127 x / m to the nearest integer, ties to even, as bytes; den = m pre, k = 127 pre / den.
__device__ __forceinline__ uint2 kv_codes(const float *x, float pre, float den, float k, bool small) {
  constexpr float kAdd = 12582912.0f;  // 3 * 2^22: adding it rounds to an integer, held in the low bits
  float z[8], far = small ? 1.f : 0.f;  // (k may be out of range there)
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float c = x[j] * k;
    z[j] = c + kAdd;
    far = fmaxf(far, fabsf(c - (z[j] - kAdd)));
  }
  if (far > 0.5f - 0x1p-14f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = __fdiv_rn(x[j] * pre * 127.0f, den) + kAdd;
  }
  uint32_t w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j)
    w[j] = __byte_perm(__byte_perm(__float_as_uint(z[4 * j]), __float_as_uint(z[4 * j + 1]), 0x0040),
                       __byte_perm(__float_as_uint(z[4 * j + 2]), __float_as_uint(z[4 * j + 3]), 0x0040), 0x5410);
  return make_uint2(w[0], w[1]);
}

template <bool kBits8>
__global__ void __launch_bounds__(kKvThreads, 5) kv_append_kernel(const KvAppendArgs a) {
  __shared__ float2 s_turn[kKvMaxBlockRows][8][16];  // cosine and sine of the rows' angles 8 i + j, at j, i
  __shared__ long long s_at[kKvMaxBlockRows];       // the rows' places; -1: not there, -2: left out
  const int tid = threadIdx.x, part = blockIdx.x % a.parts, row0 = blockIdx.x / a.parts * a.per;
  const int rows = min(a.per, a.T - row0);
  const bool tracer = a.trace && blockIdx.x == 0 && tid == 0;
  if (tracer) trace_min(a.trace, kTrEntry);
  pdl_wait();
  pdl_launch_dependents();
  if (tracer) trace_min(a.trace, kTrWaited);
  const int D = a.c.D, pairs = D / 16, turned = a.rot / 16;
  const int log_lanes = pairs <= 1 ? 0 : 32 - __clz(pairs - 1);  // threads of a head's row: a power of two
  const int me = tid & ((1 << log_lanes) - 1), heads = a.Hq + 2 * a.c.heads, units = rows * heads;
  const int va = me < turned ? me : 2 * me, vb = me < turned ? me + turned : 2 * me + 1;  // my two vectors
  const int step = kKvThreads >> log_lanes;  // head rows that the block takes at once
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const float per_head = 1.0f / (float)heads;
  bool ready = false;
  // (whole warps go round together: the shuffles below need every lane)
  for (int i0 = part * kKvUnits * step; i0 < units; i0 += a.parts * kKvUnits * step) {
    uint4 xa[kKvUnits], xb[kKvUnits];
    int row[kKvUnits], head[kKvUnits];
#pragma unroll
    for (int n = 0; n < kKvUnits; ++n) {
      const int i = i0 + n * step + (tid >> log_lanes);
      const bool mine = i < units && me < pairs;
      row[n] = mine ? (int)(((float)i + 0.5f) * per_head) : -1;  // (i / heads: exact below 2^20)
      head[n] = mine ? i - row[n] * heads : 0;
      const size_t t = (size_t)(row0 + max(row[n], 0));
      const int h = head[n], k = h - a.Hq, v = k - a.c.heads;
      const uint16_t *from = h < a.Hq ? a.q + t * a.ldq + (size_t)h * D : k < a.c.heads ? a.k + t * a.ldk + (size_t)k * D
                                                                                          : a.v + t * a.ldv + (size_t)v * D;
      xa[n] = mine ? *(reinterpret_cast<const uint4 *>(from) + va) : zero;
      xb[n] = mine ? *(reinterpret_cast<const uint4 *>(from) + vb) : zero;
    }
    if (!ready) {  // the rows' places and angles, while the values are on their way
      ready = true;
      if (tid < rows) {
        const int pos = __ldg(a.pos + row0 + tid);
        const long long at = pos < 0 ? -2 : kv_row(a.c, a.seq ? __ldg(a.seq + row0 + tid) : row0 + tid, pos);
        s_at[tid] = at;
        if (at == -1 && part == 0) set_error(a.err, kErrBadId);
      }
      for (int i = tid; i < rows * a.rot / 2; i += kKvThreads) {
        const int r = i / (a.rot / 2), p = i - r * (a.rot / 2);
        const float f = __ldg(a.freq + p);
        const int turn = (int)((kv_turns(f) * (unsigned)max(__ldg(a.pos + row0 + r), 0)) >> 32);  // in 2^-32 of one
        float s, c;
        sincospif((float)turn * 0x1p-31f, &s, &c);
        s_turn[r][p & 7][p >> 3] = make_float2(fmaf(f, 0.f, c), fmaf(f, 0.f, s));  // (an infinite frequency: NaN)
      }
      __syncthreads();
    }
#pragma unroll
    for (int n = 0; n < kKvUnits; ++n) {
      if (__all_sync(0xffffffffu, row[n] < 0)) continue;
      const long long at = row[n] >= 0 ? s_at[row[n]] : -2;
      const bool is_q = head[n] < a.Hq, is_k = !is_q && head[n] < a.Hq + a.c.heads, mine = is_q ? at > -2 : at >= 0;
      float x[16];
      kv_unpack(xa[n], x);
      kv_unpack(xb[n], x + 8);
      if ((is_q || is_k) && me < turned && row[n] >= 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 t = s_turn[row[n]][j][me];
          const float u = x[j], w = x[j + 8];
          x[j] = u * t.x - w * t.y;
          x[j + 8] = w * t.x + u * t.y;
        }
      }
      if (is_q && mine) {
        uint4 *to = reinterpret_cast<uint4 *>(a.q_out + (size_t)(row0 + row[n]) * a.ldo + (size_t)head[n] * D);
        to[va] = kv_pack8(x);
        to[vb] = kv_pack8(x + 8);
      }
      const int kv_head = is_q ? 0 : is_k ? head[n] - a.Hq : head[n] - a.Hq - a.c.heads;
      const size_t place = (size_t)(at + (long long)kv_head * a.c.rows);  // of the head's row in the pages
      if (!kBits8) {
        if (mine && !is_q) {
          uint4 *to = reinterpret_cast<uint4 *>((is_k ? a.c.k : a.c.v) + place * D * 2);
          to[va] = kv_pack8(x);
          to[vb] = kv_pack8(x + 8);
        }
        continue;
      }
      if (__all_sync(0xffffffffu, is_q)) continue;
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) m = kv_max(m, fabsf(x[j]));
      for (int off = (1 << log_lanes) / 2; off > 0; off >>= 1) m = kv_max(m, __shfl_xor_sync(0xffffffffu, m, off));
      if (!mine || is_q) continue;
      const bool bad = !(m < INFINITY);
      // a power of two that keeps 127 x and the divisor in range (exact)
      const float pre = m > 0x1p100f ? 0x1p-24f : m < 0x1p-80f ? 0x1p40f : 1.0f;
      const float den = m * pre, k = __fdividef(127.0f * pre, den);
      uint2 lo = make_uint2(0u, 0u), hi = lo;
      if (!bad && m > 0.f) {
        lo = kv_codes(x, pre, den, k, m < 0x1p-80f);
        hi = kv_codes(x + 8, pre, den, k, m < 0x1p-80f);
      }
      uint2 *to = reinterpret_cast<uint2 *>((is_k ? a.c.k : a.c.v) + place * D);
      to[va] = lo;
      to[vb] = hi;
      if (me == 0) (is_k ? a.c.ks : a.c.vs)[place] = bad ? NAN : m / 127.0f;
      if (me == 0 && bad) set_error(a.err, kErrNonFinite);
    }
  }
  if (a.trace && tid == 0) trace_max(a.trace, kTrExit);
}

// A block has the rows that its threads take at once; D / 16 threads (of a power of
// two) have a head's key or value, 16 values each.  Small threads, many of them:
// 32768 rows of 8 x 128 in 8 bits took 47 us with two units a thread, 52 with four,
// 39 so (201 MB, 5.2 TB/s); units of 8 values, with twice the look-ups, 75.
template <bool kBits8>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const KvReadArgs a) {
  const int tid = threadIdx.x, row0 = blockIdx.x * a.per, rows = min(a.per, a.T - row0);
  const bool tracer = a.trace && blockIdx.x == 0 && tid == 0;
  if (tracer) trace_min(a.trace, kTrEntry);
  pdl_wait();
  pdl_launch_dependents();
  if (tracer) trace_min(a.trace, kTrWaited);
  const int D = a.c.D, vecs = D / 16, H = a.c.heads, both = a.k && a.v ? 2 : 1, units = rows * both * H;
  const int log_lanes = vecs <= 1 ? 0 : 32 - __clz(vecs - 1), vec = tid & ((1 << log_lanes) - 1);
  const int step = kKvThreads >> log_lanes;
  const float per_row = 1.0f / (float)H;
  if (vec >= vecs) return;
  for (int i = tid >> log_lanes; i < units; i += step) {
    const int r2 = (int)(((float)i + 0.5f) * per_row), head = i - r2 * H;  // (i / H: exact below 2^20)
    const int r = row0 + (both == 2 ? r2 >> 1 : r2);
    const bool is_k = both == 2 ? !(r2 & 1) : a.k != nullptr;
    const int pos = __ldg(a.pos + r);
    if (pos < 0) continue;  // left out
    const long long at = kv_row(a.c, a.seq ? __ldg(a.seq + r) : r, pos);
    uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
    if (at < 0) {
      set_error(a.err, kErrBadId);
    } else {
      const size_t place = (size_t)(at + (long long)head * a.c.rows);
      const uint8_t *from = is_k ? a.c.k : a.c.v;
      if (kBits8) {
        const float s = (is_k ? a.c.ks : a.c.vs)[place];
        const uint4 x = __ldcs(reinterpret_cast<const uint4 *>(from + place * D) + vec);
        const uint32_t c[4] = {x.x ^ 0x80808080u, x.y ^ 0x80808080u, x.z ^ 0x80808080u, x.w ^ 0x80808080u};
        float f[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)  // 2^23 + code + 128, a float; less 2^23 + 128 the code
          f[j] = (__uint_as_float(__byte_perm(c[j / 4], 0x4B000000u, 0x7440u + j % 4)) - 8388736.f) * s;
        lo = kv_pack8(f);
        hi = kv_pack8(f + 8);
      } else {
        lo = __ldcs(reinterpret_cast<const uint4 *>(from + place * D * 2) + 2 * vec);
        hi = __ldcs(reinterpret_cast<const uint4 *>(from + place * D * 2) + 2 * vec + 1);
      }
    }
    uint4 *to = reinterpret_cast<uint4 *>((is_k ? a.k : a.v) + (size_t)r * (is_k ? a.ldk : a.ldv) + head * D) + 2 * vec;
    __stcs(to, lo);
    __stcs(to + 1, hi);
  }
  if (a.trace && tid == 0) trace_max(a.trace, kTrExit);
}
}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs &a0, int n_sm, cudaStream_t st, bool pdl) {
  KvAppendArgs a = a0;
  // Many rows: as many per block as its threads' units take, twice over; few rows:
  // blocks for parts of a row.
  const int pairs = a.c.D / 16, heads = a.Hq + 2 * a.c.heads;
  int lanes = 1;
  while (lanes < pairs) lanes *= 2;
  const int at_once = kKvThreads / lanes;  // head rows
  a.per = 2 * kKvUnits * at_once / heads;
  a.per = a.per < 1 || a.T < 4 * n_sm ? 1 : a.per > kKvMaxBlockRows ? kKvMaxBlockRows : a.per;
  a.parts = 1;
  if (a.T < 4 * n_sm) {
    a.parts = (heads + at_once - 1) / at_once;
    a.parts = (a.parts + kKvUnits - 1) / kKvUnits;
  }
  const unsigned blocks = (unsigned)((a.T + a.per - 1) / a.per) * (unsigned)a.parts;
  return launch_k(a.c.ks ? kv_append_kernel<true> : kv_append_kernel<false>, dim3(blocks), dim3(kKvThreads), 0, st, pdl, a);
}

cudaError_t launch_kv_read(const KvReadArgs &a0, int n_sm, cudaStream_t st, bool pdl) {
  KvReadArgs a = a0;
  int lanes = 1;
  while (lanes < a.c.D / 16) lanes *= 2;
  const int rows = kKvThreads / lanes / ((a.k && a.v ? 2 : 1) * a.c.heads);  // that a block reads at once
  a.per = rows < 1 || a.T < 2 * n_sm ? 1 : rows;
  return launch_k(a.c.ks ? kv_read_kernel<true> : kv_read_kernel<false>, dim3((unsigned)((a.T + a.per - 1) / a.per)),
                  dim3(kKvThreads), 0, st, pdl, a);
}

}  // namespace moe
