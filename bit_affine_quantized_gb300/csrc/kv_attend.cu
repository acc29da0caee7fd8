// Attention of one new token per sequence over the paged cache (moe_kv_attend).
// Per query head, with z_p = cap(scale q.k_p) over the positions looked at:
//
//   out = sum_p e^(z_p - m) v_p / sum_p e^(z_p - m),  m = max z,  lse = m + log(sum)
//
// in one pass: a running maximum and sum, and the output's sum scaled down when
// the maximum grows.  A block has a query head of a sequence; its warps take
// positions in turn, a lane every 32nd dimension, and join at the end.
#include <math.h>

#include "kernels.h"

namespace moe {

namespace {
constexpr int kAtWarps = 8;

template <bool kBits8>
__global__ void __launch_bounds__(32 * kAtWarps) kv_attend_kernel(const KvAttendArgs a) {
  __shared__ float s_m[kAtWarps], s_l[kAtWarps], s_o[kAtWarps][256];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int seq = blockIdx.x / a.Hq, head = blockIdx.x % a.Hq, D = a.c.D, kv = head / (a.Hq / a.c.heads);
  const bool tracer = a.trace && blockIdx.x == 0 && tid == 0;
  if (tracer) trace_min(a.trace, kTrEntry);
  pdl_wait();
  pdl_launch_dependents();
  if (tracer) trace_min(a.trace, kTrWaited);
  const int len = max(0, min(__ldg(a.lengths + seq), a.c.stride * a.c.rows));
  const int first = a.window ? max(0, len - a.window) : 0;
  float q[8], o[8], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int d = lane + 32 * j;
    q[j] = d < D ? bf16_bits_to_float(a.q[(size_t)seq * a.ldq + (size_t)head * D + d]) : 0.f;
    o[j] = 0.f;
  }
  auto value = [&](const uint8_t *from, const float *scales, size_t place, int d) {
    if (d >= D) return 0.f;
    return kBits8 ? (float)(int8_t)from[place * D + d] * scales[place]
                  : bf16_bits_to_float(reinterpret_cast<const uint16_t *>(from)[place * D + d]);
  };
  bool lost = false;
  for (int p = first + warp; p < len; p += kAtWarps) {
    const long long at = kv_row(a.c, seq, p);
    if (at < 0) {
      lost = true;
      continue;
    }
    const size_t place = (size_t)(at + (long long)kv * a.c.rows);
    float z = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) z = fmaf(q[j], value(a.c.k, a.c.ks, place, lane + 32 * j), z);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
    z *= a.scale;
    if (a.softcap > 0.f) z = a.softcap * tanhf(z / a.softcap);
    const float top = fmaxf(m, z), keep = m > -INFINITY ? expf(m - top) : 0.f, w = z > -INFINITY ? expf(z - top) : z == z ? 0.f : z;
    m = top;
    l = l * keep + w;
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = o[j] * keep + w * value(a.c.v, a.c.vs, place, lane + 32 * j);
  }
  if (lost && lane == 0) set_error(a.err, kErrBadId);
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) s_o[warp][lane + 32 * j] = o[j];
  __syncthreads();
  float top = -INFINITY, sum = 0.f, w[kAtWarps];
  for (int i = 0; i < kAtWarps; ++i) top = fmaxf(top, s_m[i]);
  for (int i = 0; i < kAtWarps; ++i) {
    w[i] = s_m[i] > -INFINITY ? expf(s_m[i] - top) : 0.f;
    sum += w[i] * s_l[i];
  }
  if (tid < D) {
    float v = 0.f;
    for (int i = 0; i < kAtWarps; ++i) v += w[i] * s_o[i][tid];
    a.out[(size_t)seq * a.ldo + (size_t)head * D + tid] = float_to_bf16_bits(sum != 0.f ? v / sum : 0.f);
  }
  if (a.lse && tid == 0) a.lse[(size_t)seq * a.Hq + head] = top + logf(sum);
  if (a.trace && tid == 0) trace_max(a.trace, kTrExit);
}
}  // namespace

size_t kv_attend_ws_bytes(const KvCache &c, int Hq) { return 256; }

cudaError_t launch_kv_attend(const KvAttendArgs &a, int n_sm, cudaStream_t st, bool pdl) {
  return launch_k(a.c.ks ? kv_attend_kernel<true> : kv_attend_kernel<false>, dim3((unsigned)(a.c.n_seqs * a.Hq)),
                  dim3(32 * kAtWarps), 0, st, pdl, a);
}

}  // namespace moe
