// A token drawn from each row's logits through temperature, min-p, top-k and
// top-p, from a given random number (moe_sample).
//
// The three filters keep a first part of the tokens in the order of their logits
// (the lower id first of equal ones), so what remains is told by one key: the
// logit as an ordered integer, then the complement of the id.  The key is found
// bit by bit, a count and a sum over the row for each; the token by bisection
// over the ids.  Sums are of weights in fixed point, 64 bits: whatever their
// order they are the same, and to 2^-34 of a weight or better.
#include <math.h>

#include "kernels.h"

namespace moe {

namespace {
constexpr int kSmThreads = 1024;

// Orders floats above -inf as unsigned integers (both zeros the same), 0 for what does not count.
__device__ __forceinline__ unsigned sm_key(float f) {
  if (!(f < INFINITY) || f == -INFINITY) return 0u;
  const unsigned u = __float_as_uint(f + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float sm_value(unsigned k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

__device__ unsigned long long sm_sum(unsigned long long v) {
  __shared__ unsigned long long s[33];
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned long long t = 0;
    for (int i = 0; i < kSmThreads / 32; ++i) t += s[i];
    s[32] = t;
  }
  __syncthreads();
  return s[32];
}

__global__ void __launch_bounds__(kSmThreads) sample_kernel(const SampleArgs a) {
  __shared__ unsigned long long s_best;
  const int tid = threadIdx.x, row = blockIdx.x;
  const bool tracer = a.trace && row == 0 && tid == 0;
  if (tracer) trace_min(a.trace, kTrEntry);
  if (tid == 0) s_best = 0;
  pdl_wait();
  pdl_launch_dependents();
  if (tracer) trace_min(a.trace, kTrWaited);
  const float *l = a.logits + (size_t)row * a.ld;
  const float temp = a.temperature ? __ldg(a.temperature + row) : 1.f;
  __syncthreads();
  unsigned long long best = 0;
  bool bad = false;
  for (int i = tid; i < a.V; i += kSmThreads) {
    const unsigned k = sm_key(l[i]);
    bad |= !(l[i] < INFINITY);
    if (k) best = max(best, ((unsigned long long)k << 32) | (0xFFFFFFFFu - (unsigned)i));
  }
  atomicMax(&s_best, best);
  if (bad) set_error(a.err, kErrNonFinite);
  __syncthreads();
  best = s_best;
  int token = best ? (int)(0xFFFFFFFFu - (unsigned)best) : -1;
  float logprob = best ? 0.f : -INFINITY;
  if (best && temp > 0.f) {
    const float top = sm_value((unsigned)(best >> 32));
    const double inv = fmin(1.0 / (double)temp, 1e300);
    const double one = (double)(1ull << (__clz(a.V) + 31));  // V weights of 1 stay below 2^63
    auto weight = [&](float f) { return (unsigned long long)__double2ll_rn(exp(((double)f - (double)top) * inv) * one); };
    // full keys; those from `low` on remain
    auto key = [&](int i) {
      const unsigned k = sm_key(l[i]);
      return k ? ((unsigned long long)k << 32) | (0xFFFFFFFFu - (unsigned)i) : 0ull;
    };
    unsigned long long low = 1;
    const float mp = a.min_p ? __ldg(a.min_p + row) : 0.f;
    if (mp > 0.f) {
      const double least = (double)temp * log((double)fminf(mp, 1.f));
      unsigned long long k = ~0ull;
      for (int i = tid; i < a.V; i += kSmThreads)
        if (key(i) && (double)l[i] - (double)top >= least) k = min(k, key(i));
      for (int off = 16; off > 0; off >>= 1) k = min(k, __shfl_xor_sync(0xffffffffu, k, off));
      __shared__ unsigned long long s_low;
      if (tid == 0) s_low = ~0ull;
      __syncthreads();
      if ((tid & 31) == 0) atomicMin(&s_low, k);
      __syncthreads();
      low = s_low;
    }
    const int top_k = a.top_k ? __ldg(a.top_k + row) : 0;
    auto find = [&](auto enough) {  // the largest key whose tokens from it on are enough
      unsigned long long k = 0;
      for (int b = 63; b >= 0; --b) {
        const unsigned long long t = k | (1ull << b);
        if (t <= low || enough(t)) k = t;
      }
      return max(k, low);
    };
    if (top_k > 0)
      low = find([&](unsigned long long t) {
        unsigned long long n = 0;
        for (int i = tid; i < a.V; i += kSmThreads) n += key(i) >= t;
        return sm_sum(n) >= (unsigned long long)top_k;
      });
    auto mass = [&](unsigned long long t, int ids) {
      unsigned long long n = 0;
      for (int i = tid; i < ids; i += kSmThreads)
        if (key(i) >= t) n += weight(l[i]);
      return sm_sum(n);
    };
    const float p = a.top_p ? __ldg(a.top_p + row) : 1.f;
    if (p < 1.f) {
      const double share = (double)p * (double)mass(low, a.V);
      low = find([&](unsigned long long t) { return t <= best && (double)mass(t, a.V) >= share; });
    }
    const float given = __ldg(a.uniform + row);
    const double u = given > 0.f ? (double)given : 0.0, all = (double)mass(low, a.V), goal = u * all;
    int from = 0, to = a.V;  // the running sum is above the goal at `to` ids, not at `from`
    while (to - from > 1) {
      const int mid = from + (to - from) / 2;
      if ((double)mass(low, mid) > goal || (u >= 1.0 && mass(low, mid) == mass(low, a.V)))
        to = mid;
      else
        from = mid;
    }
    token = to - 1;
    logprob = (float)(((double)l[token] - (double)top) * inv - log(all / one));
  }
  if (tid == 0) {
    a.tokens[row] = token;
    if (a.logprobs) a.logprobs[row] = logprob;
    if (a.trace) trace_max(a.trace, kTrExit);
  }
}
}  // namespace

cudaError_t launch_sample(const SampleArgs &a, int n_sm, cudaStream_t st, bool pdl) {
  return launch_k(sample_kernel, dim3((unsigned)a.T), dim3(kSmThreads), 0, st, pdl, a);
}

}  // namespace moe
