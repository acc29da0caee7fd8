// Penalties for repeated tokens, sparse biases, a grammar mask and the greedy
// token of the result, in one pass over the logits (moe_logits_process).
// Per row t and token v with logit l, n the times v occurs in the row's
// history after its prompt:
//
//   v anywhere in the history:  l <- l > 0 ? l / repetition : l * repetition
//   n > 0:                      l <- l - frequency * n - presence
//   v in the bias list:         l <- l + bias            (its last entry)
//   v not allowed by the mask:  l <- -inf
//   token = argmax l, ties to the lower id, -1 if nothing is left
//
// A block takes one slice of a row's vocabulary.  It scans the row's whole
// history and counts the tokens of its slice in shared memory (integer
// atomics: the result does not depend on their order), which needs no table
// in global memory and no clearing of one; the history comes from L2 after
// its first reader.  A table word holds the count after the prompt in its low
// 31 bits and "occurs in the prompt" in bit 31.  A second table holds, per
// token of the slice, the number of its last bias entry.
// The blocks of a row merge their best (logit, id) with one 64-bit atomicMax
// each; the last of them writes the token and clears the row's state.
#include <math.h>

#include "kernels.h"

namespace moe {

namespace {
constexpr int kLgThreads = 256;
constexpr unsigned kInPrompt = 0x80000000u;

// Orders finite floats as unsigned integers (larger float, larger key; both
// zeros the same); with the id's complement the lower id of equals wins.
__device__ __forceinline__ unsigned long long lg_key(float f, unsigned id) {
  const unsigned u = __float_as_uint(f + 0.0f);
  const unsigned k = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return ((unsigned long long)k << 32) | (0xFFFFFFFFu - id);
}

struct RowRules {
  float rep, pres, freq;
  const float *bias;  // the row's bias values
};

// One logit through the rules; c, b: its words of the two tables.
__device__ __forceinline__ float lg_apply(float l, unsigned c, unsigned b, bool allowed, const RowRules &r) {
  if (c != 0u) {
    l = l > 0.f ? __fdiv_rn(l, r.rep) : __fmul_rn(l, r.rep);
    const unsigned n = c & ~kInPrompt;
    if (n != 0u) l = __fsub_rn(__fsub_rn(l, __fmul_rn(r.freq, (float)n)), r.pres);
  }
  if (b != 0u) l = __fadd_rn(l, __ldg(r.bias + b - 1));
  return allowed ? l : -INFINITY;
}

template <bool kHist, bool kBias>
__global__ void __launch_bounds__(kLgThreads) logits_kernel(const LogitsArgs a) {
  extern __shared__ __align__(16) unsigned lsm[];
  __shared__ unsigned long long s_best[kLgThreads / 32];
  const int tid = threadIdx.x, t = blockIdx.y, V = a.V;
  const int v0 = blockIdx.x * a.slice, n = min(a.slice, V - v0);
  unsigned *cnt = lsm, *bix = lsm + (kHist ? a.slice : 0);
  const bool tracer = blockIdx.x == 0 && t == 0 && tid == 0;
  if (tracer) trace_min(a.trace, kTrEntry);
  pdl_wait();
  pdl_launch_dependents();
  if (tracer) trace_min(a.trace, kTrWaited);

  bool bad_id = false, bad = false;
  RowRules rr = {1.f, 0.f, 0.f, nullptr};
  if (kHist || kBias) {
    for (int i = tid; i < ((kHist ? a.slice : 0) + (kBias ? a.slice : 0)); i += kLgThreads) lsm[i] = 0u;
    __syncthreads();
  }
  if (kHist) {
    const int len = max(0, min(__ldcg(a.history_len + t), a.history_stride));
    const int p = a.prompt_len ? __ldcg(a.prompt_len + t) : 0;
    const int32_t *hist = a.history + (size_t)t * a.history_stride;
    for (int i = tid; i < len; i += kLgThreads) {
      const int id = __ldcg(hist + i);
      const unsigned d = (unsigned)(id - v0);
      if (d < (unsigned)n) {
        if (i < p)
          atomicOr(cnt + d, kInPrompt);
        else
          atomicAdd(cnt + d, 1u);
      }
      bad_id = bad_id || id < 0 || id >= V;
    }
    if (a.repetition) rr.rep = __ldcg(a.repetition + t);
    if (a.presence) rr.pres = __ldcg(a.presence + t);
    if (a.frequency) rr.freq = __ldcg(a.frequency + t);
  }
  if (kBias) {
    const int len = max(0, min(__ldcg(a.bias_len + t), a.bias_stride));
    const int32_t *ids = a.bias_ids + (size_t)t * a.bias_stride;
    rr.bias = a.bias_values + (size_t)t * a.bias_stride;
    for (int i = tid; i < len; i += kLgThreads) {
      const int id = __ldcg(ids + i);
      const unsigned d = (unsigned)(id - v0);
      if (d < (unsigned)n) atomicMax(bix + d, (unsigned)(i + 1));
      bad_id = bad_id || id < 0 || id >= V;
    }
  }
  if (kHist || kBias) __syncthreads();
  if (bad_id) set_error(a.err, kErrBadId);

  const float *in = a.logits + (size_t)t * a.ld + v0;
  float *out = a.out ? a.out + (size_t)t * a.ld_out + v0 : nullptr;
  const uint32_t *mask = a.mask ? a.mask + (size_t)t * a.mask_stride + (v0 >> 5) : nullptr;
  unsigned long long best = 0ull;
  for (int i = tid; i < n; i += kLgThreads) {
    const bool allowed = !mask || ((__ldcg(mask + (i >> 5)) >> (i & 31)) & 1u);
    const float l = lg_apply(__ldcs(in + i), kHist ? cnt[i] : 0u, kBias ? bix[i] : 0u, allowed, rr);
    if (out) out[i] = l;
    if (l < INFINITY) {  // not NaN, not +inf
      if (l > -INFINITY) best = max(best, lg_key(l, (unsigned)(v0 + i)));
    } else {
      bad = true;
    }
  }
  if (bad) set_error(a.err, kErrNonFinite);
  if (a.tokens) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, off));
    if ((tid & 31) == 0) s_best[tid >> 5] = best;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
      for (int w = 1; w < kLgThreads / 32; ++w) best = max(best, s_best[w]);
      if (best != 0ull) atomicMax(a.best + t, best);
      __threadfence();  // this block's maximum is visible before it takes its ticket
      if (atomicAdd(a.tickets + t, 1u) == gridDim.x - 1) {  // the row's last block
        __threadfence();
        const unsigned long long v = atomicExch(a.best + t, 0ull);
        atomicExch(a.tickets + t, 0u);
        a.tokens[t] = v ? (int32_t)(0xFFFFFFFFu - (unsigned)(v & 0xFFFFFFFFull)) : -1;
      }
    }
  }
  if (tracer) trace_max(a.trace, kTrExit);
}
}  // namespace

cudaError_t launch_logits(const LogitsArgs &a0, cudaStream_t st, bool pdl) {
  LogitsArgs a = a0;
  a.slice = 4096;
  const bool h = a.history != nullptr, b = a.bias_ids != nullptr;
  const dim3 grid((a.V + a.slice - 1) / a.slice, a.T), block(kLgThreads);
  const size_t smem = (size_t)a.slice * 4 * ((h ? 1 : 0) + (b ? 1 : 0));
  if (h && b) return launch_k(logits_kernel<true, true>, grid, block, smem, st, pdl, a);
  if (h) return launch_k(logits_kernel<true, false>, grid, block, smem, st, pdl, a);
  if (b) return launch_k(logits_kernel<false, true>, grid, block, smem, st, pdl, a);
  return launch_k(logits_kernel<false, false>, grid, block, smem, st, pdl, a);
}

}  // namespace moe
