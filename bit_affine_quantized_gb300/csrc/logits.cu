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
// The rows' vocabularies go in segments; a block takes a run of consecutive
// segments.  Per segment it counts the history's tokens in a table in shared
// memory (integer atomics: the result does not depend on their order), so no
// table in global memory has to be kept or cleared; the start of a row's
// history stays in registers over the block's segments.  A table word holds
// the count after the prompt, a bitmap which tokens occur at all.  A second
// table holds, per token of the segment, the number of its last bias entry, a
// second bitmap which tokens have one.  A segment is up to two slices of eight
// tokens per thread: every token of the history is looked at once per segment,
// which at 4096-token segments and as many history tokens was a third of the
// time.  The logits are copied slices ahead into a ring in shared memory
// (cp.async) in which every thread has places of its own, so that tables are
// built while logits are on their way and only a segment's ends need barriers.
// A slice's rules are applied in the ring, to the tokens whose bits are set, by
// the warp that the tokens belong to; the pass over all tokens is free of them.
//
// 64 x 262144 with a history of 4096, 300 biases and a mask: 32 us; the logits
// alone, read and written, 27.6 (134 MB, 20 at the copy rate): the rest are the
// two barriers and the counting per segment.  A ring of three or four slices was
// slower (28.7, 29.1), two blocks of 512 threads per SM gained 0.7 on the logits
// alone and lost 1.3 with the histories, tables read for every token took 36.
// 17 x 100003 with a history of 20000, biases and a mask: 13.7 us.
// The blocks of a row merge their best (logit, id) with one 64-bit atomicMax
// each; the one that adds the row's last segments writes the token and clears
// the row's state.
#include <math.h>

#include <type_traits>

#include "kernels.h"

namespace moe {

namespace {
constexpr int kLgThreads = 1024;
constexpr int kLgGroups = 2;     // groups of four tokens per thread and slice
constexpr int kLgGroup = 4 * kLgThreads;        // tokens that the block's groups of one kind cover
constexpr int kLgSlice = kLgGroups * kLgGroup;
constexpr int kLgRing = 2;       // slices of logits in shared memory
constexpr int kMaskSlice = kLgSlice / 32;       // mask words of a slice
constexpr int kLgSegMax = 2;     // slices per segment, at most
constexpr int kHistRegs = 4;     // history entries per thread that stay in registers

// Orders finite floats as unsigned integers (larger float, larger key; both
// zeros the same); with the id's complement the lower id of equals wins.
__device__ __forceinline__ unsigned long long lg_key(float f, unsigned id) {
  const unsigned u = __float_as_uint(f + 0.0f);
  const unsigned k = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return ((unsigned long long)k << 32) | (0xFFFFFFFFu - id);
}

struct RowRules {
  float rep, pres, freq;
  const float *bias;   // the row's bias values
  const float *first;  // the first of them, one per thread of the block, in shared memory
};

// One logit through the rules; in: it occurs in the history, n times of those
// after the prompt; b: 1 + its bias entry, 0 for none.
__device__ __forceinline__ float lg_apply(float l, bool in, unsigned n, unsigned b, const RowRules &r) {
  if (in) l = l > 0.f ? __fdiv_rn(l, r.rep) : __fmul_rn(l, r.rep);
  if (n != 0u) l = __fsub_rn(__fsub_rn(l, __fmul_rn(r.freq, (float)n)), r.pres);
  if (b != 0u) l = __fadd_rn(l, b <= (unsigned)kLgThreads ? r.first[b - 1] : __ldg(r.bias + b - 1));
  return l;
}

// The larger of two, NaN if one of them is.
__device__ __forceinline__ float lg_max(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ void lg_copy16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void lg_copy4(void *dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void lg_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void lg_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// kQuad: rows start on 16-byte boundaries, and a thread's tokens of a slice are
// four neighbours per group, 4 tid + k + 4096 g; else tid + k threads + 4096 g.
template <bool kHist, bool kBias, bool kMask, bool kQuad>
__global__ void __launch_bounds__(kLgThreads, 1) logits_kernel(const LogitsArgs a) {
  extern __shared__ __align__(16) unsigned lsm[];
  __shared__ unsigned long long s_best[kLgThreads / 32];
  __shared__ float s_first[kBias ? kLgThreads : 1];  // the row's first bias values: from memory each would stall its warp
  const int tid = threadIdx.x, V = a.V;
  constexpr int kStep = kQuad ? 1 : kLgThreads;  // distance of a thread's tokens
  const int own = kQuad ? 4 * tid : tid;         // its first token of a group
  const int seg = a.seg * kLgSlice;
  float *const ring = reinterpret_cast<float *>(lsm) + own;
  unsigned *const cnt = lsm + kLgRing * kLgSlice, *const bix = cnt + (kHist ? seg : 0);
  // a bit per token: it is in the history, it has a bias
  unsigned *const hbits = bix + (kBias ? seg : 0), *const bbits = hbits + (kHist ? seg / 32 : 0);
  // mask words of the slices in the ring, per group four for the 128 tokens of a warp
  uint32_t *const mring = bbits + (kBias ? seg / 32 : 0) + (tid >> 5) * 4;
  constexpr int kMaskGroup = kLgGroup / 32;
  const bool tracer = blockIdx.x == 0 && tid == 0;
  if (tracer) trace_min(a.trace, kTrEntry);
  const int ns = (V + seg - 1) / seg;  // segments per row
  const long long units = (long long)ns * a.T;
  const long long u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
  if (kHist || kBias)
    for (int i = tid; i < ((kHist ? 1 : 0) + (kBias ? 1 : 0)) * (seg + seg / 32) / 4; i += kLgThreads)
      reinterpret_cast<uint4 *>(cnt)[i] = make_uint4(0u, 0u, 0u, 0u);
  pdl_wait();
  pdl_launch_dependents();
  if (tracer) trace_min(a.trace, kTrWaited);

  int t = (int)(u0 / ns), sg = (int)(u0 % ns);
  // Copies run ahead.  cin: this thread's first token of the next slice to
  // copy; cleft: tokens from the slice's start to the row's end; the block's
  // part ends cend tokens before the end of row et.
  const float *cin = a.logits + (size_t)t * a.ld + (size_t)sg * seg + own;
  // lanes 4 g + j < 8 of a warp copy word j of its group g, whose first token is mown
  const int mg = (tid >> 2) & (kLgGroups - 1);
  const int mown = mg * kLgGroup + (kQuad ? (tid & ~31) * 4 + (tid & 3) * 32 : (tid & ~31) + (tid & 3) * kStep);
  const uint32_t *cmask = kMask ? a.mask + (size_t)t * a.mask_stride + ((sg * seg + mown) >> 5) : nullptr;
  int ct = t, cleft = V - sg * seg;
  const int et = (int)((u1 - 1) / ns), cend = max(0, V - ((int)((u1 - 1) % ns) + 1) * seg);
  auto copy_next = [&](int place) {  // the next slice into a place of the ring
    if (ct < et || (ct == et && cleft > cend)) {
      float *to = ring + place * kLgSlice;
#pragma unroll
      for (int g = 0; g < kLgGroups; ++g) {
        if (kQuad && (cleft >= kLgSlice || own + g * kLgGroup + 4 <= cleft)) {
          lg_copy16(to + g * kLgGroup, cin + g * kLgGroup);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (own + g * kLgGroup + k * kStep < cleft) lg_copy4(to + g * kLgGroup + k * kStep, cin + g * kLgGroup + k * kStep);
        }
      }
      cin += kLgSlice;
      if (kMask) {
        if ((tid & 31) < 4 * kLgGroups && mown < cleft)
          lg_copy4(mring + place * kMaskSlice + mg * kMaskGroup + (tid & 3), cmask);
        cmask += kLgSlice / 32;
      }
      cleft -= kLgSlice;
      if (cleft <= 0) {  // the next row
        ++ct;
        cin = a.logits + (size_t)ct * a.ld + own;
        if (kMask) cmask = a.mask + (size_t)ct * a.mask_stride + (mown >> 5);
        cleft = V;
      }
    }
    lg_commit();
  };
#pragma unroll
  for (int i = 0; i < kLgRing - 1; ++i) copy_next(i);  // one slice ahead of the reads

  __shared__ unsigned s_queue[kHist ? kLgThreads / 32 : 1][64];
  bool fresh = true, bad_id = false, bad = false;
  RowRules rr = {1.f, 0.f, 0.f, nullptr, s_first};
  float bw = 0.f;
  int hlen = 0, plen = 0, blen = 0, hv[kHistRegs], bv = 0, done = 0;
  float best = -INFINITY;  // the thread's best of the row so far
  int best_id = 0;
  int place = 0;  // of the slice to read, in the ring
  // Of the warp's tokens of a slice, eight whose rules this lane applies (they
  // are copied and read by the warp's lanes alone).
  const int pg = (tid >> 4) & 1, pk = (tid >> 2) & 3, pb = 8 * (tid & 3);
  const int patch = pg * kLgGroup + (kQuad ? (tid & ~31) * 4 + pk * 32 : pk * kLgThreads + (tid & ~31)) + pb;
  static_assert(kLgGroups == 2, "a warp's 256 tokens of a slice: eight per lane");
  for (long long u = u0; u < u1; ++u) {
    const int v0 = sg * seg, n = min(seg, V - v0);
    // this thread's places of the segment's first slice
    float *out = a.out ? a.out + (size_t)t * a.ld_out + v0 + own : nullptr;
    if (kHist || kBias) {
      const bool begun = fresh;
      const int32_t *hist = a.history + (size_t)t * a.history_stride, *bids = a.bias_ids + (size_t)t * a.bias_stride;
      if (fresh) {  // a row begins: its rules and its lists' first entries (a list's buffer is a stride long whatever its length)
        fresh = false;
        if (kHist) {
          hlen = __ldcg(a.history_len + t);
          plen = a.prompt_len ? __ldcg(a.prompt_len + t) : 0;
          if (a.repetition) rr.rep = __ldcg(a.repetition + t);
          if (a.presence) rr.pres = __ldcg(a.presence + t);
          if (a.frequency) rr.freq = __ldcg(a.frequency + t);
#pragma unroll
          for (int k = 0; k < kHistRegs; ++k)
            hv[k] = tid + k * kLgThreads < a.history_stride ? __ldcg(hist + tid + k * kLgThreads) : 0;
        }
        if (kBias) {
          blen = __ldcg(a.bias_len + t);
          rr.bias = a.bias_values + (size_t)t * a.bias_stride;
          bv = tid < a.bias_stride ? __ldcg(bids + tid) : 0;
          bw = tid < a.bias_stride ? __ldcg(rr.bias + tid) : 0.f;
        }
        hlen = max(0, min(hlen, a.history_stride));
        blen = max(0, min(blen, a.bias_stride));
      }
      __syncthreads();  // every thread is done with the segment before: the tables are clear
      if (kBias && begun) s_first[tid] = bw;
      if (kHist) {
        auto count = [&](unsigned e) {  // a token of the segment, "in the prompt" in bit 31
          const unsigned d = e & 0x7FFFFFFFu;
          if (d == e) atomicAdd(cnt + d, 1u);
          atomicOr(hbits + (d >> 5), 1u << (d & 31u));
        };
#pragma unroll
        for (int k = 0; k < kHistRegs; ++k) {
          const int i = tid + k * kLgThreads;
          const unsigned d = (unsigned)hv[k] - (unsigned)v0;
          if (i < hlen && d < (unsigned)n) count(i < plen ? d | 0x80000000u : d);
          bad_id = bad_id || (i < hlen && (unsigned)hv[k] >= (unsigned)V);
        }
        if (hlen > kHistRegs * kLgThreads) {
          // Few of a longer history's tokens are the segment's.  A warp collects
          // those and counts them 32 at a time: an atomic takes as long for one lane
          // as for all (17 x 100003, history 20000: 13.3 us without, 11.9 so; for the tokens
          // above, which cost no loads, collecting takes longer than it saves).
          const int lane = tid & 31;
          unsigned *const queue = s_queue[tid >> 5];
          int held = 0;
          auto look = [&](int id, int i) {  // (every lane of the warp; past the history: not there)
            const unsigned d = (unsigned)id - (unsigned)v0;
            const bool there = i < hlen, here = there && d < (unsigned)n;
            bad_id = bad_id || (there && (unsigned)id >= (unsigned)V);
            const unsigned m = __ballot_sync(0xffffffffu, here);
            if (here) queue[held + __popc(m & ((1u << lane) - 1u))] = i < plen ? d | 0x80000000u : d;
            held += __popc(m);
            if (held >= 32) {
              __syncwarp();
              count(queue[lane]);
              held -= 32;
              const unsigned e = queue[32 + lane];
              __syncwarp();
              if (lane < held) queue[lane] = e;
            }
          };
          if ((reinterpret_cast<uintptr_t>(hist) & 15u) == 0) {
#pragma unroll 2
            for (int i = kHistRegs * kLgThreads + 4 * tid; i - 4 * lane < hlen; i += 4 * kLgThreads) {
              int4 q = make_int4(0, 0, 0, 0);
              if (i + 3 < a.history_stride) {
                q = __ldcg(reinterpret_cast<const int4 *>(hist + i));
              } else {  // the buffer's last one to three
                if (i < hlen) q.x = __ldcg(hist + i);
                if (i + 1 < hlen) q.y = __ldcg(hist + i + 1);
                if (i + 2 < hlen) q.z = __ldcg(hist + i + 2);
              }
              look(q.x, i);
              look(q.y, i + 1);
              look(q.z, i + 2);
              look(q.w, i + 3);
            }
          } else {
#pragma unroll 4
            for (int i = kHistRegs * kLgThreads + tid; i - lane < hlen; i += kLgThreads)
              look(i < hlen ? __ldcg(hist + i) : 0, i);
          }
          __syncwarp();
          if (lane < held) count(queue[lane]);
        }
      }
      if (kBias) {
        auto enter = [&](int id, int i) {
          const unsigned d = (unsigned)id - (unsigned)v0;
          if (d < (unsigned)n) {
            atomicMax(bix + d, (unsigned)(i + 1));
            atomicOr(bbits + (d >> 5), 1u << (d & 31u));
          }
          bad_id = bad_id || (unsigned)id >= (unsigned)V;
        };
        if (tid < blen) enter(bv, tid);
#pragma unroll 4
        for (int i = kLgThreads + tid; i < blen; i += kLgThreads) enter(__ldcg(bids + i), i);
      }
      __syncthreads();  // the tables are complete
    }
    int v = v0 + own;
    int at = patch;  // this lane's eight, in the segment
    // one slice; `whole`: all its tokens are there, else `left` of them
    auto slice = [&](auto whole, int left) {
      constexpr bool kWhole = decltype(whole)::value;
      copy_next((place + kLgRing - 1) % kLgRing);  // into the place that the thread read last
      lg_wait<kLgRing - 1>();                      // the thread's part of this slice has landed
      if (kMask || kHist || kBias) __syncwarp();   // and its warp's
      if (kHist || kBias) {
        uint8_t *const hb = reinterpret_cast<uint8_t *>(hbits) + (at >> 3), *const bb = reinterpret_cast<uint8_t *>(bbits) + (at >> 3);
        const unsigned in = kHist ? *hb : 0u;
        unsigned todo = in | (kBias ? *bb : 0u);
        if (todo != 0u) {
          if (kHist) *hb = 0;
          if (kBias) *bb = 0;
          float *const lg = reinterpret_cast<float *>(lsm) + place * kLgSlice + patch;
          do {
            const int k = __ffs(todo) - 1;
            todo &= todo - 1u;
            lg[k] = lg_apply(lg[k], in >> k & 1u, kHist ? cnt[at + k] : 0u, kBias ? bix[at + k] : 0u, rr);
            if (kHist) cnt[at + k] = 0u;
            if (kBias) bix[at + k] = 0u;
          } while (todo != 0u);
        }
        at += kLgSlice;
        __syncwarp();
      }
      const uint32_t *words = mring + place * kMaskSlice;
      const float *from = ring + place * kLgSlice;
#pragma unroll
      for (int g = 0; g < kLgGroups; ++g) {
        uint32_t m = 15u;
        if (kMask) {
          if (kQuad) {
            m = words[g * kMaskGroup + ((tid & 31) >> 3)] >> (4 * (tid & 7));
          } else {
            const uint4 w = *reinterpret_cast<const uint4 *>(words + g * kMaskGroup);
            const int i = tid & 31;
            m = ((w.x >> i) & 1u) | (((w.y >> i) & 1u) << 1) | (((w.z >> i) & 1u) << 2) | (((w.w >> i) & 1u) << 3);
          }
        }
        float l[4];
        const float *in = from + g * kLgGroup;
        if (kQuad) {
          const float4 f = *reinterpret_cast<const float4 *>(in);
          l[0] = f.x;
          l[1] = f.y;
          l[2] = f.z;
          l[3] = f.w;
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) l[k] = in[k * kStep];
        }
        if (kMask) {
#pragma unroll
          for (int k = 0; k < 4; ++k) l[k] = m & (1u << k) ? l[k] : -INFINITY;
        }
        float *o = out + g * kLgGroup;
        if (kWhole) {
          if (out) {
            if (kQuad) {
              __stcs(reinterpret_cast<float4 *>(o), make_float4(l[0], l[1], l[2], l[3]));
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) __stcs(o + k * kStep, l[k]);
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const bool there = own + g * kLgGroup + k * kStep < left;
            l[k] = there ? l[k] : -INFINITY;
            if (out && there) __stcs(o + k * kStep, l[k]);
          }
        }
        float top = lg_max(lg_max(l[0], l[1]), lg_max(l[2], l[3]));
        if (!(top < INFINITY)) {  // NaN and +inf are not for the token
          bad = true;
#pragma unroll
          for (int k = 0; k < 4; ++k) l[k] = l[k] < INFINITY ? l[k] : -INFINITY;
          top = lg_max(lg_max(l[0], l[1]), lg_max(l[2], l[3]));
        }
        if (top > best) {
          best = top;
          best_id = v + g * kLgGroup + kStep * (l[0] == top ? 0 : l[1] == top ? 1 : l[2] == top ? 2 : 3);  // the first of them
        }
      }
      if (kMask) __syncwarp();  // every lane has its bits before the place is filled again
      place = (place + 1) % kLgRing;
      if (out) out += kLgSlice;
      v += kLgSlice;
    };
    int left = n;
    for (; left >= kLgSlice; left -= kLgSlice) slice(std::true_type{}, left);
    if (left > 0) slice(std::false_type{}, left);
    ++done;
    if (++sg == ns || u + 1 == u1) {  // the row ends, or the block's part of it
      if (a.tokens) {
        unsigned long long key = best > -INFINITY ? lg_key(best, (unsigned)best_id) : 0ull;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, off));
        if ((tid & 31) == 0) s_best[tid >> 5] = key;
        __syncthreads();
        if (tid < 32) {
          key = s_best[tid];
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, off));
        }
        if (tid == 0) {
          bool last = done == ns;  // the whole row was this block's
          if (!last) {
            if (key != 0ull) atomicMax(a.best + t, key);
            __threadfence();  // this block's maximum is visible before it takes its ticket
            last = atomicAdd(a.tickets + t, (unsigned)done) + done == (unsigned)ns;
            if (last) {
              __threadfence();
              key = atomicExch(a.best + t, 0ull);
              atomicExch(a.tickets + t, 0u);
            }
          }
          if (last) a.tokens[t] = key ? (int32_t)(0xFFFFFFFFu - (unsigned)(key & 0xFFFFFFFFull)) : -1;
        }
        __syncthreads();  // s_best is free again
      }
      best = -INFINITY;
      done = 0;
      sg = 0;
      ++t;
      fresh = true;
    }
  }
  lg_wait<0>();
  if (bad_id) set_error(a.err, kErrBadId);
  if (bad) set_error(a.err, kErrNonFinite);
  if (tid == 0) trace_max(a.trace, kTrExit);
}

size_t lg_smem(bool h, bool b, int seg) {
  return (size_t)kLgSlice * 4 * kLgRing + (size_t)(kLgSlice * 4 + kLgSlice / 8) * seg * ((h ? 1 : 0) + (b ? 1 : 0)) +
         (size_t)kLgRing * kMaskSlice * 4;
}

using LgKernel = void (*)(const LogitsArgs);
template <bool kHist, bool kBias>
LgKernel lg_pick(bool mask, bool quad) {
  if (mask) return quad ? logits_kernel<kHist, kBias, true, true> : logits_kernel<kHist, kBias, true, false>;
  return quad ? logits_kernel<kHist, kBias, false, true> : logits_kernel<kHist, kBias, false, false>;
}
LgKernel lg_kernel(bool h, bool b, bool mask, bool quad) {
  if (h) return b ? lg_pick<true, true>(mask, quad) : lg_pick<true, false>(mask, quad);
  return b ? lg_pick<false, true>(mask, quad) : lg_pick<false, false>(mask, quad);
}
}  // namespace

cudaError_t logits_set_attributes() {
  for (int i = 0; i < 16; ++i) {
    const cudaError_t e = cudaFuncSetAttribute(lg_kernel(i & 1, i & 2, i & 4, i & 8),
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)lg_smem(i & 1, i & 2, kLgSegMax));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_logits(const LogitsArgs &a0, int n_sm, cudaStream_t st, bool pdl) {
  LogitsArgs a = a0;
  const bool h = a.history != nullptr, b = a.bias_ids != nullptr;
  const bool quad = (((uintptr_t)a.logits | (uintptr_t)a.out) & 15u) == 0 && a.ld % 4 == 0 && (!a.out || a.ld_out % 4 == 0);
  // Slices per segment: the fewest slices for the block that has most of them,
  // a segment's own work counted as a quarter of a slice and one per 12000
  // tokens of history.
  const double own = 0.25 + (h ? a.history_stride / 12000.0 : 0.0);
  double least = 0.0;
  long long blocks = 0;
  for (int s = 1; s <= kLgSegMax; s *= 2) {
    const long long segs = ((long long)a.V + (long long)s * kLgSlice - 1) / ((long long)s * kLgSlice) * a.T;
    const long long n = segs < n_sm ? segs : n_sm;
    const double cost = (double)((segs + n - 1) / n) * (s + own);
    if (s == 1 || cost < least) {
      least = cost;
      a.seg = s;
      blocks = n;
    }
  }
  return launch_k(lg_kernel(h, b, a.mask != nullptr, quad), dim3((unsigned)blocks), dim3(kLgThreads), lg_smem(h, b, a.seg), st, pdl, a);
}

}  // namespace moe
