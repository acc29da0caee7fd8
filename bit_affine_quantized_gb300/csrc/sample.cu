// A token drawn from each row's logits through temperature, min-p, top-k and
// top-p, from a given random number (moe_sample).
//
// The three filters keep a first part of the tokens in the order of their logits
// (the lower id first of equal ones), so what remains is told by one key: the
// logit as an ordered integer, then the complement of the id.  Nothing is sorted;
// the key is found by histograms, and the token by a running sum over the ids.
//
// A cluster of up to 16 blocks has a row, each block a run of its tokens in
// shared memory, so that every logit is read once.  While the logits land every
// thread takes the maximum of its own; from these maxima alone follow bounds
// below which no token can remain:
//   top-k:  some block has k threads with a maximum above a value, or every block
//           has k / blocks such threads: k tokens lie above it;
//   top-p:  the tokens of less than (1 - p) S / V each have less than (1 - p) S
//           together, for S any lower bound of the sum (here of the maxima).
// The tokens above the bound are few: for a small k they go to the first block's
// list at once, else a histogram of their distance to the maximum (512 bins, a
// count and a sum each, refined by 9 bits where needed) says in which bin the cut
// falls, and a list takes what lies above its lower end, or in the bin alone.  The
// blocks tell each other their bins 16 at a time, then the 16 in question.  A list
// is sorted.  Where a bin cannot be refined (many equal logits) the key is found
// bit by bit, a sweep and two meetings each: rows of 262144 equal logits, top-p 0.5,
// take 393 us for one, 2450 for 64; a few hundred likely tokens, values rounded to
// bf16, 144 for 64 with top-p 0.9 (142 not rounded).
//
// What bounds it: the row's chain of phases (landing, maxima, histogram, two
// meetings, list, sort, the running sum), each 0.5 to 4 us with the SM mostly
// waiting (issue slots 30 % used), times the rounds of clusters; of the logits'
// bytes alone 64 x 262144 would take 10 us.  One row of 262144: top-k 50 11.0 us,
// top-p 0.9 25.2, no filter 13.8; 64 rows: 40, 118, 69; top-p 0.9 of flat rows, of
// which most tokens stay, 209.  What made it (64 x 262144, mixed filters): 64-bit
// floating point in every thread 137 us instead of 105, bins read out of the other
// blocks' memory one by one 105 instead of 85.
//
// Weights e^((l - M) / T) are summed in fixed point, 64 bits: any order, and any
// number of blocks, gives the same sums.  The unit is 2^-34 of a weight of 1 for the
// most tokens, 2^-44 for 262144.  A weight is within 2^-21 of its value before that
// rounding: the argument's rounding errors are carried along (a difference's and a
// product's), what is left is the exponential's.
#include <math.h>

#include "kernels.h"

namespace moe {

namespace {
typedef unsigned long long u64;
constexpr int kSmThreads = 512, kSmWarps = kSmThreads / 32;
constexpr int kSmCluster = kSampleMaxCluster;  // blocks of a row, at most
constexpr int kSmSeg = 22528;        // tokens of a block that leave room for another block on the SM
constexpr int kSmFew = 4096;         // tokens of a block where blocks are plenty: 8 a thread
constexpr int kSmSegMax = 49152;     // that fit shared memory at all; rows of more are read again in every pass
constexpr int kSmChunk = 4096;       // tokens of a bulk copy
constexpr int kSmBins = kSmThreads;  // a thread per bin
constexpr int kSmBits = 27;          // of a token's distance to the maximum: three times 9
constexpr int kSmList = kSmThreads;  // a thread per token of the list
constexpr int kSmSorted = kSmThreads / 4;  // tokens of a short one, which four threads each rank

// Orders floats above -inf as unsigned integers (both zeros the same); 0 for -inf.
__device__ __forceinline__ unsigned sm_key(float f) {
  if (f == -INFINITY) return 0u;
  const unsigned u = __float_as_uint(f + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float sm_value(unsigned k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ u64 sm_full(float f, int id) { return ((u64)sm_key(f) << 32) | (0xFFFFFFFFu - (unsigned)id); }
__device__ __forceinline__ int sm_id(u64 k) { return (int)(0xFFFFFFFFu - (unsigned)k); }

// ---- the other blocks' shared memory
__device__ __forceinline__ uint32_t sm_far(const void *p, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void sm_put(uint32_t at, u64 v) { asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory"); }
__device__ __forceinline__ void sm_put(uint32_t at, u64 a, u64 b) {
  asm volatile("st.shared::cluster.v2.u64 [%0], {%1, %2};" ::"r"(at), "l"(a), "l"(b) : "memory");
}
__device__ __forceinline__ void sm_put(uint32_t at, unsigned v) { asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory"); }
__device__ __forceinline__ void sm_put(uint32_t at, float v) { sm_put(at, __float_as_uint(v)); }
__device__ __forceinline__ unsigned sm_get(uint32_t at) {
  unsigned v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ unsigned sm_count(uint32_t at, unsigned n) {
  unsigned v;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(v) : "r"(at), "r"(n) : "memory");
  return v;
}
// Every thread of the cluster's blocks, which run at the same time.
__device__ __forceinline__ void sm_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void sm_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void sm_meet() {
  sm_arrive();
  sm_wait();
}

struct SmWeight {
  float top, c, c_lo, one;  // the maximum; log2(e) / temperature in two parts; the unit
  __device__ __forceinline__ float units(float l) const {
    const float d = l - top, y = d * c;
    const float b = d - l, e = (l - (d - b)) + (-top - b);        // what the difference lost
    const float lo = fmaf(d, c, -y) + fmaf(d, c_lo, e * c);       // and the product
    float w;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(y));
    return y > -70.f ? fmaf(w, lo * 0.69314718f, w) * one : 0.f;
  }
  __device__ __forceinline__ u64 operator()(float l) const { return __float2ull_rn(units(l)); }
};

__device__ __forceinline__ u64 sm_warp_sum(u64 v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
// Over the 16 lanes of a half warp.
__device__ __forceinline__ u64 sm_half_sum(u64 v) {
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
__device__ __forceinline__ u64 sm_warp_scan(u64 v, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off *= 2) {
    const u64 o = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += o;
  }
  return v;
}

// f * n rounded down, or up, for 0 <= f < 1: exact, in integers (64-bit floating point is scarce on this chip).
__device__ __forceinline__ u64 sm_share(float f, u64 n, bool up) {
  const unsigned b = __float_as_uint(f), e = b >> 23;
  const u64 m = e ? (b & 0x7FFFFFu) | 0x800000u : b & 0x7FFFFFu;  // f = m 2^-shift
  const int shift = 150 - (int)(e ? e : 1u);                        // 24 .. 149
  const u64 lo = m * n, hi = __umul64hi(m, n);
  if (shift >= 128) return up && (lo | hi) ? 1 : 0;
  const u64 q = shift >= 64 ? hi >> (shift - 64) : hi << (64 - shift) | lo >> shift;
  const u64 left = shift >= 64 ? lo | (shift > 64 ? hi & ((1ull << (shift - 64)) - 1) : 0) : lo & ((1ull << shift) - 1);
  return q + (up && left ? 1 : 0);
}

// What a block tells the others of its tokens.
struct SmTold {
  float top, least, cut_all, cut_part, sum, lost;  // lost: 1 where its tokens did not land in time
};
struct __align__(16) SmBin {
  u64 mass, count;
};

// Where a cut falls: the least key that stays, the sum down to it.
struct SmCut {
  u64 key, mass;
};

// kHeld: the block's tokens lie in shared memory.
template <bool kHeld>
__global__ void __launch_bounds__(kSmThreads, kHeld ? 2 : 1) sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) float seg[];
  // The bins, then, when they are read, the lists: the row's (the first block's is used) and the block's own.  A
  // bin's sum is three sums of 16 bits of a weight each (the last of what is left), for shared memory adds 32 bits
  // at once and 64 by trial only; rows that are not held have more tokens than the 16 bits allow for.
  __shared__ __align__(16) unsigned s_space[4][kSmBins];
  unsigned *const s_cnt = s_space[0], (*const s_m)[kSmBins] = s_space + 1;
  u64 *const s_list = reinterpret_cast<u64 *>(s_space[0]), *const s_own_list = reinterpret_cast<u64 *>(s_space[2]);
  static_assert(kSmList * 8 <= 2 * kSmBins * 4, "a list in the place of two of the arrays");
  __shared__ u64 s_mass[kHeld ? 1 : kSmBins], s_warp[kSmWarps], s_far[kSmCluster], s_one[4];
  __shared__ SmBin s_wide[kSmCluster][32], s_fine[kSmCluster][16];  // the blocks' bins: 16 at a time, then one by one
  __shared__ u64 s_sums[2][32];
  __shared__ unsigned s_n, s_own, s_base;
  __shared__ uint64_t s_bar[(kSmSegMax + kSmChunk) / kSmChunk + 1];
  __shared__ float s_red[3][kSmWarps];
  __shared__ SmTold s_told[kSmCluster];
  __shared__ SmCut s_cut;
  __shared__ double s_least;
  __shared__ float s_slope[2], s_low;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = a.cluster, row = blockIdx.x / C, rank = blockIdx.x % C, V = a.V;
  const bool tracer = a.trace && blockIdx.x == 0 && tid == 0;
  if (tracer) trace_min(a.trace, kTrEntry);
  const int per = a.per, n = max(0, min(per, V - rank * per));  // (per: a multiple of 4)
  const float *const from = a.logits + (size_t)row * a.ld + (size_t)rank * per;
  // Place j of the run is token j - skew, so that places of four are 16 bytes in memory as well.
  const int skew = (int)((reinterpret_cast<uintptr_t>(from) >> 2) & 3), id0 = rank * per - skew;
  const int places = (skew + n + 3) & ~3, quads = n > 0 ? places / 4 : 0;
  const int in0 = skew ? 4 : 0, in1 = (skew + n) & ~3;  // whole fours
  const int chunks = kHeld && in1 > in0 ? (in1 + kSmChunk - 1) / kSmChunk : 0;
  if (tid < chunks) mbar_init(&s_bar[tid], 1);
  fence_mbar_init();
  auto clear_bins = [&] {
    s_cnt[tid] = 0u;
    s_m[0][tid] = s_m[1][tid] = s_m[2][tid] = 0u;
    if (!kHeld) s_mass[tid] = 0;
  };
  clear_bins();
  if (tid == 0) s_n = s_own = 0u;
  __syncthreads();
  sm_arrive();  // this block runs; a block that does not run yet has no memory to write to
  pdl_wait();
  pdl_launch_dependents();
  if (tracer) trace_min(a.trace, kTrWaited);
  if (kHeld && tid < chunks) {
    const int j0 = max(in0, tid * kSmChunk), j1 = min(in1, (tid + 1) * kSmChunk);
    mbar_arrive_expect_tx(&s_bar[tid], (uint32_t)(j1 - j0) * 4);
    bulk_g2s(seg + j0, from + (j0 - skew), (uint32_t)(j1 - j0) * 4, &s_bar[tid]);
  }
  if (kHeld && tid >= 32 && tid < 40 && n > 0) {  // the places at the ends that are not whole fours
    const int j = tid < 36 ? tid - 32 : places - 4 + tid - 36;
    if (j < in0 || j >= in1) seg[j] = j >= skew && j < skew + n ? __ldcg(from + (j - skew)) : -INFINITY;
  }
  // the row's filters; a greedy row is one of top-k 1
  const float temp0 = a.temperature ? __ldg(a.temperature + row) : 1.f;
  const bool greedy = !(temp0 > 0.f);
  const float temp = greedy ? 1.f : temp0, given = __ldg(a.uniform + row);
  const float min_p = a.min_p ? fminf(__ldg(a.min_p + row), 1.f) : 0.f;
  const float top_p0 = a.top_p ? __ldg(a.top_p + row) : 1.f;
  int top_k = a.top_k ? __ldg(a.top_k + row) : 0;
  if (greedy || top_p0 <= 0.f) top_k = 1;
  if (top_k <= 0 || top_k >= V) top_k = 0;
  const bool cut_p = top_p0 < 1.f && top_p0 > 0.f;
  const bool has_min = (a.min_p ? __ldg(a.min_p + row) : 0.f) > 0.f;
  const float u = given > 0.f ? given : 0.f;
  if (tid == 64) {  // 64-bit floating point by one thread, while the logits land
    const double slope = fmin(1.4426950408889634 / (double)temp, 3.0e38);
    s_slope[0] = (float)slope;
    s_slope[1] = (float)(slope - (double)(float)slope);
    s_least = has_min ? (double)temp * log((double)min_p) : 0.0;
  }
  SmWeight weight;
  weight.one = __uint_as_float((unsigned)(127 + 31 + __clz(V)) << 23);  // 2^(31 + clz): V weights of 1 stay below 2^63
  __syncthreads();
  weight.c = s_slope[0];
  weight.c_lo = s_slope[1];

  auto quad = [&](int i) {  // four places
    if (kHeld) return reinterpret_cast<const float4 *>(seg)[i];
    const int j = 4 * i;
    float4 f;
    if (j >= in0 && j < in1) {
      f = __ldcg(reinterpret_cast<const float4 *>(from + (j - skew)));
    } else {
      f.x = j >= skew && j < skew + n ? __ldcg(from + (j - skew)) : -INFINITY;
      f.y = j + 1 >= skew && j + 1 < skew + n ? __ldcg(from + (j + 1 - skew)) : -INFINITY;
      f.z = j + 2 >= skew && j + 2 < skew + n ? __ldcg(from + (j + 2 - skew)) : -INFINITY;
      f.w = j + 3 >= skew && j + 3 < skew + n ? __ldcg(from + (j + 3 - skew)) : -INFINITY;
    }
    f.x = f.x < INFINITY ? f.x : -INFINITY;
    f.y = f.y < INFINITY ? f.y : -INFINITY;
    f.z = f.z < INFINITY ? f.z : -INFINITY;
    f.w = f.w < INFINITY ? f.w : -INFINITY;
    return f;
  };

  // ---- the block's largest and least logit, its threads' maxima
  float mine = -INFINITY, least = INFINITY;
  bool bad = false, late = false;
  auto take = [&](float4 f, int i) {
    float *v = &f.x;
    float t = -INFINITY;
    bool odd = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool fine = v[k] < INFINITY;  // NaN and +inf are not for the token
      odd = odd || !fine;
      v[k] = fine ? v[k] : -INFINITY;
      t = fmaxf(t, v[k]);
      least = fminf(least, v[k] > -INFINITY ? v[k] : INFINITY);
    }
    mine = fmaxf(mine, t);
    if (odd) {
      bad = true;
      if (kHeld) reinterpret_cast<float4 *>(seg)[i] = f;
    }
  };
  if (kHeld) {
    for (int q = 0; q < max(chunks, 1); ++q) {
      if (q < chunks && !mbar_wait(&s_bar[q], 0)) {
        late = true;
        break;
      }
      for (int i = q * (kSmChunk / 4) + tid; i < min(quads, (q + 1 < chunks ? q + 1 : 1 << 20) * (kSmChunk / 4)); i += kSmThreads)
        take(reinterpret_cast<const float4 *>(seg)[i], i);
    }
  } else {
    for (int i = tid; i < quads; i += kSmThreads) {
      const int j = 4 * i;
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = j + k >= skew && j + k < skew + n ? __ldcg(from + (j + k - skew)) : -INFINITY;
      take(make_float4(v[0], v[1], v[2], v[3]), i);
    }
  }
  if (bad) set_error(a.err, kErrNonFinite);
  auto block_max = [&](float v, int k) {  // of one value per thread; k: its place
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    if (lane == 0) s_red[k][warp] = v;
  };
  auto of_warps = [&](int k) {
    float v = s_red[k][lane & (kSmWarps - 1)];
#pragma unroll
    for (int off = kSmWarps / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
  };
  block_max(mine, 0);
  block_max(-least, 1);
  block_max(mine > -INFINITY ? -mine : -INFINITY, 2);
  const bool lost = __syncthreads_or(late) != 0;
  if (lost) {  // the copies under way land, or run out too, before the block's memory is anyone's again
    if (tid == 0) set_error(a.err, kErrTimeout);
    for (int q = 0; q < chunks; ++q) mbar_wait(&s_bar[q], 0, 1000000ull);
  }
  const float block_top = of_warps(0), low_max = -of_warps(2);  // (of the threads that have a token)
  {
    SmTold told = {block_top, -of_warps(1), -INFINITY, -INFINITY, 0.f, lost ? 1.f : 0.f};
    const float wide = block_top - low_max;
    if (top_k > 0 && block_top > -INFINITY && wide < 1e37f) {
      // a histogram of the threads' maxima: the values that k, or k / C, of them reach
      const float f = wide > 0.f ? fminf((kSmBins - 1) / wide, 1e30f) : 0.f;
      if (mine > -INFINITY) atomicAdd(&s_cnt[min(kSmBins - 1, (int)((block_top - mine) * f))], 1u);
      __syncthreads();
      unsigned run = s_cnt[tid];
#pragma unroll
      for (int off = 1; off < 32; off *= 2) {
        const unsigned o = __shfl_up_sync(0xffffffffu, run, off);
        if (lane >= off) run += o;
      }
      if (lane == 31) s_warp[warp] = run;
      __syncthreads();
      const unsigned own = s_cnt[tid];
      for (int w = 0; w < warp; ++w) run += (unsigned)s_warp[w];
      // a bin's lower end, and what fp32 may have moved
      const float edge = f > 0.f ? block_top - (tid + 1.01f) / f - 1e-6f * (fabsf(block_top) + wide) : block_top;
      const unsigned part = (unsigned)((top_k + C - 1) / C);
      if (run >= (unsigned)top_k && run - own < (unsigned)top_k) s_one[0] = __float_as_uint(edge);
      if (run >= part && run - own < part) s_one[1] = __float_as_uint(edge);
      if (tid == kSmThreads - 1) s_one[2] = run;
      __syncthreads();
      if (s_one[2] >= (unsigned)top_k) told.cut_all = __uint_as_float((unsigned)s_one[0]);
      if (s_one[2] >= part) told.cut_part = __uint_as_float((unsigned)s_one[1]);
    } else if (cut_p) {
      float e = mine > -INFINITY ? exp2f((mine - block_top) * weight.c) : 0.f;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) e += __shfl_xor_sync(0xffffffffu, e, off);
      __syncthreads();
      if (lane == 0) s_red[0][warp] = e;
      __syncthreads();
      for (int w = 0; w < kSmWarps; ++w) told.sum += s_red[0][w];
    }
    sm_wait();  // the others run (they had the logits' landing to begin in)
    if (tid < C) {
      const uint32_t to = sm_far(&s_told[rank], tid);
      sm_put(to, told.top);
      sm_put(to + 4, told.least);
      sm_put(to + 8, told.cut_all);
      sm_put(to + 12, told.cut_part);
      sm_put(to + 16, told.sum);
      sm_put(to + 20, told.lost);
    }
  }
  sm_meet();
  // ---- what every block knows now
  const SmTold &of = s_told[min(lane, C - 1)];
  auto lanes_max = [&](float v) {
#pragma unroll
    for (int off = kSmCluster / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return __shfl_sync(0xffffffffu, v, 0);
  };
  const float their_top = of.top, top = lanes_max(their_top), bottom = -lanes_max(-of.least);
  const float cut_all = lanes_max(of.cut_all), cut_part = -lanes_max(-of.cut_part);
  if (top == -INFINITY || lanes_max(of.lost) > 0.f) {  // (the same for all blocks: they leave together)
    if (rank == 0 && tid == 0) {
      a.tokens[row] = -1;
      if (a.logprobs) a.logprobs[row] = -INFINITY;
      if (a.trace) trace_max(a.trace, kTrExit);
    }
    return;
  }
  float sum = 1.f;  // a lower bound of the sum (with min-p: of the largest alone, the others may not count)
  if (cut_p && !has_min) {
    sum = lane < C && their_top > -INFINITY ? of.sum * exp2f((their_top - top) * weight.c) : 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  }
  weight.top = top;
  // min-p: the least logit with l - top >= temperature * ln(min_p), in 64 bits
  float low = bottom;
  if (has_min) {
    if (tid == 0) {
      float f = (float)((double)top + s_least);
      f = (double)f - (double)top >= s_least ? f : nextafterf(f, INFINITY);
      const float g = nextafterf(f, -INFINITY);
      s_low = (double)g - (double)top >= s_least ? g : f;
    }
    __syncthreads();
    low = fmaxf(low, s_low);
  }
  const uint32_t first_n = sm_far(&s_n, 0), first_list = sm_far(s_list, 0);

  auto write = [&](u64 key, u64 all) {  // one thread
    const float l = sm_value((unsigned)(key >> 32));
    a.tokens[row] = sm_id(key);
    // (the sum is at least the token's weight: of a part of 1 no more than fp32 holds is lost)
    if (a.logprobs) a.logprobs[row] = greedy ? 0.f : __fdiv_rn(l - top, temp) - logf(__ull2float_rn(all) / weight.one);
  };
  // The running sum that the token's has to reach.
  auto goal_of = [&](u64 all) { return u >= 1.f ? all : min(all, sm_share(u, all, false) + 1); };
  auto value = [&](int j) {  // of place j, 0 .. 4 quads
    if (kHeld) return seg[j];
    const float v = j >= skew && j < skew + n ? __ldcg(from + (j - skew)) : -INFINITY;
    return v < INFINITY ? v : -INFINITY;
  };
  // Quads first, first + step, .. below end: `look` at every value, which says whether it is to go through `make`
  // and what that makes of it through `put`.  A lane goes through its own picks, kPicks at a time: where they are
  // few, a warp's turns are the most that one lane has; where they are many, there is something to overlap.  With `many`
  // a warp of which a lane picks half or more goes through the quads in their order, without a search for the next
  // (64 x 262144 without a filter 67.5 us instead of 70, top-p 0.9 of flat rows, then, 227 instead of 237).
  auto sweep = [&](bool many, int first, int end, int step, auto look, auto make, auto put) {
    constexpr int kPicks = 2;
    for (int i0 = first; i0 < end; i0 += 8 * step) {
      unsigned picks = 0;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int i = i0 + q * step;
        if (i >= end) continue;
        const float4 f = quad(i);
        picks |= ((look(f.x) ? 1u : 0u) | (look(f.y) ? 2u : 0u) | (look(f.z) ? 4u : 0u) | (look(f.w) ? 8u : 0u)) << (4 * q);
      }
      if (many && __any_sync(__activemask(), __popc(picks) >= 16)) {
#pragma unroll 1
        for (int q = 0; q < 8 && picks >> (4 * q); ++q) {
          const float4 f = quad(i0 + q * step);
          const int id = id0 + 4 * (i0 + q * step);
          const decltype(make(0.f, 0)) made[4] = {make(f.x, id), make(f.y, id + 1), make(f.z, id + 2), make(f.w, id + 3)};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (picks >> (4 * q + k) & 1u) put(made[k]);
        }
        continue;
      }
      while (picks) {
        float v[kPicks];
        int id[kPicks];
        bool is[kPicks];
#pragma unroll
        for (int k = 0; k < kPicks; ++k) {  // (none left: the last again, to no avail)
          is[k] = picks != 0u;
          const int b = is[k] ? __ffs(picks) - 1 : 0, j = is[k] ? 4 * (i0 + (b >> 2) * step) + (b & 3) : id[0] - id0;
          picks &= picks - 1u;
          v[k] = value(j);
          id[k] = id0 + j;
        }
        decltype(make(0.f, 0)) made[kPicks];
#pragma unroll
        for (int k = 0; k < kPicks; ++k) made[k] = make(v[k], id[k]);
#pragma unroll
        for (int k = 0; k < kPicks; ++k)
          if (is[k]) put(made[k]);
      }
    }
  };
  // The tokens from `bound` on that `yes` names go to the first block's list, as far as it reaches; s_n there
  // counts them.  (The list's order varies; nothing depends on it.)
  auto gather = [&](float bound, auto yes) {
    sweep(false, tid, quads, kSmThreads, [&](float v) { return v >= bound && v > -INFINITY; },
          [&](float v, int id) -> u64 { return yes(v, id) ? sm_full(v, id) : 0; },
          [&](u64 key) {
            if (key == 0) return;
            const unsigned at = atomicAdd(&s_own, 1u);
            if (at < (unsigned)kSmList) s_own_list[at] = key;
          });
    __syncthreads();
    const unsigned many = s_own;
    if (tid == 0 && many) s_base = sm_count(first_n, many);
    __syncthreads();
    if (tid < many && s_base + tid < (unsigned)kSmList) sm_put(first_list + 8 * (s_base + tid), s_own_list[tid]);
    if (tid == 0) s_own = 0u;
  };
  // Over the block: the sum of one value per thread.
  auto block_sum = [&](u64 v) {
    v = sm_warp_sum(v);
    __syncthreads();
    if (lane == 0) s_warp[warp] = v;
    __syncthreads();
    u64 t = 0;
#pragma unroll
    for (int w = 0; w < kSmWarps; ++w) t += s_warp[w];
    return t;
  };
  // Running sum over the block, of one value per thread.
  auto block_scan = [&](u64 v) {
    const u64 own = sm_warp_scan(v, lane);
    __syncthreads();
    if (lane == 31) s_warp[warp] = own;
    __syncthreads();
    u64 before = 0;
#pragma unroll
    for (int w = 0; w < kSmWarps - 1; ++w) before += w < warp ? s_warp[w] : 0;
    return own + before;
  };
  // Sorts `count` keys, one per thread (0: none), the largest first; s_list is its own to use.  Few by their ranks, four
  // threads to a key; more by sorting each warp's 32 and a search for the place among every other warp's (top-k 50, then
  // the drawn order, of lists of 200 of 262144: 10.9 us a call, with a bitonic network over the block 12.5).
  auto sort = [&](u64 key, int count) {
    if (count <= kSmSorted) {
      __syncthreads();
      s_list[tid] = key;
      __syncthreads();
      const u64 mine = s_list[tid / 4];
      int place = 0;
#pragma unroll 4
      for (int i = tid % 4; i < count; i += 4) place += s_list[i] > mine;
      place += __shfl_xor_sync(0xffffffffu, place, 1);
      place += __shfl_xor_sync(0xffffffffu, place, 2);
      __syncthreads();
      if (tid / 4 < count && tid % 4 == 0) s_list[place] = mine;
      __syncthreads();
      return tid < count ? s_list[tid] : 0;
    }
#pragma unroll
    for (int k = 2; k <= 32; k *= 2)
#pragma unroll
      for (int j = k / 2; j > 0; j /= 2) {
        const u64 other = __shfl_xor_sync(0xffffffffu, key, j);
        const bool larger = ((lane & j) == 0) == ((lane & k) == 0);  // this thread keeps the larger
        key = larger ? (key > other ? key : other) : (key < other ? key : other);
      }
    __syncthreads();
    s_list[tid] = key;
    __syncthreads();
    int place = lane;
#pragma unroll 4
    for (int w = 0; 32 * w < count; ++w) {  // how many of a warp's 32 are larger
      const u64 *run = s_list + 32 * w;
      int n = 0;
#pragma unroll
      for (int step = 16; step > 0; step /= 2) n += run[n + step - 1] > key ? step : 0;
      n += run[n] > key;
      place += w != warp ? n : 0;
    }
    __syncthreads();
    if (key) s_list[place] = key;
    __syncthreads();
    return tid < count ? s_list[tid] : 0;
  };
  // The first block alone: the list has every token that may remain.
  auto finish = [&](int count, int k, u64 all) {
    u64 key = sort(tid < count ? s_list[tid] : 0, count);
    const u64 w = key ? weight(sm_value((unsigned)(key >> 32))) : 0, upto = block_scan(w);
    bool stays = key != 0 && (k == 0 || tid < k);
    if (k > 0) {
      if (tid == min(k, count) - 1) s_one[0] = upto;
      __syncthreads();
      all = s_one[0];
    }
    if (cut_p) stays = stays && (tid == 0 || upto - w < sm_share(top_p0, all, true));
    const int many = __syncthreads_count(stays);  // (a first part of the order)
    if (tid == many - 1) s_one[1] = upto;
    __syncthreads();
    all = s_one[1];
    const u64 goal = goal_of(all);
    key = sort(stays ? key << 32 | key >> 32 : 0, many);  // by the ids
    key = key << 32 | key >> 32;
    const u64 w2 = key ? weight(sm_value((unsigned)(key >> 32))) : 0, run = block_scan(w2);
    if (run >= goal && run - w2 < goal) write(key, all);
  };

  u64 tau = (u64)sm_key(low) << 32;  // what remains: keys from here on
  bool done = false;
  // ---- a small k: every token above the bound to the first block
  float cut_k = fmaxf(low, top_k > 0 ? fmaxf(cut_all, cut_part) : low);
  if (top_k > 0 && top_k <= kSmList / 2) {
    gather(cut_k, [&](float, int) { return true; });
    sm_meet();
    const unsigned count = sm_get(first_n);
    if (count <= (unsigned)kSmList) {
      // the other blocks are done; the first stays while they may look into its memory
      sm_arrive();
      if (rank != 0) return;
      finish((int)count, top_k, 0);
      sm_wait();
      if (tid == 0 && a.trace) trace_max(a.trace, kTrExit);
      return;
    }
    sm_meet();
    if (tid == 0) s_n = 0u;
    sm_meet();
  }

  // Sum over the cluster; every thread of every block calls it.
  auto cluster_sum = [&](u64 v) {
    const u64 t = block_sum(v);
    if (tid < C) sm_put(sm_far(&s_far[rank], tid), t);
    sm_meet();
    u64 all = 0;
    for (int r = 0; r < C; ++r) all += s_far[r];
    sm_meet();
    return all;
  };

  // ---- the cuts, one after the other
  u64 all = 0;  // sum of what remains, where known
  bool known = false;
#pragma unroll 1
  for (int stage = 0; stage < 2 && !done; ++stage) {
    const bool by_count = stage == 0;
    if (by_count ? top_k == 0 : !cut_p) continue;
    // the bound below which nothing remains
    float cut = low;
    bool narrow = false;  // weights below it fit 32 bits
    if (by_count) {
      cut = cut_k;
    } else if (known) {
      cut = fmaxf(low, sm_value((unsigned)(tau >> 32)));
    } else {
      const float least_w = (1.f - top_p0) * 0.99f * sum / (float)V - 1.f / weight.one;  // (what rounding to units may add)
      const float f = top + (log2f(least_w) - 0.01f) / weight.c;
      if (f < top) cut = fmaxf(low, f - 1e-6f * (fabsf(top) + fabsf(f)));
      narrow = f < top && least_w * weight.one < 0x1p31f;
    }
    const float wide = top - cut, scale = wide > 0.f ? fminf((float)((1 << kSmBits) - 256) / wide, 3e38f) : 0.f;
    auto far_of = [&](float v) { return (unsigned)fminf((top - v) * scale, (float)((1 << kSmBits) - 1)); };
    // about the largest and the least value at a distance, and a little over
    auto value_at = [&](unsigned y, float over) {
      const float d = scale > 0.f ? (float)y / scale : 0.f;
      return top - d + over * (1e-6f * (fabsf(top) + d) + 1e-30f);
    };
    const bool by_key = (unsigned)tau != 0u;  // (else tau is a value's first key: values tell)
    auto outside = [&](float v, int id) { return by_key && sm_full(v, id) < tau; };
    unsigned prefix = 0;
    u64 need = by_count ? (u64)top_k : known ? sm_share(top_p0, all, true) : 0;
    u64 above = 0, above_mass = 0;  // what lies above the bin at hand
    bool found = false;
    float lo = cut, hi = INFINITY;  // what the bin at hand may hold, and a little over
#pragma unroll 1
    for (int level = 1; level <= 3 && !found; ++level) {
      const int shift = kSmBits - 9 * level;
      const bool tail = !by_count && !known && level == 1;
      clear_bins();
      __syncthreads();
      // Below the bound each weight is less than the share of one of V in 1 - p.  They are summed as all the others are,
      // for which tokens lie below it follows from how many blocks the row has, and the sum must not: 64 x 262144 with
      // top-p 0.9 and temperature 1 141 us, where fp32 sums of plain exponentials took 131 and were off by 2^-15 at 2^25
      // tokens; with every weight to 64 bits, not 32 where they fit, and within the sweep below, 156.
      u64 rest = 0;
      auto add_below = [&](auto whole) {
        for (int i = tid; i < quads; i += kSmThreads) {
          const float4 f = quad(i);
          const float v[4] = {f.x, f.y, f.z, f.w};
          if (!(fminf(fminf(f.x, f.y), fminf(f.z, f.w)) < cut)) continue;
#pragma unroll
          for (int k = 0; k < 4; ++k) rest += whole(v[k] < cut && v[k] >= low ? weight.units(v[k]) : 0.f);
        }
      };
      if (tail && narrow) add_below([](float w) { return __float2uint_rn(w); });
      if (tail && !narrow) add_below([](float w) -> u64 { return __float2ull_rn(w); });
      sweep(true, tid, quads, kSmThreads,
            [&](float v) {
              return v >= lo && v <= hi;
            },
            [&](float v, int id) {
              const unsigned y = far_of(v) >> shift;
              return SmBin{weight(v), y >> 9 != prefix || outside(v, id) ? (u64)kSmBins : (u64)(y & 511u)};
            },
            [&](const SmBin &b) {  // (the sum and the bin)
              if (b.count == kSmBins) return;
              const u64 w = b.mass;
              atomicAdd(&s_cnt[b.count], 1u);
              if (kHeld) {
                atomicAdd(&s_m[0][b.count], (unsigned)w & 0xFFFFu);
                atomicAdd(&s_m[1][b.count], (unsigned)w >> 16);
                if (w >> 32) atomicAdd(&s_m[2][b.count], (unsigned)(w >> 32));
              } else if (w) {
                atomicAdd(&s_mass[b.count], w);
              }
            });
      if (tail) {
        rest = block_sum(rest);
        if (tid < C) sm_put(sm_far(&s_far[rank], tid), rest);
      }
      __syncthreads();
      // The bin in which the cut falls: every block learns the others' bins 16 at a time, then the 16 that matter.
      auto mass_of = [&](int b) { return kHeld ? s_m[0][b] + ((u64)s_m[1][b] << 16) + ((u64)s_m[2][b] << 32) : s_mass[b]; };
      const int half = tid / 16, peer = tid % 16;
      {
        const u64 cnt = sm_half_sum(s_cnt[tid]), mass = sm_half_sum(mass_of(tid));
        if (peer < C) sm_put(sm_far(&s_wide[rank][half], peer), mass, cnt);
      }
      sm_meet();
      unsigned bin = 0;
      u64 in = 0, in_mass = 0;
      bool few = false;  // fewer remain than are needed
#pragma unroll 1
      for (int part = 0; part < 2; ++part) {
        SmBin b = {0, 0};
        if (peer < C && (part == 0 || half < 16)) b = part == 0 ? s_wide[peer][half] : s_fine[peer][half];
        const u64 m16 = sm_half_sum(b.mass), c16 = sm_half_sum(b.count);
        if (peer == 0) {
          s_sums[0][half] = m16;
          s_sums[1][half] = c16;
        }
        __syncthreads();
        const u64 mass = s_sums[0][lane], cnt = s_sums[1][lane], mr = sm_warp_scan(mass, lane), cr = sm_warp_scan(cnt, lane);
        if (part == 0 && tail) {
          all = __shfl_sync(0xffffffffu, mr, 31);
          for (int r = 0; r < C; ++r) all += s_far[r];
          known = true;
          need = sm_share(top_p0, all, true);
        }
        const unsigned hit = __ballot_sync(0xffffffffu, (by_count ? above + cr : above_mass + mr) >= need);
        few = few || hit == 0u;
        const int at = hit ? __ffs(hit) - 1 : part == 0 ? 31 : 15;  // (few: the last bin, so that all are counted)
        above += __shfl_sync(0xffffffffu, cr - cnt, at);
        above_mass += __shfl_sync(0xffffffffu, mr - mass, at);
        in = __shfl_sync(0xffffffffu, cnt, at);
        in_mass = __shfl_sync(0xffffffffu, mass, at);
        bin = 16 * bin + (unsigned)at;
        if (part == 0) {
          const int f = 16 * at + (half & 15);
          if (half < 16 && peer < C) sm_put(sm_far(&s_fine[rank][half], peer), mass_of(f), (u64)s_cnt[f]);
          sm_meet();
        }
      }
      prefix = prefix << 9 | bin;
      lo = prefix == (1u << (9 * level)) - 1u || !(wide < 1e37f) ? cut : fmaxf(cut, value_at((prefix + 1) << shift, -1.f));
      hi = wide < 1e37f ? value_at(prefix << shift, 1.f) : INFINITY;
      // all that may remain is a list: a short one, or a longer that saves the second cut (400 by top-k, then top-p,
      // 64 x 262144: 77 us instead of 118; but top-p of 64 x 16000 20.2 us with short ones, 21.6 with any)
      if (above + in <= (u64)(by_count && cut_p ? kSmList : kSmSorted)) {
        gather(lo, [&](float v, int id) { return far_of(v) >> shift <= prefix && !outside(v, id); });
        sm_meet();
        if (rank == 0) finish((int)(above + in), by_count ? top_k : 0, all);
        done = found = true;
      } else if (few) {  // all of them stay (by the count alone: a part of the sum is there); the last bin may be empty
        all = above_mass + in_mass;
        known = found = true;
      } else if (in <= (u64)kSmList) {
        gather(lo, [&](float v, int id) { return v <= hi && far_of(v) >> shift == prefix && !outside(v, id); });
        sm_meet();
        if (rank == 0) {
          const u64 key = sort(tid < (int)in ? s_list[tid] : 0, (int)in);
          const u64 w = key ? weight(sm_value((unsigned)(key >> 32))) : 0, upto = block_scan(w), place = tid + 1;
          // the last that stays: the place k, or the one whose sum reaches the share
          const bool last = key != 0 && (by_count ? above + place == (u64)top_k
                                                       : above_mass + upto >= need && above_mass + upto - w < need);
          if (last) {  // (one thread: the bin is the one in which the count, or the sum, passes what is needed)
            for (int r = 0; r < C; ++r) {
              const uint32_t to = sm_far(&s_cut, r);
              sm_put(to, key);
              sm_put(to + 8, above_mass + upto);
            }
          }
          if (tid == 0) s_n = 0u;
        }
        sm_meet();
        tau = s_cut.key;
        if (by_count) {
          all = s_cut.mass;
          known = true;
        }
        found = true;
        __syncthreads();  // (s_cut is free again)
      }
    }
    if (!found) {  // many equal logits: the largest key from which on there is enough, bit by bit
      u64 k = 0;
#pragma unroll 1
      for (int b = 63; b >= 0; --b) {
        const u64 t = k | (1ull << b);
        u64 part = 0;
        if (t > tau) {  // (else everything that remains lies above it, which is enough)
          const float bound = sm_value((unsigned)(t >> 32));
          sweep(false, tid, quads, kSmThreads, [&](float v) { return !(v < bound) && v > -INFINITY; },
                [&](float v, int id) -> u64 { return sm_full(v, id) < t ? 0 : by_count ? 1 : weight(v); },
                [&](u64 w) { part += w; });
          if (cluster_sum(part) >= need) k = t;
        } else {
          k = t;
        }
      }
      tau = max(tau, k);
      if (by_count) {
        u64 part = 0;
        const float bound = sm_value((unsigned)(tau >> 32));
        sweep(false, tid, quads, kSmThreads, [&](float v) { return v >= bound; },
              [&](float v, int id) -> u64 { return sm_full(v, id) >= tau ? weight(v) : 0; }, [&](u64 w) { part += w; });
        all = cluster_sum(part);
        known = true;
      }
    }
  }

  // ---- the token: running sums over blocks, warps, lanes
  if (!done) {
    const float tau_v = sm_value((unsigned)(tau >> 32));
    const bool by_key = (unsigned)tau != 0u;
    const int q0 = (int)((long long)quads * warp / kSmWarps), q1 = (int)((long long)quads * (warp + 1) / kSmWarps);
    auto kept = [&](float v, int id) -> u64 {
      return v >= tau_v && v > -INFINITY && (!by_key || sm_full(v, id) >= tau) ? weight(v) : 0;
    };
    u64 part = 0;
    sweep(true, q0 + lane, q1, 32, [&](float v) { return v >= tau_v && v > -INFINITY; }, kept,
          [&](u64 w) { part += w; });
    const u64 own = block_sum(part);
    if (tid < C) sm_put(sm_far(&s_far[rank], tid), own);
    sm_meet();
    u64 before = 0, whole = 0;
    for (int r = 0; r < C; ++r) {
      if (r < rank) before += s_far[r];
      whole += s_far[r];
    }
    const u64 goal = goal_of(whole);
    if (before < goal && before + own >= goal) {  // it is this block's
      int w = 0;
      while (w < kSmWarps - 1 && before + s_warp[w] < goal) before += s_warp[w++];
      const int end = (int)((long long)quads * (w + 1) / kSmWarps);
      for (int i0 = (int)((long long)quads * w / kSmWarps); i0 < end && before < goal; i0 += kSmThreads) {
        float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (i0 + tid < end) f = quad(i0 + tid);
        const int id = id0 + 4 * (i0 + tid);
        const u64 w4[4] = {kept(f.x, id), kept(f.y, id + 1), kept(f.z, id + 2), kept(f.w, id + 3)};
        const u64 mine4 = w4[0] + w4[1] + w4[2] + w4[3], run = block_scan(mine4);
        u64 at = before + run - mine4;
        if (at < goal && before + run >= goal) {
          const float v[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const bool was = at >= goal;
            at += w4[k];
            if (!was && at >= goal) write(sm_full(v[k], id + k), whole);
          }
        }
#pragma unroll
        for (int k = 0; k < kSmWarps; ++k) before += s_warp[k];
      }
    }
  }
  if (a.trace && tid == 0) trace_max(a.trace, kTrExit);  // (no block looks into another's memory past the last meeting)
}
}  // namespace

// The launch of a row's cluster of `cluster` blocks with `per` tokens each, T rows.
namespace {
void sm_config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute *attr, int T, int cluster, size_t smem) {
  cfg.gridDim = dim3((unsigned)(T * cluster));
  cfg.blockDim = dim3(kSmThreads);
  cfg.dynamicSmemBytes = smem;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
}
size_t sm_bytes(int per) { return (size_t)(per + 8) * 4; }
}  // namespace

cudaError_t sample_set_attributes(int *clusters) {
  const void *k[2] = {(const void *)sample_kernel<true>, (const void *)sample_kernel<false>};
  cudaError_t e;
  for (const void *f : k)
    if ((e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1))) return e;
  if ((e = cudaFuncSetAttribute(k[0], cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm_bytes(kSmSegMax)))) return e;
  for (int c = 1; c <= kSmCluster; ++c) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    sm_config(cfg, attr, 1, c, sm_bytes(kSmSeg));
    if ((e = cudaOccupancyMaxActiveClusters(&clusters[c], sample_kernel<true>, &cfg))) return e;
  }
  return cudaSuccess;
}

// A row's blocks: as many as leave every thread 8 tokens, up to 16, where all rows run
// at once so; with more rows the most with which they still do, or the fewest that
// hold the row two blocks to an SM.  (Of clusters of 16 the device holds 16 at once,
// of clusters of 12 24: 64 x 262144 with mixed filters took 82 us and took 79 so, one
// row 13 with 16 blocks; 17 x 32000 with 16384 tokens a block 21, with 4096 17.)
cudaError_t launch_sample(const SampleArgs &a0, const int *clusters, cudaStream_t st, bool pdl) {
  SampleArgs a = a0;
  const int least = (a.V + kSmSeg - 1) / kSmSeg;
  int c = (a.V + kSmFew - 1) / kSmFew;
  c = c < kSmCluster ? c : kSmCluster;
  while (c > 1 && c > least && clusters[c] < a.T) --c;
  a.cluster = c;
  a.per = ((a.V + c - 1) / c + 3) & ~3;
  const bool held = a.per <= kSmSegMax;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  sm_config(cfg, attr, a.T, c, held ? sm_bytes(a.per) : 0);
  cfg.stream = st;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, held ? sample_kernel<true> : sample_kernel<false>, a);
}

}  // namespace moe
