// Attention of one new token per sequence over the paged cache (moe_kv_attend).
// Per query head, with z_p = cap(scale q.k_p) over the positions looked at:
//
//   out = sum_p e^(z_p - m) v_p / sum_p e^(z_p - m),  m = max z,  lse = m + log(sum)
//
// in one pass over the keys and values: a running maximum and sum per head, and
// the output's sum scaled down when the maximum grows.
//
// A position's key and value are used once per query head of their group, a few
// products per byte, so memory bounds the call and the work is shared out by
// bytes: the tiles (32 positions of a key head of a sequence, 16 where a tile
// would pass 16 KB) of all sequences and heads form one list, of which every
// block has an even run, and every warp of it an even part, whatever the
// lengths.  A warp works alone: it copies its own tiles (TMA, with the swizzle
// that makes the reads below free of conflicts) into its own places in shared
// memory, stages ahead, and no barrier stands between warps until its run ends.
//
// Within a tile the group's query heads are the eight columns (or twice eight)
// of mma.sync products: S^T = K Q^T with 16 positions as rows, then O^T += V^T P^T
// with 16 dimensions as rows.  The accumulator of the first has positions along
// its rows and heads along its columns; movmatrix turns its 8 x 8 parts into the
// operand of the second, and a lane has the same two heads in both accumulators,
// so maxima, sums and factors need no exchange but the maximum's three shuffles.
//
// 8-bit rows become fp16 operands as they are read: code + 128 in the low bits of
// 1024 is an fp16 number, less 1152 the code itself, exact.  A key's scale goes
// onto its score, in fp32.  A value's scale goes onto its weight, which is rounded
// to fp16: the tiles' largest scale so far gives a power of two that the weights
// are held in units of, times 2^14, so that weights keep 11 bits down to 2^-28 of
// the largest.  Queries are fp16 in units of a power of two per head (exact down
// to 2^-16 of the head's largest value, to 2^-25 of it below).  With a bf16 cache
// queries stay as they are and weights are rounded to bf16.
//
// Weights have 16 bits in the second product because the tensor cores take no more
// of an operand whose other side is a row of the cache as it lies; the sum of the
// weights, which divides, is of fp32 ones.  A weight is off by half a step on its own,
// one up, one down, so an output's error stays below that of its own rounding:
// against 64 bits 1.7e-3 (of the outputs' size) for one sequence of 4096 in bf16 and for
// a window in 8 bits, 1.1e-3 for 23 ragged ones, with weights in fp32 the same to two
// digits.  (The two sides differ by 7e-4 to 1.2e-3: values near a rounding border.)
//
// An item (a sequence's key head) that one warp has whole is written at once.
// Where warps share one, the block joins its warps' parts; where blocks share a long
// one, each leaves a part in the workspace, and the last of them, by a counter,
// joins them in the order of the blocks: the result does not depend on who was last.
//
// What it takes (us of a call in a CUDA graph; 152 blocks):
//   32 sequences of up to 32768, 4 x 128, eight queries a head, 8 bits: 116, 738 MB
//   at 6.4 TB/s; 16 of 32768 in bf16 with pages of 16: 164, 1074 MB at 6.5.
//   64 sequences, window 1024, 8 x 256, 8 bits: 67 (272 MB: 41 at the copy rate): three
//   or four whole items a block, then the slowest warp (3 to 6) and the warps' parts (4).
//   One sequence of 4096, 8 x 256, bf16: 18 (5): lengths and first tiles 2.5, one or
//   two tiles a warp 2.5 to 4, the joins 8.
//   256 sequences of 64, 8 x 128, bf16: 20 (11); 16 of 500, 8 x 64: 7.4 (1.6).
// Tiles of 16 positions for rows of 256 bytes: window 1024 75 us instead of 71; eight
// warps a block: the 32 sequences 140 instead of 120; scores and outputs in one
// chain of products, with their loops' trip counts from the head's size: 146.
#include <math.h>

#include "kernels.h"
#include "tma_maps.h"

namespace moe {

namespace {
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kAtMaxGrid = 192;  // blocks
constexpr int kAtSums = 14;  // 8-bit values' weights are held times 2^14

template <bool kBits8, int kD, int kN>
struct AtShape {
  static constexpr int kBytes = kD * (kBits8 ? 1 : 2);
  static constexpr int kBox = kBytes <= 64 ? 64 : 128;  // bytes of a row in one copy
  static constexpr int kRow = (kBytes + kBox - 1) / kBox * kBox;  // and in shared memory
  static constexpr int kTile = kRow <= 256 ? 32 : 16;  // positions
  static constexpr int kHalf = kTile * kRow;           // bytes of a tile's keys, and of its values
  // Warps: as many as the registers of a lane's share of the outputs allow, for a
  // warp waits out its own products and shuffles (heads of 64 in 8 bits, 47 sequences of 16384: 95 us with 16 warps, 106
  // with 12; with 16 queries a head 126 with 12, 147 with 8; heads of 128 and 16 queries 103 with 8, 119 with 12, spilled).
  static constexpr int kWarps = kN == 1 ? (kD == 64 ? 16 : 12) : (kD == 64 && kBits8 ? 12 : 8);
  static constexpr int kFit = (int)(200 * 1024 / ((size_t)kWarps * 2 * kHalf));
  static constexpr int kStages = kFit > 4 ? 4 : kFit;
  static constexpr int kPart = 16 * kN + kD / 16 * kN * 128;  // floats of a part: maxima, sums, the output's sum
  static constexpr size_t kTiles = (size_t)kWarps * kStages * 2 * kHalf, kParts = (size_t)kWarps * kPart * 4;
  // Parts lie where the tiles lay: those of items left open, and where there is room those of items that ended.
  static constexpr bool kBoth = 2 * kParts <= 200 * 1024;
  static constexpr size_t kAllParts = kBoth ? 2 * kParts : kParts, kRoom = kTiles > kAllParts ? kTiles : kAllParts;
  static constexpr size_t kScales = kBits8 ? (size_t)kWarps * kStages * 2 * kTile * 4 : 0;
  static constexpr size_t kSmem = 1024 + kRoom + kScales;
};

struct AtParams {
  CUtensorMap k, v;  // rows of the pages {D, n_pages * heads * rows}, boxes of kBox bytes by min(rows, kTile) rows
  KvAttendArgs a;
  int heads;         // query heads of an item
  int blocks_of;     // items per key head
};

__device__ __forceinline__ void at_tma(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void at_copy16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void at_prefetch(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void at_ldsm(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void at_ldsm_t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ uint32_t at_turn(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ void at_mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool kBits8>
__device__ __forceinline__ void at_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (kBits8)
    mma_f16(d, a, b0, b1);
  else
    at_mma_bf16(d, a, b0, b1);
}
// Two of the four codes of w (plus 128 each) as fp16: those that the selector names.
template <unsigned kSel>
__device__ __forceinline__ uint32_t at_codes(uint32_t w) {
  const uint32_t u = __byte_perm(w, 0x64646464u, kSel), k = 0x64806480u;  // 1024 + code + 128; 1152
  const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&u), *reinterpret_cast<const __half2 *>(&k));
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t at_bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t at_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float at_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// cap tanh(z / cap) in units of log 2, to 2^-19 of itself whatever the cap (an
// exponent's error is a weight's: one of a part of the cap would be 9 % at a cap of
// 10^6).  With x = z / cap, inv = 1 / cap: below 1/4 the series of tanh to x^9, which
// leaves out 2^-26; from there on 1 - 2 / (e^(2 x) + 1), which is a quarter or more and
// whose terms are within 2^-21.  From infinities +-cap, a NaN stays one.  (16 sequences
// of 32768, 8 x 64, four queries a head, 8 bits: 132 us, with the second form alone 126;
// a vote of the warp, and the series alone where it holds for all, 132.)
__device__ __forceinline__ float at_cap(float z, float inv, float cap) {
  const float x = z * inv, s = x * x;
  float t = fmaf(s, 62.f / 2835.f, -17.f / 315.f);
  t = fmaf(fmaf(fmaf(s, t, 2.f / 15.f), s, -1.f / 3.f), s, 1.f);
  const float far = fmaf(-2.f, __fdividef(1.f, at_exp2(2.f * kLog2e * x) + 1.f), 1.f);
  return fabsf(x) < 0.25f ? z * kLog2e * t : far * cap;
}
// The power of two 2^(e - 127), e in 1 .. 254.
__device__ __forceinline__ float at_pow2(int e) { return __uint_as_float((unsigned)e << 23); }
// Over the eight lanes that hold a column's rows.
__device__ __forceinline__ float at_rows_max(float v) {
#pragma unroll
  for (int off = 4; off < 32; off *= 2) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}
__device__ __forceinline__ float at_rows_sum(float v) {
#pragma unroll
  for (int off = 4; off < 32; off *= 2) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
// e^x of the difference to a maximum, in units of log 2; nothing there yet: 0.
__device__ __forceinline__ float at_keep(float m, float top) { return m == -INFINITY ? 0.f : at_exp2(m - top); }

// A place in the list of tiles.
template <int kTile>
struct AtCursor {
  int seq, len, first, t0, nt, item, tile;
  __device__ __forceinline__ void load(const KvAttendArgs &a) {
    len = max(0, min(__ldg(a.lengths + seq), a.c.stride * a.c.rows));
    first = a.window ? max(0, len - a.window) : 0;
    t0 = first / kTile;
    nt = len > 0 ? (len + kTile - 1) / kTile - t0 : 0;
  }
  __device__ __forceinline__ void next(const KvAttendArgs &a, int items) {
    if (++tile < nt) return;
    tile = 0;
    if (++item < items) return;
    item = 0;
    nt = 0;
    while (nt == 0 && ++seq < a.c.n_seqs) load(a);
  }
};

// What the warps of a block tell each other of their parts.
struct AtWarpParts {
  bool ends;     // an item that began before the warp's run ended within it: its part is in the workspace
  bool open;     // the run ends within an item: its part is in shared memory
  bool began;    // and that item began within the run
  int seq[2], item[2], nt[2];  // of the one that ended, the open one
  unsigned at[2];              // their first tiles
};

template <bool kBits8, int kD, int kN>
__global__ void __launch_bounds__(32 * AtShape<kBits8, kD, kN>::kWarps, 1)
    kv_attend_kernel(const __grid_constant__ AtParams prm) {
  using S = AtShape<kBits8, kD, kN>;
  constexpr int kTile = S::kTile, kWarps = S::kWarps, kStages = S::kStages, kMt = kTile / 16, kSteps = kD / 16;
  constexpr int kThreads = 32 * kWarps, kHeads = 8 * kN;
  extern __shared__ uint8_t at_raw[];
  uint8_t *const sm = at_raw + ((1024 - (smem_addr(at_raw) & 1023)) & 1023);
  float *const s_scales = reinterpret_cast<float *>(sm + S::kRoom);
  __shared__ uint64_t s_keys[kWarps][kStages], s_values[kWarps][kStages];
  __shared__ unsigned s_pre[kThreads + 1], s_sums[kWarps + 1], s_start[kWarps + 1];
  __shared__ AtWarpParts s_parts[kWarps];
  __shared__ __align__(16) float s_m[2 * kWarps][kHeads], s_l[2 * kWarps][kHeads];  // of the warps' parts; then their weights
  __shared__ int s_last[2], s_count[2], s_from[2];
  const KvAttendArgs &a = prm.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int D = a.c.D, steps = D / 16, H = a.c.heads, group = a.Hq / H, items = H * prm.blocks_of;
  const int shift = a.c.log_rows, box = min(a.c.rows, kTile), box_shift = 31 - __clz(box);
  const bool tracer = a.trace && blockIdx.x == 0 && tid == 0;
  if (tracer) trace_min(a.trace, kTrEntry);
  if (lane < kStages) {  // (a warp's own: no other waits on them)
    mbar_init(&s_keys[warp][lane], 1);
    mbar_init(&s_values[warp][lane], 1);
  }
  if (tid == 0) {
    at_prefetch(&prm.k);
    at_prefetch(&prm.v);
  }
  fence_mbar_init();
  pdl_wait();
  pdl_launch_dependents();
  if (tracer) trace_min(a.trace, kTrWaited);

  // ---- the list of tiles: prefix sums over the sequences, up to 32 by every warp, more
  // by chunks of sequences, one per thread
  const int n = a.c.n_seqs, chunk = (n + kThreads - 1) / kThreads;
  static_assert((kKvMaxSeqs + kThreads - 1) / kThreads <= 32, "a warp looks through a chunk at once");
  AtCursor<kTile> cur;
  auto tiles_of = [&](int seq, bool is) {  // and the sequence in the cursor
    cur.seq = seq;
    cur.load(a);
    return is ? (unsigned)cur.nt * items : 0u;
  };
  auto scan = [&](unsigned v) {
#pragma unroll
    for (int off = 1; off < 32; off *= 2) {
      const unsigned o = __shfl_up_sync(0xffffffffu, v, off);
      if (lane >= off) v += o;
    }
    return v;
  };
  unsigned total, mine = 0, run = 0;  // of a lane's sequence, and up to it
  // Parts that blocks share cost 5 us, so items stay whole where that costs less.  An item of kWhole tiles a warp or
  // fewer is no longer to a block than its join, to which the others' idling adds: where all are (fits), each of them
  // has a block, or more of them the even cuts between blocks moved to an item's end (the same cut anywhere, us: 8
  // sequences of up to 100, 4 x 128, 8 bits, 7.7 instead of 13.1; 32 of 1500 in bf16 17.9, 22.9; 128 of 600, 8 x 128,
  // 45, 50; window 1024 of 64, 67, 70; 1000 of up to 1500, 2 x 128, bf16, 167, 172; 4000 of up to 400, 1 x 64, 8 bits, 55,
  // 62; but 57 of 1500, 4 x 128, 8 bits, 27.3 instead of 26.7).  With 8 tiles a warp 23 of up to 1999, 3 x 80, take 16.5
  // instead of 15.4, one of 2000 15.3 instead of 12.4.
  constexpr int kWhole = 4;
  bool fits;
  if (n <= 32) {
    mine = tiles_of(min(lane, n - 1), lane < n);
    run = scan(mine);
    total = __shfl_sync(0xffffffffu, run, 31);
    fits = __all_sync(0xffffffffu, mine <= (unsigned)(kWhole * kWarps * items));
  } else {
    unsigned sum = 0, largest = 0;
    for (int i = tid * chunk; i < min(n, (tid + 1) * chunk); ++i) {
      const unsigned tiles = tiles_of(i, true);
      sum += tiles;
      largest = max(largest, tiles);
    }
    sum = scan(sum);
    if (lane == 31) s_sums[warp + 1] = sum;
    __syncthreads();
    if (warp == 0) {  // over the warps
      const unsigned all = scan(lane > 0 && lane <= kWarps ? s_sums[lane] : 0);
      if (lane <= kWarps) s_sums[lane] = all;
    }
    __syncthreads();
    s_pre[tid + 1] = sum + s_sums[warp];
    if (tid == 0) s_pre[0] = 0;
    fits = __syncthreads_and(largest <= (unsigned)(kWhole * kWarps * items));
    total = s_pre[kThreads];
  }
  // as many blocks as have a tile for each warp
  const int blocks = (int)min((total + kWarps - 1) / kWarps, gridDim.x);
  const bool works = (int)blockIdx.x < blocks;
  const unsigned each = works ? total / blocks : 0, rest = works ? total % blocks : 0;
  auto block_at = [&](int b) { return each * b + rest * b / blocks; };  // first tile of block b
  unsigned bu0 = works ? block_at(blockIdx.x) : 0, bu1 = works ? block_at(blockIdx.x + 1) : 0;
  const bool whole_items = fits && n * items <= (int)gridDim.x;
  if (whole_items) {
    const int s = (int)blockIdx.x / items;
    const unsigned all = n <= 32 ? __shfl_sync(0xffffffffu, mine, s & 31) : s < n ? s_pre[s + 1] - s_pre[s] : 0;
    const unsigned before = n <= 32 ? __shfl_sync(0xffffffffu, run - mine, s & 31) : s < n ? s_pre[s] : 0, nt = all / items;
    bu0 = s < n ? before + (blockIdx.x - s * items) * nt : 0;
    bu1 = s < n ? bu0 + nt : 0;
  }
  // ---- the warp's first tile
  auto locate = [&](unsigned u) {
    int ch = 0;
    unsigned base = 0, m = mine, r = run;
    if (n > 32) {  // the chunk: of which warp, then of which lane
      ch = 32 * __popc(__ballot_sync(0xffffffffu, lane < kWarps && s_sums[min(lane, kWarps - 1) + 1] <= u));
      ch += __popc(__ballot_sync(0xffffffffu, s_pre[ch + lane + 1] <= u));
      m = tiles_of(min(n - 1, ch * chunk + lane), lane < chunk && ch * chunk + lane < n);
      r = scan(m);
      base = s_pre[ch];
    }
    const int who = __popc(__ballot_sync(0xffffffffu, base + r <= u));  // lanes whose sequences end before
    const unsigned left = u - base - __shfl_sync(0xffffffffu, r - m, who);
    cur.seq = (n > 32 ? ch * chunk : 0) + who;
    cur.load(a);
    cur.item = (int)(left / (unsigned)cur.nt);
    cur.tile = (int)(left % (unsigned)cur.nt);
  };
  // Short items stay whole in a warp too, up to kShort tiles, where they have 6 on average and fill all warps, or 2.5: a
  // run that would begin within one begins with the next (256 sequences of 64, 8 x 128: 20 us, cut anywhere 27; 256 of
  // 180 41.5, whole in the block alone 45.5; with few items the other way: 64 of up to 360, 4 x 128, 13.6, and 23 so).
  constexpr int kShort = 8;
  const unsigned many = (unsigned)(items * n);
  const bool is_short = !whole_items && total != 0 && 2ull * total <= (unsigned long long)many * (many >= gridDim.x * kWarps ? 12 : 5);
  auto next_start = [&](unsigned u, int limit) {  // tile u, or the next item's first where u is within one of few
    locate(u);
    return cur.tile != 0 && cur.nt <= limit ? u + (cur.nt - cur.tile) : u;
  };
  const int block_limit = fits ? kWhole * kWarps : kShort;
  if (fits && !whole_items && !is_short) {
    if (warp < 2) {
      const unsigned at = warp == 0 ? bu0 : bu1, to = works && at < total ? next_start(at, block_limit) : at;
      if (lane == 0) s_start[warp] = to;
    }
    __syncthreads();
    bu0 = s_start[0];
    bu1 = s_start[1];
  }
  const unsigned w_each = (bu1 - bu0) / kWarps, w_rest = (bu1 - bu0) % kWarps;
  unsigned u0 = bu0 + w_each * warp + w_rest * warp / kWarps;
  unsigned u1 = bu0 + w_each * (warp + 1) + w_rest * (warp + 1) / kWarps;
  if (is_short) {
    if (warp == kWarps - 1) {  // where the next block begins
      const unsigned end = works && bu1 < total ? next_start(bu1, block_limit) : bu1;
      if (lane == 0) s_start[kWarps] = end;
    }
    const unsigned start = works && u0 < total ? next_start(u0, warp == 0 ? block_limit : kShort) : u0;
    if (lane == 0) s_start[warp] = start;
    __syncthreads();
    u0 = max(start, s_start[0]);  // (the block's own begins with an item that the warps would cut)
    u1 = max(s_start[warp + 1], s_start[0]);
  }
  cur.seq = cur.item = cur.tile = cur.nt = 0;
  if (u0 < u1) locate(u0);
  AtCursor<kTile> is = cur;  // of the next tile to copy

  uint8_t *const tiles = sm + (size_t)warp * kStages * 2 * S::kHalf;
  float *const scales = s_scales + warp * kStages * 2 * kTile;
  const int boxes = kTile / box;
  constexpr int kColumns = S::kRow / S::kBox;  // dimensions from D on are copied as zeros
  const int rows_all = a.c.n_pages * H * a.c.rows;
  constexpr uint32_t kBytes = S::kHalf + (kBits8 ? kTile * 4 : 0);
  bool lost = false, late = false;
  int page = 0, row = 0;        // of the tile at `is`, lane b < boxes its box b
  bool need = false;
  uint32_t there[kStages];      // the stages' boxes that are on pages that are there
  auto look = [&] {             // asks for the pages of the tile at `is`, well ahead of their use
    const int pos = (is.t0 + is.tile) * kTile + lane * box;
    need = lane < boxes && pos < is.len && pos + box > is.first;
    if (need) page = __ldg(a.c.table + (size_t)is.seq * a.c.stride + (pos >> shift));
  };
  auto find = [&] {             // the rows of the tile at `is`; its boxes that are there
    const bool ok = need && (unsigned)page < (unsigned)a.c.n_pages;
    const int pos = (is.t0 + is.tile) * kTile + lane * box;
    lost = lost || (need && !ok);
    row = ok ? (page * H + is.item / prm.blocks_of) * a.c.rows + (pos & (a.c.rows - 1)) : -1;
    return __ballot_sync(0xffffffffu, ok);
  };
  auto copy = [&](const CUtensorMap *map, const float *from, uint64_t *bar, int st, int half) {
    if (lane == 0) mbar_arrive_expect_tx(bar, kBytes);
    __syncwarp();
    if (lane < boxes) {
      uint8_t *to = tiles + (size_t)(2 * st + half) * S::kHalf + lane * box * S::kBox;
      const int y = row >= 0 ? row : rows_all;  // (a box that is not there: past the end, filled with zeros)
#pragma unroll
      for (int i = 0; i < kColumns; ++i)
        at_tma(to + i * kTile * S::kBox, map, i * (S::kBox / (kBits8 ? 1 : 2)), y, bar);
      if (kBits8) bulk_g2s(scales + (2 * st + half) * kTile + lane * box, from + max(row, 0), box * 4, bar);
    }
  };
  auto copy_keys = [&](int st) { copy(&prm.k, a.c.ks, &s_keys[warp][st], st, 0); };
  auto copy_values = [&](int st) { copy(&prm.v, a.c.vs, &s_values[warp][st], st, 1); };
  // Byte in a half of a stage of the 16-byte piece x + y of row r, x even and y 0 or
  // 1, as the copies' swizzle lays it: place(r, y) once, then piece(that, x).
  auto place = [&](int r, int y) { return S::kBox == 128 ? r * 128 + ((y ^ (r & 7)) << 4) : r * 64 + ((y ^ ((r >> 1) & 3)) << 4); };
  auto piece = [&](uint32_t at, int x) { return (at ^ (uint32_t)((x & 7) << 4)) + (uint32_t)((x >> 3) * kTile * 128); };

  const bool capped = a.softcap > 0.f;
  const float most = 3e38f;  // (finite: a score of 0 stays one)
  const float factor = capped ? a.scale : fminf(fmaxf(a.scale * kLog2e, -most), most);
  const float softcap = fminf(a.softcap, 2e38f), cap = softcap * kLog2e, inv = fminf(1.f / softcap, most);  // (in range)
  // ---- state of the item at hand: lane (g, c) has the heads 8 i + 2 c and the one after
  uint32_t q[kSteps][kN][2];
  float m[kN][2], l[kN][2], o[kSteps][kN][4], qs[kN][2];
  int unit = 1;  // 8 bits: values' weights in units of 2^(unit - 127 - kAtSums)
  auto begin = [&] {
    const int kv = cur.item / prm.blocks_of, h0 = kv * group + cur.item % prm.blocks_of * prm.heads;
    const int heads = min(prm.heads, group - cur.item % prm.blocks_of * prm.heads);
    unit = 1;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const uint16_t *from = a.q + (size_t)cur.seq * a.ldq + (size_t)(h0 + 8 * i + g) * D;
      const bool is_there = 8 * i + g < heads;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        q[s][i][0] = q[s][i][1] = 0u;
        if (s < steps && is_there) {
          if (kBits8) {  // the operand's order of k follows the codes' order in a word
            const uint2 w = __ldg(reinterpret_cast<const uint2 *>(from + 16 * s + 4 * c));
            q[s][i][0] = w.x;
            q[s][i][1] = w.y;
          } else {
            q[s][i][0] = __ldg(reinterpret_cast<const uint32_t *>(from + 16 * s + 2 * c));
            q[s][i][1] = __ldg(reinterpret_cast<const uint32_t *>(from + 16 * s + 8 + 2 * c));
          }
        }
      }
      if (kBits8) {
        unsigned top = 0;  // the largest magnitude's bits, over the lanes of a head
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int j = 0; j < 2; ++j) top = max(top, max((q[s][i][j] << 16) & 0x7FFFFFFFu, q[s][i][j] & 0x7FFF0000u));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = min(max((int)(top >> 23), 1), 253);
        const float down = at_pow2(254 - e);
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            q[s][i][j] = at_f16x2(__uint_as_float(q[s][i][j] << 16) * down, __uint_as_float(q[s][i][j] & 0xFFFF0000u) * down);
#pragma unroll
        for (int j = 0; j < 2; ++j)  // (finite, as the factor is)
          qs[i][j] = fminf(fmaxf(at_pow2(__shfl_sync(0xffffffffu, e, 4 * (2 * c + j))) * factor, -most), most);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m[i][j] = -INFINITY;
        l[i][j] = 0.f;
      }
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[s][i][j] = 0.f;
    }
  };
  // The item's output, written whole.
  auto finish = [&] {
    const int kv = cur.item / prm.blocks_of, part = cur.item % prm.blocks_of * prm.heads, h0 = kv * group + part;
    const int heads = min(prm.heads, group - part);
    uint16_t *const out = a.out + (size_t)cur.seq * a.ldo + (size_t)h0 * D;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      float f[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float sum = at_rows_sum(l[i][j]);
        const int h = 8 * i + 2 * c + j;
        if (a.lse && g == 0 && h < heads)
          a.lse[(size_t)cur.seq * a.Hq + h0 + h] = m[i][j] * kLn2 + logf(sum);
        f[j] = sum != 0.f ? (kBits8 ? at_pow2(127 - kAtSums) : 1.f) / sum : 0.f;
      }
      const float up = kBits8 ? at_pow2(unit) : 1.f;
      uint16_t *const to = out + (size_t)(8 * i + g) * D;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        if (s >= steps) continue;
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = kBits8 ? o[s][i][j] * f[j & 1] * up : o[s][i][j] * f[j & 1];
        // turned, a lane has head g and dimensions that lie together
        const uint32_t lo = at_turn(at_bf16x2(v[0], v[1])), hi = at_turn(at_bf16x2(v[2], v[3]));
        if (8 * i + g < heads) {
          if (kBits8) {
            *reinterpret_cast<uint2 *>(to + 16 * s + 4 * c) =
                make_uint2(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
          } else {
            *reinterpret_cast<uint32_t *>(to + 16 * s + 2 * c) = lo;
            *reinterpret_cast<uint32_t *>(to + 16 * s + 8 + 2 * c) = hi;
          }
        }
      }
    }
  };
  // The state as a part: maxima and sums per head, and the output's sum as the lanes hold it.
  auto leave = [&](float *to, int k) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float sum = at_rows_sum(l[i][j]);
        if (g == 0) {
          s_m[k][8 * i + 2 * c + j] = m[i][j];
          s_l[k][8 * i + 2 * c + j] = sum;
        }
      }
      const float up = kBits8 ? at_pow2(unit) : 1.f, down = kBits8 ? at_pow2(127 - kAtSums) : 1.f;
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
        if (s < steps)
          reinterpret_cast<float4 *>(to + 2 * kHeads)[(s * kN + i) * 32 + lane] =
              make_float4(o[s][i][0] * down * up, o[s][i][1] * down * up, o[s][i][2] * down * up, o[s][i][3] * down * up);
    }
  };

  float *const work = reinterpret_cast<float *>(a.work);
  float *const my_end = work + (size_t)(blockIdx.x * kWarps + warp) * S::kPart;      // part of an item that ends in my run
  float *const block_parts = work + (size_t)gridDim.x * kWarps * S::kPart;           // [grid][2]
  if (u0 < u1) {
#pragma unroll
    for (int i = 0; i < kStages; ++i) {
      there[i] = 0;
      if (u0 + i < u1) {
        look();
        there[i] = find();
        copy_keys(i);
        copy_values(i);
        is.next(a, items);
      }
    }
    if (u0 + kStages < u1) look();
  }
  bool ends = false, began = false;
  int st = 0;
  uint32_t phase = 0;
  bool fresh = true;
#pragma unroll 1
  for (unsigned u = u0; u < u1; ++u) {
    if (fresh) {
      began = cur.tile == 0;
      begin();
      fresh = false;
    }
    const bool more = u + kStages < u1;
    const uint32_t keys = smem_addr(tiles + (size_t)st * 2 * S::kHalf), values = keys + S::kHalf;
    const float *ks = scales + st * 2 * kTile, *vs = ks + kTile;
    // which positions count
    const int p0 = (cur.t0 + cur.tile) * kTile;
    uint32_t ok = there[0];
#pragma unroll
    for (int i = 1; i < kStages; ++i) ok = st == i ? there[i] : ok;
    constexpr unsigned kAll = kTile == 32 ? 0xffffffffu : 0xffffu;
    const bool whole = p0 >= cur.first && p0 + kTile <= cur.len && ok == (1u << boxes) - 1u;
    unsigned mask = kAll;
    if (!whole)
      mask = __ballot_sync(0xffffffffu, lane < kTile && p0 + lane >= cur.first && p0 + lane < cur.len &&
                                            (ok >> (lane >> box_shift) & 1u));
    late = __any_sync(0xffffffffu, !mbar_wait(&s_keys[warp][st], phase));
    if (late) break;

    // ---- scores of the tile's positions, in units of log 2 (those that are capped, then)
    float z[kMt][kN][4], y[kN][4];  // (odd steps apart: two chains of products)
#pragma unroll
    for (int t = 0; t < kMt; ++t) {
#pragma unroll
      for (int i = 0; i < kN; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) z[t][i][j] = y[i][j] = 0.f;
      const uint32_t rows = keys + place(16 * t + (lane & 15), lane >> 4);
      if (kBits8) {
#pragma unroll
        for (int s = 0; s < kSteps; s += 2) {
          uint32_t w[4];
          at_ldsm(w, piece(rows, s));
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] ^= 0x80808080u;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x[4] = {at_codes<0x4140>(w[2 * h]), at_codes<0x4140>(w[2 * h + 1]),
                                   at_codes<0x4342>(w[2 * h]), at_codes<0x4342>(w[2 * h + 1])};
#pragma unroll
            for (int i = 0; i < kN; ++i) at_mma<true>(h ? y[i] : z[t][i], x, q[s + h][i][0], q[s + h][i][1]);
          }
        }
      } else {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          uint32_t w[4];
          at_ldsm(w, piece(rows, 2 * s));
#pragma unroll
          for (int i = 0; i < kN; ++i) at_mma<false>(s & 1 ? y[i] : z[t][i], w, q[s][i][0], q[s][i][1]);
        }
      }
      const float f[2] = {kBits8 ? ks[16 * t + g] : factor, kBits8 ? ks[16 * t + 8 + g] : factor};
#pragma unroll
      for (int i = 0; i < kN; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          z[t][i][j] = (z[t][i][j] + y[i][j]) * f[j >> 1];
          if (kBits8) z[t][i][j] *= qs[i][j & 1];
        }
    }
    if (capped) {
#pragma unroll
      for (int t = 0; t < kMt; ++t)
#pragma unroll
        for (int i = 0; i < kN; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) z[t][i][j] = at_cap(z[t][i][j], inv, cap);
    }
    if (!whole) {
#pragma unroll
      for (int t = 0; t < kMt; ++t)
#pragma unroll
        for (int i = 0; i < kN; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (!(mask >> (16 * t + 8 * (j >> 1) + g) & 1u)) z[t][i][j] = -INFINITY;
    }
    __syncwarp();  // every lane has read the keys
    if (more) {
      const uint32_t boxes_there = find();
#pragma unroll
      for (int i = 0; i < kStages; ++i) there[i] = st == i ? boxes_there : there[i];
      copy_keys(st);
    }
    // ---- weights
    float up[kN][2], top[kN][2];
    bool grows = false;
#pragma unroll
    for (int i = 0; i < kN; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float v = m[i][j];
#pragma unroll
        for (int t = 0; t < kMt; ++t) v = fmaxf(v, fmaxf(z[t][i][j], z[t][i][j + 2]));
        v = at_rows_max(v);
        grows = grows || v != m[i][j];
        top[i][j] = v == -INFINITY ? 0.f : v;
        up[i][j] = at_keep(m[i][j], top[i][j]);
        m[i][j] = v;
      }
    late = __any_sync(0xffffffffu, !mbar_wait(&s_values[warp][st], phase));
    if (late) break;
    int e = unit;
    if (kBits8) {
      const unsigned most = __reduce_max_sync(
          0xffffffffu, mask >> lane & 1u ? __float_as_uint(vs[lane & (kTile - 1)]) & 0x7FFFFFFFu : 0u);
      e = max(e, min((int)(most >> 23), 253));
    }
    if (__any_sync(0xffffffffu, grows) || e != unit) {
      const float less = kBits8 && e > unit ? (e - unit < 127 ? at_pow2(127 + unit - e) : 0.f) : 1.f;
      unit = e;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        l[i][0] *= up[i][0];
        l[i][1] *= up[i][1];
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[s][i][j] *= kBits8 ? up[i][j & 1] * less : up[i][j & 1];
      }
    }
    // ---- the output's sum
    const float per = kBits8 ? at_pow2(254 - unit) : 1.f;
#pragma unroll
    for (int t = 0; t < kMt; ++t) {
      uint32_t p[kN][2];
      float f[2] = {1.f, 1.f};
      if (kBits8) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = 16 * t + 8 * j + g;
          f[j] = whole || (mask >> r & 1u) ? vs[r] * per * (float)(1 << kAtSums) : 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        float w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          w[j] = at_exp2(z[t][i][j] - top[i][j & 1]);
          l[i][j & 1] += w[j];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
          p[i][j] = at_turn(kBits8 ? at_f16x2(w[2 * j] * f[j], w[2 * j + 1] * f[j]) : at_bf16x2(w[2 * j], w[2 * j + 1]));
      }
      if (kBits8) {
        const uint32_t rows = values + place(16 * t + (lane & 15), lane >> 4);
#pragma unroll
        for (int s = 0; s < kSteps; s += 2) {
          uint32_t w[4];
          at_ldsm_t(w, piece(rows, s));
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] ^= 0x80808080u;
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // rows g and g + 8 of the product are dimensions 2 g and 2 g + 1
            const uint32_t x[4] = {at_codes<0x4240>(w[2 * h]), at_codes<0x4341>(w[2 * h]),
                                   at_codes<0x4240>(w[2 * h + 1]), at_codes<0x4341>(w[2 * h + 1])};
#pragma unroll
            for (int i = 0; i < kN; ++i) at_mma<true>(o[s + h][i], x, p[i][0], p[i][1]);
          }
        }
      } else {
        const uint32_t rows = values + place(16 * t + (lane & 7) + 8 * (lane >> 4), lane >> 3 & 1);
        uint32_t keep[2] = {~0u, ~0u};  // rows that do not count may hold anything: nothing of them is multiplied
        if (!whole) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const unsigned b = mask >> (16 * t + 8 * j + 2 * c);
            keep[j] = (b & 1u ? 0xFFFFu : 0u) | (b & 2u ? 0xFFFF0000u : 0u);
          }
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          uint32_t w[4];
          at_ldsm_t(w, piece(rows, 2 * s));
          if (!whole) {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] &= keep[j >> 1];
          }
#pragma unroll
          for (int i = 0; i < kN; ++i) at_mma<false>(o[s][i], w, p[i][0], p[i][1]);
        }
      }
    }
    __syncwarp();  // every lane has read the values
    if (more) {
      copy_values(st);
      is.next(a, items);
      if (u + kStages + 1 < u1) look();
    }
    if (++st == kStages) {
      st = 0;
      phase ^= 1u;
    }
    if (cur.tile + 1 == cur.nt) {
      fresh = true;
      if (began) {
        finish();
      } else {
        leave(my_end, 2 * warp);
        ends = true;
        if (lane == 0) {
          AtWarpParts &p = s_parts[warp];
          p.seq[0] = cur.seq;
          p.item[0] = cur.item;
          p.nt[0] = cur.nt;
          p.at[0] = u + 1 - (unsigned)cur.nt;
        }
      }
    }
    if (u + 1 < u1) cur.next(a, items);
  }
  if (lane < boxes && lost) set_error(a.err, kErrBadId);
  if (late) {  // the copies under way land, or run out too, before the warp's memory is anyone's again
    if (lane == 0) set_error(a.err, kErrTimeout);
    for (int i = 0; i < 4 * kStages; ++i)
      mbar_wait(i & 1 ? &s_values[warp][i / 4] : &s_keys[warp][i / 4], i >> 1 & 1, 1000000ull);
  }

  // ---- the block's warps join their parts
  const bool open = u0 < u1 && !fresh && !late;
  if (lane == 0) {
    AtWarpParts &p = s_parts[warp];
    p.ends = ends;
    p.open = open;
    p.began = began;
    p.seq[1] = cur.seq;
    p.item[1] = cur.item;
    p.nt[1] = cur.nt;
    p.at[1] = u1 - 1 - (unsigned)cur.tile;
  }
  // the tiles are read: parts take their places.  After a wait that ran out nothing is joined (the error tells).
  const bool joins = !__syncthreads_or(late);
  float *const s_open = reinterpret_cast<float *>(sm);
  if (open && joins) leave(s_open + (size_t)warp * S::kPart, 2 * warp + 1);
  __syncthreads();
  // An item's output in bf16, from the sums of a part (divided already) in shared memory.
  auto write_out = [&](int seq, int item, const float *p) {
    const int first = item % prm.blocks_of * prm.heads, heads = min(prm.heads, group - first);
    uint16_t *const out = a.out + (size_t)seq * a.ldo + (size_t)(item / prm.blocks_of * group + first) * D;
    for (int i = 2 * tid; i < heads * D; i += 2 * kThreads) {
      const int h = i / D, d = i % D, r = d & 15;
      const float *f = p + 2 * kHeads + ((d >> 4) * kN + (h >> 3)) * 128 + ((h & 7) >> 1) * 4 + (h & 1);
      // rows g and g + 8 of a product: dimensions 2 g and 2 g + 1 in 8 bits, else g and g + 8
      const float lo = kBits8 ? f[(r >> 1) * 16] : f[(r & 7) * 16 + (r >> 3) * 2];
      const float hi = kBits8 ? f[(r >> 1) * 16 + 2] : f[((r & 7) + 1) * 16 + (r >> 3) * 2];
      *reinterpret_cast<uint32_t *>(out + i) = at_bf16x2(lo, hi);
    }
  };
  auto write_lse = [&](int seq, int item, int h, float top, float sum) {
    const int part = item % prm.blocks_of * prm.heads, heads = min(prm.heads, group - part);
    if (a.lse && h < heads)
      a.lse[(size_t)seq * a.Hq + item / prm.blocks_of * group + part + h] = top * kLn2 + logf(sum);
  };
  const int slots = steps * kN * 32;
  float *const block_part0 = block_parts + (size_t)(2 * blockIdx.x) * S::kPart, *const block_part1 = block_part0 + S::kPart;
  // The parts in their order are, per warp, 2 w: one that ends an item, 2 w + 1: one
  // of an item left open; a run of parts up to one that ends, or to the last, is of
  // one item.  It was begun in this block if one of them was.
  static_assert(2 * kWarps <= 32, "a lane per part");
  const AtWarpParts &lp = s_parts[min(lane / 2, kWarps - 1)];
  const bool counts = joins && lane < 2 * kWarps;
  const uint32_t ends_at = __ballot_sync(0xffffffffu, counts && !(lane & 1) && lp.ends);
  const uint32_t open_at = __ballot_sync(0xffffffffu, counts && (lane & 1) && lp.open);
  const uint32_t began_at = __ballot_sync(0xffffffffu, counts && (lane & 1) && lp.open && lp.began);
  const uint32_t all_at = ends_at | open_at;
  auto run_of = [&](int k) {  // the parts of part k's item
    const uint32_t before = ends_at & ((1u << k) - 1u), from = ends_at >> k << k;
    const uint32_t to = from ? (from & -from) : 0x80000000u;  // the one that ends it, or the last
    return (to | (to - 1u)) & (before ? ~((2u << (31 - __clz(before))) - 1u) : ~0u);
  };
  const uint32_t first_run = run_of(0);
  const bool last_open = open_at > ends_at;  // (the highest of the parts)
  const uint32_t last_run = last_open ? run_of(31 - __clz(all_at)) : 0u;
  // of items that other blocks share: the first, not begun here; the last, begun here and open
  const bool first_part = (first_run & all_at) && !(first_run & began_at), last_part = (last_run & began_at) != 0u;
  if (all_at != 0u) {
    float *const s_ends = s_open + kWarps * S::kPart;
    if (S::kBoth) {  // the parts in the workspace, on their way while the weights are worked out
#pragma unroll 1
      for (uint32_t left = ends_at; left; left &= left - 1u) {
        const size_t at = (size_t)((__ffs(left) - 1) / 2) * S::kPart + 2 * kHeads;
        for (int slot = tid; slot < slots; slot += kThreads)
          at_copy16(s_ends + at + 4 * slot, work + (size_t)(blockIdx.x * kWarps) * S::kPart + at + 4 * slot);
      }
    }
    if (joins) {
#pragma unroll 1
      for (int h = warp; h < kHeads; h += kWarps) {  // the parts' weights, with 1 / sum where the item ends here
        const uint32_t run = run_of(lane);
        const int from = __ffs(run) - 1, to = 31 - __clz(run);
        const bool is_there = all_at >> lane & 1u, ended = ends_at >> to & 1u, here = (run & began_at) != 0u;
        const float mine = is_there ? s_m[min(lane, 2 * kWarps - 1)][h] : -INFINITY;
        float top = mine;
#pragma unroll
        for (int off = 1; off < 32; off *= 2) {
          const float o = __shfl_down_sync(0xffffffffu, top, off);
          if (lane + off <= to) top = fmaxf(top, o);
        }
        top = __shfl_sync(0xffffffffu, top, from);
        float w = at_keep(mine, top == -INFINITY ? 0.f : top), sum = is_there ? w * s_l[min(lane, 2 * kWarps - 1)][h] : 0.f;
#pragma unroll
        for (int off = 1; off < 32; off *= 2) {
          const float o = __shfl_down_sync(0xffffffffu, sum, off);
          if (lane + off <= to) sum += o;
        }
        sum = __shfl_sync(0xffffffffu, sum, from);
        if (ended && here) w *= sum != 0.f ? 1.f / sum : 0.f;
        if (is_there) s_m[lane][h] = w;
        if (lane == from && (run & all_at)) {
          if (ended && here) {
            write_lse(s_parts[to / 2].seq[0], s_parts[to / 2].item[0], h, top, sum);
          } else {
            float *const part = here ? block_part1 : block_part0;
            part[h] = top;
            part[kHeads + h] = sum;
          }
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
#pragma unroll 1
    for (int slot = tid; slot < slots; slot += kThreads) {
      const int h = 8 * (slot / 32 % kN) + 2 * (slot & 3);
#pragma unroll 1
      for (uint32_t left = all_at; left;) {
        const uint32_t run = run_of(__ffs(left) - 1) & all_at;
        left &= ~run;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (uint32_t m = run; m; m &= m - 1u) {
          const int k = __ffs(m) - 1, w = k / 2;
          const float *const in = (k & 1 ? s_open : s_ends) + (size_t)w * S::kPart + 2 * kHeads;
          const float *const ws = work + (size_t)(blockIdx.x * kWarps + w) * S::kPart + 2 * kHeads;
          const float4 f = (k & 1) || S::kBoth ? reinterpret_cast<const float4 *>(in)[slot]
                                               : __ldcg(reinterpret_cast<const float4 *>(ws) + slot);
          const float2 w2 = *reinterpret_cast<const float2 *>(&s_m[k][h]);
          v.x = fmaf(f.x, w2.x, v.x);
          v.y = fmaf(f.y, w2.y, v.y);
          v.z = fmaf(f.z, w2.x, v.z);
          v.w = fmaf(f.w, w2.y, v.w);
        }
        // an item that began and ends here: to its last open part's place
        const bool here = (run & began_at) != 0u, ended = (run & ends_at) != 0u;
        float *const to = !here ? block_part0 : ended ? s_open + (size_t)((31 - __clz(run & open_at)) / 2) * S::kPart : block_part1;
        reinterpret_cast<float4 *>(to + 2 * kHeads)[slot] = v;
      }
    }
    __syncthreads();
#pragma unroll 1
    for (uint32_t left = ends_at; left; left &= left - 1u) {  // items that warps shared and that began and ended here
      const int k = __ffs(left) - 1;
      const uint32_t run = run_of(k);
      if (run & began_at)
        write_out(s_parts[k / 2].seq[0], s_parts[k / 2].item[0], s_open + (size_t)((31 - __clz(run & open_at)) / 2) * S::kPart);
    }

    // ---- the last block of an item joins the blocks' parts
    if (first_part || last_part) {  // (the same for every thread)
      __threadfence();
      __syncthreads();
      const int first_k = 31 - __clz(first_run & all_at), last_k = 31 - __clz(last_run & all_at);  // a part that tells the item
      if (tid < 2) {
        s_last[tid] = 0;
        if (tid == 0 ? first_part : last_part) {
          const int k = tid == 0 ? first_k : last_k;
          const AtWarpParts &p = s_parts[k / 2];
          // the blocks of its first and its last tile: the largest b with total * b / blocks <= tile
          auto of = [&](unsigned t) { return (int)((((unsigned long long)t + 1) * (unsigned)blocks - 1) / total); };
          const int from = of(p.at[k & 1]), count = of(p.at[k & 1] + (unsigned)p.nt[k & 1] - 1) - from + 1;
          s_from[tid] = from;
          s_count[tid] = count;
          if (atomicAdd(a.tickets + from, 1u) + 1u == (unsigned)count) {
            __threadfence();
            a.tickets[from] = 0u;
            s_last[tid] = 1;
          }
        }
      }
      __syncthreads();
#pragma unroll 1
      for (int which = 0; which < 2; ++which) {
        if (!s_last[which]) continue;
        const int n_parts = s_count[which], f = s_from[which];
        // the parts' maxima, then weights, and sums; 1 / sum; the output's sum
        float *const s_stat = reinterpret_cast<float *>(sm), *const s_sum = s_stat + n_parts * 2 * kHeads;
        float *const s_out = s_sum + 2 * kHeads;
        auto part = [&](int b) { return block_parts + (size_t)(2 * (f + b) + (b == 0 ? 1 : 0)) * S::kPart; };
        const AtWarpParts &p = s_parts[(which ? last_k : first_k) / 2];
        const int o = (which ? last_k : first_k) & 1;
        // sixteen parts' share of a slot at a time, the first of them before the weights are known
        constexpr int kAhead = 16;
        float4 v[kAhead];
        auto fetch = [&](int slot, int b0) {
#pragma unroll
          for (int i = 0; i < kAhead; ++i)
            if (b0 + i < n_parts) v[i] = __ldcg(reinterpret_cast<const float4 *>(part(b0 + i) + 2 * kHeads) + slot);
        };
        __syncthreads();
        for (int i = tid; i < n_parts * 2 * kHeads; i += kThreads) s_stat[i] = __ldcg(part(i / (2 * kHeads)) + i % (2 * kHeads));
        if (tid < slots) fetch(tid, 0);
        __syncthreads();
#pragma unroll 1
        for (int h = warp; h < kHeads; h += kWarps) {
          float top = -INFINITY, sum = 0.f;
          for (int b = lane; b < n_parts; b += 32) top = fmaxf(top, s_stat[b * 2 * kHeads + h]);
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
          const float use = top == -INFINITY ? 0.f : top;
          for (int b = lane; b < n_parts; b += 32) {
            const float w = at_keep(s_stat[b * 2 * kHeads + h], use);
            s_stat[b * 2 * kHeads + h] = w;
            sum += w * s_stat[b * 2 * kHeads + kHeads + h];
          }
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
          if (lane == 0) {
            s_sum[h] = sum != 0.f ? 1.f / sum : 0.f;
            write_lse(p.seq[o], p.item[o], h, top, sum);
          }
        }
        __syncthreads();
#pragma unroll 1
        for (int slot = tid; slot < slots; slot += kThreads) {
          const int h = 8 * (slot / 32 % kN) + 2 * (slot & 3);
          float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
          for (int b0 = 0; b0 < n_parts; b0 += kAhead) {
            if (slot != tid || b0 != 0) fetch(slot, b0);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
              if (b0 + i >= n_parts) continue;
              const float2 w = *reinterpret_cast<const float2 *>(s_stat + (b0 + i) * 2 * kHeads + h);
              t.x = fmaf(v[i].x, w.x, t.x);
              t.y = fmaf(v[i].y, w.y, t.y);
              t.z = fmaf(v[i].z, w.x, t.z);
              t.w = fmaf(v[i].w, w.y, t.w);
            }
          }
          const float f0 = s_sum[h], f1 = s_sum[h + 1];
          reinterpret_cast<float4 *>(s_out + 2 * kHeads)[slot] = make_float4(t.x * f0, t.y * f1, t.z * f0, t.w * f1);
        }
        __syncthreads();
        write_out(p.seq[o], p.item[o], s_out);
      }
    }

  }

  // ---- sequences without a position to look at
  for (int s = blockIdx.x; s < n; s += gridDim.x) {
    if (max(0, min(__ldg(a.lengths + s), a.c.stride * a.c.rows)) > 0) continue;
    for (int i = tid; i < a.Hq * D / 8; i += kThreads)
      reinterpret_cast<uint4 *>(a.out + (size_t)s * a.ldo)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (a.lse)
      for (int i = tid; i < a.Hq; i += kThreads) a.lse[(size_t)s * a.Hq + i] = -INFINITY;
  }
  if (a.trace && tid == 0) trace_max(a.trace, kTrExit);
}

template <bool kBits8, int kD, int kN>
cudaError_t at_launch(const KvAttendArgs &a, int n_sm, cudaStream_t st, bool pdl) {
  using S = AtShape<kBits8, kD, kN>;
  const EncodeTiledFn enc = encode_tiled();
  if (!enc) return cudaErrorNotSupported;
  AtParams p;
  p.a = a;
  const int group = a.Hq / a.c.heads;
  p.heads = 8 * kN;
  p.blocks_of = (group + p.heads - 1) / p.heads;
  const int es = kBits8 ? 1 : 2;
  const cuuint64_t dims[2] = {(cuuint64_t)a.c.D, (cuuint64_t)a.c.n_pages * a.c.heads * a.c.rows};
  const cuuint64_t strides[1] = {(cuuint64_t)a.c.D * es};
  const cuuint32_t box[2] = {(cuuint32_t)(S::kBox / es), (cuuint32_t)(a.c.rows < S::kTile ? a.c.rows : S::kTile)};
  const CUtensorMapDataType dt = kBits8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUtensorMapSwizzle sw = S::kBox == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  if (!encode_map(enc, &p.k, dt, 2, a.c.k, dims, strides, box, sw) ||
      !encode_map(enc, &p.v, dt, 2, a.c.v, dims, strides, box, sw))
    return cudaErrorInvalidValue;
  return launch_k(kv_attend_kernel<kBits8, kD, kN>, dim3((unsigned)(n_sm < kAtMaxGrid ? n_sm : kAtMaxGrid)),
                  dim3(32 * S::kWarps), S::kSmem, st, pdl, p);
}

template <bool kBits8, int kD, int kN>
cudaError_t at_attribute() {
  return cudaFuncSetAttribute(kv_attend_kernel<kBits8, kD, kN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)AtShape<kBits8, kD, kN>::kSmem);
}

template <bool kBits8, int kN>
cudaError_t at_size(const KvAttendArgs &a, int n_sm, cudaStream_t st, bool pdl) {
  if (a.c.D <= 64) return at_launch<kBits8, 64, kN>(a, n_sm, st, pdl);
  // the products of 8-bit rows bound what memory bounds in bf16: two sizes more (192 in place of 256, 15 sequences of
  // 16384 x 4: 74 us instead of 78, with 16 queries a head 93 instead of 131; 80 in place of 128: 130 instead of 149)
  if (kBits8 && a.c.D <= 96) return at_launch<true, 96, kN>(a, n_sm, st, pdl);
  if (a.c.D <= 128) return at_launch<kBits8, 128, kN>(a, n_sm, st, pdl);
  if (kBits8 && a.c.D <= 192) return at_launch<true, 192, kN>(a, n_sm, st, pdl);
  return at_launch<kBits8, 256, kN>(a, n_sm, st, pdl);
}
}  // namespace

size_t kv_attend_ws_bytes(const KvCache &c, int Hq) {
  const int kN = Hq / c.heads > 8 ? 2 : 1, kD = c.D <= 64 ? 64 : c.D <= 128 ? 128 : 256;
  return (size_t)kAtMaxGrid * (16 + 2) * (16 * kN + kD / 16 * kN * 128) * 4;
}

cudaError_t kv_attend_set_attributes() {
  const cudaError_t e[16] = {
      at_attribute<false, 64, 1>(), at_attribute<false, 128, 1>(), at_attribute<false, 256, 1>(),
      at_attribute<false, 64, 2>(), at_attribute<false, 128, 2>(), at_attribute<false, 256, 2>(),
      at_attribute<true, 64, 1>(),  at_attribute<true, 128, 1>(),  at_attribute<true, 256, 1>(),
      at_attribute<true, 64, 2>(),  at_attribute<true, 128, 2>(),  at_attribute<true, 256, 2>(),
      at_attribute<true, 96, 1>(),  at_attribute<true, 192, 1>(),  at_attribute<true, 96, 2>(), at_attribute<true, 192, 2>()};
  for (const cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

cudaError_t launch_kv_attend(const KvAttendArgs &a, int n_sm, cudaStream_t st, bool pdl) {
  if (a.Hq / a.c.heads > 8)
    return a.c.ks ? at_size<true, 2>(a, n_sm, st, pdl) : at_size<false, 2>(a, n_sm, st, pdl);
  return a.c.ks ? at_size<true, 1>(a, n_sm, st, pdl) : at_size<false, 1>(a, n_sm, st, pdl);
}

}  // namespace moe
