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
// An item (a sequence's key head) that one warp has whole is written at once.
// Where warps share one, the block joins its warps' parts; where blocks do, each
// leaves a part in the workspace, and the last of them, by a counter, joins them
// in the order of the blocks: the result does not depend on who was last.
#include <math.h>

#include "kernels.h"
#include "tma_maps.h"

namespace moe {

namespace {
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kAtSums = 14;  // 8-bit values' weights are held times 2^14

template <bool kBits8, int kD, int kN>
struct AtShape {
  static constexpr int kRow = kD * (kBits8 ? 1 : 2);   // bytes of a row in shared memory
  static constexpr int kBox = kRow < 128 ? kRow : 128; // bytes of a row in one copy
  static constexpr int kTile = kRow >= 512 ? 16 : 32;  // positions
  static constexpr int kHalf = kTile * kRow;           // bytes of a tile's keys, and of its values
  static constexpr int kWarps = kHalf >= 8192 ? 6 : 8;
  static constexpr int kStages = kHalf >= 8192 ? 2 : kHalf >= 4096 ? 3 : 4;
  static constexpr int kPart = 16 * kN + kD / 16 * kN * 128;  // floats of a part: maxima, sums, the output's sum
  static constexpr size_t kScales = kBits8 ? (size_t)kWarps * kStages * 2 * kTile * 4 : 0;
  static constexpr size_t kSmem = 1024 + (size_t)kWarps * kStages * 2 * kHalf + kScales;
  static_assert((size_t)kWarps * kPart * 4 <= (size_t)kWarps * kStages * 2 * kHalf, "parts lie where the tiles lay");
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
  int seq, item; // of the one that ended
  int open_seq, open_item, open_nt;
  unsigned long long open_at;  // first tile of the open one
};

template <bool kBits8, int kD, int kN>
__global__ void __launch_bounds__(32 * AtShape<kBits8, kD, kN>::kWarps, 1)
    kv_attend_kernel(const __grid_constant__ AtParams prm) {
  using S = AtShape<kBits8, kD, kN>;
  constexpr int kTile = S::kTile, kWarps = S::kWarps, kStages = S::kStages, kMt = kTile / 16, kSteps = kD / 16;
  constexpr int kThreads = 32 * kWarps;
  extern __shared__ uint8_t at_raw[];
  uint8_t *const sm = at_raw + ((1024 - (smem_addr(at_raw) & 1023)) & 1023);
  float *const s_scales = reinterpret_cast<float *>(sm + (size_t)kWarps * kStages * 2 * S::kHalf);
  __shared__ uint64_t s_full[kWarps][kStages];
  __shared__ unsigned s_ok[kWarps][kStages];
  __shared__ unsigned long long s_pre[kThreads + 1];
  __shared__ AtWarpParts s_parts[kWarps];
  __shared__ int s_last[2];
  const KvAttendArgs &a = prm.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int D = a.c.D, steps = D / 16, H = a.c.heads, group = a.Hq / H, items = H * prm.blocks_of;
  const int shift = 31 - __clz(a.c.rows), box = min(a.c.rows, kTile), box_shift = 31 - __clz(box);
  const bool tracer = a.trace && blockIdx.x == 0 && tid == 0;
  if (tracer) trace_min(a.trace, kTrEntry);
  if (tid < kWarps * kStages) mbar_init(&s_full[0][0] + tid, 1);
  fence_mbar_init();
  pdl_wait();
  pdl_launch_dependents();
  if (tracer) trace_min(a.trace, kTrWaited);

  // ---- the list of tiles: prefix sums over chunks of sequences, one per thread
  const int n = a.c.n_seqs, chunk = (n + kThreads - 1) / kThreads;
  static_assert((kKvMaxSeqs + kThreads - 1) / kThreads <= 32, "a warp looks through a chunk at once");
  AtCursor<kTile> cur;
  {
    unsigned long long sum = 0;
    for (int i = tid * chunk; i < min(n, (tid + 1) * chunk); ++i) {
      cur.seq = i;
      cur.load(a);
      sum += (unsigned long long)cur.nt * items;
    }
    unsigned long long run = sum;
#pragma unroll
    for (int off = 1; off < 32; off *= 2) {
      const unsigned long long o = __shfl_up_sync(0xffffffffu, run, off);
      if (lane >= off) run += o;
    }
    s_pre[tid + 1] = run;
    if (tid == 0) s_pre[0] = 0;
    __syncthreads();
    unsigned long long before = 0;
    for (int w = 0; w < warp; ++w) before += s_pre[32 * (w + 1)];
    __syncthreads();
    s_pre[tid + 1] = run + before;
    __syncthreads();
  }
  const unsigned long long total = s_pre[kThreads];
  // as many blocks as have a tile for each warp
  const unsigned long long want = (total + kWarps - 1) / kWarps;
  const int blocks = want < gridDim.x ? (int)want : (int)gridDim.x;
  const bool works = (int)blockIdx.x < blocks;
  auto block_at = [&](int b) { return total / blocks * b + total % blocks * b / blocks; };  // first tile of block b
  const unsigned long long bu0 = works ? block_at(blockIdx.x) : 0, bu1 = works ? block_at(blockIdx.x + 1) : 0;
  const unsigned long long u0 = bu0 + (bu1 - bu0) * warp / kWarps, u1 = bu0 + (bu1 - bu0) * (warp + 1) / kWarps;

  // ---- the warp's first tile
  cur.seq = cur.item = cur.tile = cur.nt = 0;
  if (u0 < u1) {
    int ch = 0;
    for (int i = lane; i - lane < kThreads; i += 32) {  // chunks that end at or before u0
      ch += __popc(__ballot_sync(0xffffffffu, i < kThreads && s_pre[i + 1] <= u0));
    }
    cur.seq = min(n - 1, ch * chunk + lane);
    cur.load(a);
    const unsigned long long mine = lane < chunk && ch * chunk + lane < n ? (unsigned long long)cur.nt * items : 0;
    unsigned long long run = mine;
#pragma unroll
    for (int off = 1; off < 32; off *= 2) {
      const unsigned long long o = __shfl_up_sync(0xffffffffu, run, off);
      if (lane >= off) run += o;
    }
    const int who = __popc(__ballot_sync(0xffffffffu, s_pre[ch] + run <= u0));
    const unsigned long long left = u0 - s_pre[ch] - __shfl_sync(0xffffffffu, run - mine, who);
    cur.seq = ch * chunk + who;
    cur.load(a);
    cur.item = (int)(left / (unsigned)cur.nt);
    cur.tile = (int)(left % (unsigned)cur.nt);
  }
  AtCursor<kTile> is = cur;  // of the next tile to copy

  uint8_t *const tiles = sm + (size_t)warp * kStages * 2 * S::kHalf;
  float *const scales = s_scales + warp * kStages * 2 * kTile;
  const int boxes = kTile / box, columns = (D * (kBits8 ? 1 : 2) + S::kBox - 1) / S::kBox;
  const int rows_all = a.c.n_pages * H * a.c.rows;
  bool lost = false, late = false;
  auto copy = [&](int st) {  // the tile at `is` into stage st
    if (lane == 0)
      mbar_arrive_expect_tx(&s_full[warp][st], 2u * (kTile * S::kBox * columns + (kBits8 ? kTile * 4 : 0)));
    __syncwarp();
    bool ok = false;
    if (lane < boxes) {
      const int pos = (is.t0 + is.tile) * kTile + lane * box, kv = is.item / prm.blocks_of;
      const bool need = pos < is.len && pos + box > is.first;
      const int page = need ? __ldg(a.c.table + (size_t)is.seq * a.c.stride + (pos >> shift)) : -1;
      ok = (unsigned)page < (unsigned)a.c.n_pages;
      lost = lost || (need && !ok);
      const int row = ok ? (page * H + kv) * a.c.rows + (pos & (a.c.rows - 1)) : 0;
      const int y = ok ? row : rows_all;  // past the end: filled with zeros
      uint8_t *k = tiles + (size_t)st * 2 * S::kHalf + lane * box * S::kBox;
      for (int i = 0; i < columns; ++i) {
        at_tma(k + i * kTile * S::kBox, &prm.k, i * (S::kBox / (kBits8 ? 1 : 2)), y, &s_full[warp][st]);
        at_tma(k + S::kHalf + i * kTile * S::kBox, &prm.v, i * (S::kBox / (kBits8 ? 1 : 2)), y, &s_full[warp][st]);
      }
      if (kBits8) {
        float *s = scales + st * 2 * kTile + lane * box;
        bulk_g2s(s, a.c.ks + row, box * 4, &s_full[warp][st]);
        bulk_g2s(s + kTile, a.c.vs + row, box * 4, &s_full[warp][st]);
      }
    }
    const unsigned oks = __ballot_sync(0xffffffffu, ok);
    if (lane == 0) s_ok[warp][st] = oks;
    is.next(a, items);
  };
  // Byte in a half of a stage of the 16-byte piece x of row r, as the copies' swizzle lays it.
  auto place = [&](int r, int x) {
    if (S::kBox == 128) return (x >> 3) * kTile * 128 + r * 128 + (((x & 7) ^ (r & 7)) << 4);
    return r * 64 + (((x & 3) ^ ((r >> 1) & 3)) << 4);
  };

  // ---- state of the item at hand: lane (g, c) has the heads 8 i + 2 c and the one after
  uint32_t q[kSteps][kN][2];
  float m[kN][2], l[kN][2], o[kSteps][kN][4], qs[kN][2];
  int unit = 1;  // 8 bits: values' weights in units of 2^(unit - 127 - kAtSums)
  auto begin = [&] {
    const int kv = cur.item / prm.blocks_of, h0 = kv * group + cur.item % prm.blocks_of * prm.heads;
    const int there = min(prm.heads, group - cur.item % prm.blocks_of * prm.heads);
    unit = 1;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const uint16_t *from = a.q + (size_t)cur.seq * a.ldq + (size_t)(h0 + 8 * i + g) * D;
      const bool is_there = 8 * i + g < there;
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
        for (int j = 0; j < 2; ++j) qs[i][j] = at_pow2(__shfl_sync(0xffffffffu, e, 4 * (2 * c + j)));
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
    const int there = min(prm.heads, group - part);
    uint16_t *const out = a.out + (size_t)cur.seq * a.ldo + (size_t)h0 * D;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      float f[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float sum = at_rows_sum(l[i][j]);
        const int h = 8 * i + 2 * c + j;
        if (a.lse && g == 0 && h < there)
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
        if (8 * i + g < there) {
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
  // The state as a part: maxima and sums per head, then the output's sum as the lanes hold it.
  auto leave = [&](float *to) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float sum = at_rows_sum(l[i][j]);
        if (g == 0) {
          to[8 * i + 2 * c + j] = m[i][j];
          to[8 * kN + 8 * i + 2 * c + j] = sum;
        }
      }
      const float up = kBits8 ? at_pow2(unit) : 1.f, down = kBits8 ? at_pow2(127 - kAtSums) : 1.f;
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
        if (s < steps)
          reinterpret_cast<float4 *>(to + 16 * kN)[(s * kN + i) * 32 + lane] =
              make_float4(o[s][i][0] * down * up, o[s][i][1] * down * up, o[s][i][2] * down * up, o[s][i][3] * down * up);
    }
  };

  float *const work = reinterpret_cast<float *>(a.work);
  float *const my_end = work + (size_t)(blockIdx.x * kWarps + warp) * S::kPart;      // part of an item that ends in my run
  float *const block_parts = work + (size_t)gridDim.x * kWarps * S::kPart;           // [grid][2]
  if (u0 < u1) {
    __syncwarp();
#pragma unroll 1
    for (int i = 0; i < kStages; ++i)
      if (u0 + i < u1) copy(i);
    __syncwarp();
  }
  bool ends = false, began = false;
  int end_seq = 0, end_item = 0, st = 0;
  uint32_t phase = 0;
  const bool capped = a.softcap > 0.f;
  const float to_cap = capped ? a.scale / a.softcap : a.scale * kLog2e, cap = a.softcap * kLog2e;
  bool fresh = true;
#pragma unroll 1
  for (unsigned long long u = u0; u < u1; ++u) {
    if (fresh) {
      began = cur.tile == 0;
      begin();
      fresh = false;
    }
    late = __any_sync(0xffffffffu, !mbar_wait(&s_full[warp][st], phase));
    if (late) {  // the copies under way land, or run out too, before the warp's memory is anyone's again
      for (int i = 0; i < kStages && u + i < u1; ++i)
        mbar_wait(&s_full[warp][(st + i) % kStages], phase ^ (st + i >= kStages ? 1u : 0u));
      break;
    }
    const uint32_t keys = smem_addr(tiles + (size_t)st * 2 * S::kHalf), values = keys + S::kHalf;
    const float *ks = scales + st * 2 * kTile, *vs = ks + kTile;
    // which positions count
    const int p0 = (cur.t0 + cur.tile) * kTile;
    const unsigned mask = __ballot_sync(
        0xffffffffu, lane < kTile && p0 + lane >= cur.first && p0 + lane < cur.len && (s_ok[warp][st] >> (lane >> box_shift) & 1u));
    const bool whole = mask == (kTile == 32 ? 0xffffffffu : 0xffffu);

    // ---- scores of the tile's positions, in units of log 2
    float z[kMt][kN][4];
#pragma unroll
    for (int t = 0; t < kMt; ++t) {
#pragma unroll
      for (int i = 0; i < kN; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) z[t][i][j] = 0.f;
      const int r = 16 * t + (lane & 15);
      if (kBits8) {
#pragma unroll
        for (int s = 0; s < kSteps; s += 2) {
          if (s >= steps) continue;
          uint32_t w[4];
          at_ldsm(w, keys + place(r, s + (lane >> 4)));
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] ^= 0x80808080u;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (s + h >= steps) continue;
            const uint32_t x[4] = {at_codes<0x4140>(w[2 * h]), at_codes<0x4140>(w[2 * h + 1]),
                                   at_codes<0x4342>(w[2 * h]), at_codes<0x4342>(w[2 * h + 1])};
#pragma unroll
            for (int i = 0; i < kN; ++i) at_mma<true>(z[t][i], x, q[s + h][i][0], q[s + h][i][1]);
          }
        }
      } else {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          if (s >= steps) continue;
          uint32_t w[4];
          at_ldsm(w, keys + place(r, 2 * s + (lane >> 4)));
#pragma unroll
          for (int i = 0; i < kN; ++i) at_mma<false>(z[t][i], w, q[s][i][0], q[s][i][1]);
        }
      }
      float f[2] = {to_cap, to_cap};
      if (kBits8) {
        f[0] *= ks[16 * t + g];
        f[1] *= ks[16 * t + 8 + g];
      }
#pragma unroll
      for (int i = 0; i < kN; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float v = z[t][i][j] * f[j >> 1];
          if (kBits8) v *= qs[i][j & 1];
          if (capped) v = cap * tanhf(v);
          if (!whole && !(mask >> (16 * t + 8 * (j >> 1) + g) & 1u)) v = -INFINITY;
          z[t][i][j] = v;
        }
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
        const int r = 16 * t + (lane & 15);
#pragma unroll
        for (int s = 0; s < kSteps; s += 2) {
          if (s >= steps) continue;
          uint32_t w[4];
          at_ldsm_t(w, values + place(r, s + (lane >> 4)));
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] ^= 0x80808080u;
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // rows g and g + 8 of the product are dimensions 2 g and 2 g + 1
            if (s + h >= steps) continue;
            const uint32_t x[4] = {at_codes<0x4240>(w[2 * h]), at_codes<0x4341>(w[2 * h]),
                                   at_codes<0x4240>(w[2 * h + 1]), at_codes<0x4341>(w[2 * h + 1])};
#pragma unroll
            for (int i = 0; i < kN; ++i) at_mma<true>(o[s + h][i], x, p[i][0], p[i][1]);
          }
        }
      } else {
        const int r = 16 * t + (lane & 7) + 8 * (lane >> 4);
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
          if (s >= steps) continue;
          uint32_t w[4];
          at_ldsm_t(w, values + place(r, 2 * s + (lane >> 3 & 1)));
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] &= keep[j >> 1];
#pragma unroll
          for (int i = 0; i < kN; ++i) at_mma<false>(o[s][i], w, p[i][0], p[i][1]);
        }
      }
    }
    __syncwarp();  // every lane has read the stage
    if (u + kStages < u1) copy(st);
    if (++st == kStages) {
      st = 0;
      phase ^= 1u;
    }
    if (cur.tile + 1 == cur.nt) {
      fresh = true;
      if (began) {
        finish();
      } else {
        leave(my_end);
        ends = true;
        end_seq = cur.seq;
        end_item = cur.item;
      }
    }
    if (u + 1 < u1) cur.next(a, items);
  }
  if (lane < boxes && lost) set_error(a.err, kErrBadId);
  if (late && lane == 0) set_error(a.err, kErrTimeout);

  // ---- the block's warps join their parts
  const bool open = u0 < u1 && !fresh && !late;
  if (lane == 0) {
    AtWarpParts &p = s_parts[warp];
    p.ends = ends;
    p.open = open;
    p.began = began;
    p.seq = end_seq;
    p.item = end_item;
    p.open_seq = cur.seq;
    p.open_item = cur.item;
    p.open_nt = cur.nt;
    p.open_at = u1 - 1 - (unsigned long long)cur.tile;
  }
  // the tiles are read: parts take their places.  After a wait that ran out nothing is joined (the error tells).
  const bool joins = !__syncthreads_or(late);
  float *const s_open = reinterpret_cast<float *>(sm);
  if (open && joins) leave(s_open + (size_t)warp * S::kPart);
  __syncthreads();
  // A lane's two heads of a slot of a part, the element's dimension.
  auto write_out = [&](int seq, int item, int slot, const float (&v)[4]) {
    const int ln = slot & 31, i = slot / 32 % kN, s = slot / (32 * kN);
    const int part = item % prm.blocks_of * prm.heads, there = min(prm.heads, group - part);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int h = 8 * i + 2 * (ln & 3) + (j & 1);
      const int d = 16 * s + (kBits8 ? 2 * (ln >> 2) + (j >> 1) : (ln >> 2) + 8 * (j >> 1));
      if (h < there)
        a.out[(size_t)seq * a.ldo + (size_t)(item / prm.blocks_of * group + part + h) * D + d] = float_to_bf16_bits(v[j]);
    }
  };
  auto write_lse = [&](int seq, int item, int h, float top, float sum) {
    const int part = item % prm.blocks_of * prm.heads, there = min(prm.heads, group - part);
    if (a.lse && h < there)
      a.lse[(size_t)seq * a.Hq + item / prm.blocks_of * group + part + h] = top * kLn2 + logf(sum);
  };
  const int slots = steps * kN * 32;
  bool first_part = false, last_part = false;  // of items that other blocks share
  for (int slot = tid; joins && slot < (slots + kThreads - 1) / kThreads * kThreads; slot += kThreads) {
    const bool mine = slot < slots;
    const int i = slot / 32 % kN, h = 8 * i + 2 * (slot & 3);
    const bool heads = slot < 32 * kN && (slot & 31) < 4;  // this thread writes its heads' maxima and sums too
    float M[2] = {-INFINITY, -INFINITY}, L[2] = {0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
    bool here = false, any = false;  // the item at hand began in this block; there is one
    auto add = [&](const float *p) {
      if (!mine) return;
      const float4 w4 = reinterpret_cast<const float4 *>(p + 16 * kN)[slot];
      const float w[4] = {w4.x, w4.y, w4.z, w4.w};
      float k0[2], k1[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float pm = p[h + j], t = fmaxf(M[j], pm), use = t == -INFINITY ? 0.f : t;
        k0[j] = at_keep(M[j], use);
        k1[j] = at_keep(pm, use);
        M[j] = t;
        L[j] = L[j] * k0[j] + p[8 * kN + h + j] * k1[j];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = v[j] * k0[j & 1] + w[j] * k1[j & 1];
    };
    auto store = [&](float *p) {
      if (!mine) return;
      reinterpret_cast<float4 *>(p + 16 * kN)[slot] = make_float4(v[0], v[1], v[2], v[3]);
      if (heads) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          p[h + j] = M[j];
          p[8 * kN + h + j] = L[j];
        }
      }
    };
    auto clear = [&] {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        M[j] = -INFINITY;
        L[j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = 0.f;
    };
    for (int w = 0; w < kWarps; ++w) {
      const AtWarpParts &p = s_parts[w];
      if (p.ends) {
        add(work + (size_t)(blockIdx.x * kWarps + w) * S::kPart);
        if (here) {
          if (mine) {
            const float f[2] = {L[0] != 0.f ? 1.f / L[0] : 0.f, L[1] != 0.f ? 1.f / L[1] : 0.f};
            const float r[4] = {v[0] * f[0], v[1] * f[1], v[2] * f[0], v[3] * f[1]};
            write_out(p.seq, p.item, slot, r);
            if (heads) {
              write_lse(p.seq, p.item, h, M[0], L[0]);
              write_lse(p.seq, p.item, h + 1, M[1], L[1]);
            }
          }
        } else {
          store(block_parts + (size_t)(2 * blockIdx.x) * S::kPart);
          first_part = true;
        }
        clear();
        any = false;
      }
      if (p.open) {
        if (p.began) {
          clear();
          here = true;
        }
        add(s_open + (size_t)w * S::kPart);
        any = true;
      }
    }
    if (any) {
      store(block_parts + (size_t)(2 * blockIdx.x + (here ? 1 : 0)) * S::kPart);
      if (here)
        last_part = true;
      else
        first_part = true;
    }
  }

  // ---- the last block of an item joins the blocks' parts
  if (works && (first_part || last_part)) {  // (the same for every thread)
    __threadfence();
    __syncthreads();
    // An item of tiles [at, at + nt) that more than one block has: the first of them, and how many.
    auto span = [&](unsigned long long at, int nt, int &from, int &count) {
      auto of = [&](unsigned long long t) {
        int b = (int)((double)t / (double)total * blocks);
        b = max(0, min(blocks - 1, b));
        while (b + 1 < blocks && block_at(b + 1) <= t) ++b;
        while (block_at(b) > t) --b;
        return b;
      };
      from = of(at);
      count = of(at + (unsigned)nt - 1) - from + 1;
    };
    int from[2] = {0, 0}, count[2] = {0, 0}, seq[2] = {0, 0}, item[2] = {0, 0};
    // the item open at the block's start: it ends in a warp, or is the last one's
    if (first_part) {
      int w = 0;
      while (w < kWarps - 1 && !s_parts[w].ends) ++w;
      const bool ended = s_parts[w].ends;
      int x = w;
      if (!ended)
        while (!s_parts[x].open) --x;
      seq[0] = ended ? s_parts[w].seq : s_parts[x].open_seq;
      item[0] = ended ? s_parts[w].item : s_parts[x].open_item;
      AtCursor<kTile> it;
      it.seq = seq[0];
      it.load(a);
      // its first tile: of the sequence's, item by item
      unsigned long long at;
      if (ended) {
        // the block's first tile lies in it: count back from there
        at = s_pre[seq[0] / chunk];
        for (int s = seq[0] / chunk * chunk; s < seq[0]; ++s) {
          AtCursor<kTile> b;
          b.seq = s;
          b.load(a);
          at += (unsigned long long)b.nt * items;
        }
        at += (unsigned long long)it.nt * item[0];
      } else {
        at = s_parts[x].open_at;
      }
      span(at, it.nt, from[0], count[0]);
    }
    if (last_part) {
      int w = kWarps - 1;
      while (!s_parts[w].began || !s_parts[w].open) --w;
      seq[1] = s_parts[w].open_seq;
      item[1] = s_parts[w].open_item;
      span(s_parts[w].open_at, s_parts[w].open_nt, from[1], count[1]);
    }
    if (tid == 0) {
      for (int k = 0; k < 2; ++k) {
        s_last[k] = 0;
        if (k == 0 ? !first_part : !last_part) continue;
        if (atomicAdd(a.tickets + from[k], 1u) + 1u == (unsigned)count[k]) {
          __threadfence();
          a.tickets[from[k]] = 0u;
          s_last[k] = 1;
        }
      }
    }
    __syncthreads();
    for (int k = 0; k < 2; ++k) {
      if (!s_last[k]) continue;
      float *const s_w = s_open, *const s_sum = s_open + (size_t)count[k] * 8 * kN;  // weights, then sums and maxima
      auto part = [&](int b) { return block_parts + (size_t)(2 * (from[k] + b) + (b == 0 ? 1 : 0)) * S::kPart; };
      __syncthreads();
      for (int h = warp; h < 8 * kN; h += kWarps) {
        float top = -INFINITY, sum = 0.f;
        for (int b = lane; b < count[k]; b += 32) top = fmaxf(top, __ldcg(part(b) + h));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        const float use = top == -INFINITY ? 0.f : top;
        for (int b = lane; b < count[k]; b += 32) {
          const float w = at_keep(__ldcg(part(b) + h), use);
          s_w[b * 8 * kN + h] = w;
          sum += w * __ldcg(part(b) + 8 * kN + h);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (lane == 0) {
          s_sum[h] = sum;
          write_lse(seq[k], item[k], h, top, sum);
        }
      }
      __syncthreads();
      for (int slot = tid; slot < slots; slot += kThreads) {
        const int h = 8 * (slot / 32 % kN) + 2 * (slot & 3);
        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (int b = 0; b < count[k]; ++b) {
          const float4 w4 = __ldcg(reinterpret_cast<const float4 *>(part(b) + 16 * kN) + slot);
          const float w0 = s_w[b * 8 * kN + h], w1 = s_w[b * 8 * kN + h + 1];
          v[0] = fmaf(w4.x, w0, v[0]);
          v[1] = fmaf(w4.y, w1, v[1]);
          v[2] = fmaf(w4.z, w0, v[2]);
          v[3] = fmaf(w4.w, w1, v[3]);
        }
        const float f0 = s_sum[h] != 0.f ? 1.f / s_sum[h] : 0.f, f1 = s_sum[h + 1] != 0.f ? 1.f / s_sum[h + 1] : 0.f;
        const float r[4] = {v[0] * f0, v[1] * f1, v[2] * f0, v[3] * f1};
        write_out(seq[k], item[k], slot, r);
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

constexpr int kAtMaxGrid = 192;

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
  if (a.c.D <= 128) return at_launch<kBits8, 128, kN>(a, n_sm, st, pdl);
  return at_launch<kBits8, 256, kN>(a, n_sm, st, pdl);
}
}  // namespace

size_t kv_attend_ws_bytes(const KvCache &c, int Hq) {
  const int kN = Hq / c.heads > 8 ? 2 : 1, kD = c.D <= 64 ? 64 : c.D <= 128 ? 128 : 256;
  return (size_t)kAtMaxGrid * (8 + 2) * (16 * kN + kD / 16 * kN * 128) * 4;
}

cudaError_t kv_attend_set_attributes() {
  const cudaError_t e[12] = {
      at_attribute<false, 64, 1>(), at_attribute<false, 128, 1>(), at_attribute<false, 256, 1>(),
      at_attribute<false, 64, 2>(), at_attribute<false, 128, 2>(), at_attribute<false, 256, 2>(),
      at_attribute<true, 64, 1>(),  at_attribute<true, 128, 1>(),  at_attribute<true, 256, 1>(),
      at_attribute<true, 64, 2>(),  at_attribute<true, 128, 2>(),  at_attribute<true, 256, 2>()};
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
