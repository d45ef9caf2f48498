// Attention over the 4-bit key-value cache for few rows: single tokens and
// drafts, and any number of rows in fp32.
//
// Mathematics.  With a key's group g of 32 channels as low + scale * n, a
// row's logit is  sum_g scale[t, g] (q_g . n[t, g]) + low[t, g] sum(q_g),  and
// its output  sum_t P[t] scale[t, g] n[t, c] + sum_t P[t] low[t, g]  over
// sum_t P[t]: the products take the levels n as they lie in memory, and scales
// and lows enter per (row, token, group) in fp32.  A 4-bit level in the low
// bits of a 16-bit word is the fp16 denormal n 2^-24, exactly; at bit 4 it is
// 16 n 2^-24.  So a fragment register of two levels costs one AND (and half a
// shift), no conversion: the powers of two are folded into q and the output.
//
// Bound: HBM, 5/4 d bytes a token and kv head.  At 6.5 TB/s an SM has about
// 110 cycles for 16 tokens (d = 128, 2560 bytes), and the work on them is
// about 280 warp instructions (70 issue cycles) at 8 rows: levels must be
// unpacked with next to nothing, which rules out a copy in fp16 through shared
// memory for tcgen05 (its writes and reads alone would exceed the shared
// memory's bandwidth).  The products therefore run on mma.sync m16n8k16, whose
// operands are registers: S = Q K^T with the rows as M (8 or 16 query rows) and
// 8 tokens as N, so that a lane's logits are in the place where P^T is the second
// operand of O^T = V^T P^T with 16 channels as M.
//
// The rows of one kv head (or listed query head) of a sequence, in tiles of
// kRows, are an item; an item's tokens fall into units of 128 (one stage).  The
// units of all items form one sequence, cut into equal runs, one for each CTA, so
// that ragged batches and single long contexts both fill the GPU.  A CTA walks its
// run: one warp copies whole pages (bulk copies, a ring of stages), 8 warps take
// 16 tokens of each stage.  At the end of an item's run the 8 warps join their
// partial results; an item shared by several CTAs is joined by a second
// small kernel.  Everything is in a fixed order: results do not change between runs.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <climits>
#include <type_traits>

#include "internal.h"
#include "kv4.cuh"
#include "ptx.cuh"
#include "tma_map.h"

namespace sbsa {
namespace {

constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr int kTile = 16;         // tokens of a warp's step
constexpr int kUnit = 8 * kTile;  // tokens of a stage: 8 warps take it
constexpr int kMaxCtas = 160;
// Weights are 2^(S - M), M = (reference of the logits) + (reference of the
// values' exponents) - kHead; each reference moves only when it is outgrown by more
// than kLazy, so the fp16 weights times a scale stay below 2^(kHead + 2 kLazy + 1) = 2^15.
constexpr float kHead = 6.f, kLazy = 4.f;

// W computing warps take the tiles of 16 tokens in turn.  8 bf16 rows leave
// registers for 12; 16 rows or two-part fp32 rows take 8 (spilled registers cost
// far more than warps gain: next to the ring the L1 has a few KB left).  The copying
// warp and its three idle neighbours are a warpgroup whose registers the computing
// warps take over.
template <int D, int NT, int W>
struct Cfg {
  static constexpr int kWarps = W;
  static constexpr int kThreads = (W + 4) * 32;
  // launched with 128 (512 threads) or 168 (384) registers a thread: 384 * 152 + 128 * 56 =
  // 512 * 128, 256 * 224 + 128 * 56 = 384 * 168
  static constexpr int kRegs = W == 12 ? 152 : 224, kRegsCopy = 56;
  static constexpr int kRows = 8 * NT;
  static constexpr int kGroups = D / 32;
  static constexpr int kStageBytes = kUnit * (D / 8) * 10;
  static constexpr int kStages = D == 64 ? 10 : 7;
  static constexpr int kOutStride = D + 4;  // floats; spreads the heads over the banks
  static constexpr int kOffOut = kStages * kStageBytes;
  static constexpr int kOffStat = kOffOut + kWarps * kRows * kOutStride * 4;
  // per warp and row: M, l, and the lows' sums of the groups
  static constexpr int kStat = 2 + kGroups;
  // per warp: its tokens' key and value scales in fp32
  static constexpr int kOffScale = kOffStat + kWarps * kRows * kStat * 4;
  static constexpr int kOffMeta = kOffScale + kWarps * 2 * kTile * kGroups * 4;
  static constexpr int kOffScan = kOffMeta + kStages * 8 * 4;
  static constexpr int kOffBar = kOffScan + (kThreads / 32 + 1) * 8 + 32;
  static constexpr int kSmem = kOffBar + 2 * kStages * 8 + 16;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static_assert(kOffBar % 8 == 0 && kOffScan % 8 == 0 && kOffScale % 16 == 0, "alignment");
};

struct Part {  // which item's first part a CTA holds, in how many parts (0: none)
  int parts, seq, head, tile;
};

constexpr int slot_floats(int d) { return 16 * (d + 2); }

struct Params {
  Kv4AttendArgs a;
  int heads;         // items per sequence and row tile: kv heads, or listed query heads
  int group;         // query heads of an item
  int kv_div;        // item head / kv_div = kv head
  float scale_log2;  // sm_scale * log2(e)
  float* slots;
  Part* parts;
};

// The sequence as an item sees it.
struct Seq {
  int first, rows, len;  // first row, number of rows, tokens
};

__device__ __forceinline__ Seq seq_of(const Params& p, int b) {
  Seq s;
  const int lo = clamp_int(p.a.b.cu[b], 0, p.a.b.n_tokens);
  const int hi = clamp_int(p.a.b.cu[b + 1], lo, p.a.b.n_tokens);
  s.first = lo;
  s.rows = hi - lo;
  s.len = kv4_len(p.a.b, b);
  return s;
}

// What an item costs a CTA besides its units (rows, joining, output), in units.  Runs are
// cut by cost: item after item, kItemCost and then the units.
constexpr int kItemCost = 4;

// Units of 128 tokens of each row tile of (sequence, head) and the number of
// tiles; a tile that sees nothing still takes one unit (it writes zeros).
template <int ROWS>
__device__ __forceinline__ void item_size(const Params& p, int b, int head, int* units,
                                          int* tiles) {
  const Seq s = seq_of(p, b);
  *tiles = (int)(((long long)s.rows * p.group + ROWS - 1) / ROWS);
  int n = s.len;
  if (p.a.list_heads)
    n = clamp_int(p.a.cnt[(long long)b * p.heads + head], 0, p.a.max_blocks) * p.a.block;
  n = (n + kUnit - 1) / kUnit;
  *units = n < 1 ? 1 : n;
}

// The CTA's place in the sequence of items.
struct Walk {
  int b, head, tile;   // current item
  int units, tiles;    // its units, its sequence's tiles
  long long cost;      // cost from the item's start to the run's first
  long long left;      // and to the run's end
  // units of the item that are the CTA's: [begin, end), empty where the run ends before the first
  __device__ int begin() const { return cost > kItemCost ? (int)cost - kItemCost : 0; }
  __device__ int end() const {
    const long long e = left - kItemCost;
    return e < 0 ? 0 : e < units ? (int)e : units;
  }
};

__device__ __forceinline__ long long units_cost(int units) { return (long long)kItemCost + units; }

template <int ROWS>
__device__ __forceinline__ void next_item(const Params& p, Walk& w) {
  w.left -= units_cost(w.units);
  w.cost = 0;
  if (w.left <= 0) return;
  if (++w.tile < w.tiles) return;
  w.tile = 0;
  do {
    if (++w.head == p.heads) {
      w.head = 0;
      if (++w.b == p.a.b.n_seqs) {
        w.left = 0;
        return;
      }
    }
    item_size<ROWS>(p, w.b, w.head, &w.units, &w.tiles);
  } while (w.tiles == 0);
}

// D += A B on fp16, 16 x 16 by 16 x 8; and D = A B.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// D = A B on bf16.
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// D += A B on tf32, 16 x 8 by 8 x 8; rows 8 to 15 of A are zero.
__device__ __forceinline__ void mma_tf32(float (&d)[4], uint32_t a0, uint32_t a2, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%5}, {%7,%8}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(0), "r"(a2), "r"(b0), "r"(b1));
}

// Two fp32 values as their bf16 parts: returns the leading parts and leaves the rest.
__device__ __forceinline__ uint32_t take_bf16(float& lo, float& hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  const uint32_t w = *reinterpret_cast<const uint32_t*>(&h);
  lo -= __uint_as_float(w << 16);
  hi -= __uint_as_float(w & 0xFFFF0000u);
  return w;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float scale_of(uint32_t pair) { return __uint_as_float(pair << 16); }
// The words of one token's chunk of levels, or its pairs, for all groups.
template <int NG>
struct Words {
  uint32_t w[NG];
};
template <int NG>
__device__ __forceinline__ Words<NG> lds_words(const void* p) {
  Words<NG> r;
  if constexpr (NG == 4) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    r.w[0] = u.x, r.w[1] = u.y, r.w[2] = u.z, r.w[3] = u.w;
  } else if constexpr (NG == 2) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    r.w[0] = u.x, r.w[1] = u.y;
  } else {
    r.w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
  return r;
}

// 8 channels of a query row, as fp32.
__device__ __forceinline__ void load_q8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load_q8(const float* p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                            *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }

// Row r of a tile: the token row and head of o (and q); false past the last.
__device__ __forceinline__ bool row_of(const Params& p, const Seq& s, int head, long long row,
                                       long long* t, int* h, int* i) {
  *i = (int)(row / p.group);
  if (*i >= s.rows) return false;
  *t = s.first + *i;
  *h = head * p.group + (int)(row % p.group);
  return true;
}

template <int THREADS>
__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// T: type of q and o.  fp32 rows enter the products as two fp16 parts (22
// bits), and so do their weights; a bf16 row is one fp16 part exactly (its
// elements are scaled by a power of two so that the largest is near 2^10) and
// the weights are rounded to fp16 once, 2^-11 of each.
template <int D, int NT, int W, typename T>
__global__ void __launch_bounds__((W + 4) * 32, 1)
    kv4_attend_kernel(const __grid_constant__ Params p) {
  using C = Cfg<D, NT, W>;
  constexpr int kWarps = C::kWarps, kThreads = C::kThreads;
  constexpr int NG = C::kGroups;
  constexpr int ROWS = C::kRows;
  constexpr int PARTS = sizeof(T) == 4 ? 2 : 1;
  extern __shared__ __align__(128) unsigned char smem[];
  float* s_out = reinterpret_cast<float*>(smem + C::kOffOut);
  float* s_stat = reinterpret_cast<float*>(smem + C::kOffStat);
  int* s_meta = reinterpret_cast<int*>(smem + C::kOffMeta);  // [stage][page]: first token's position
  long long* s_scan = reinterpret_cast<long long*>(smem + C::kOffScan);
  int* s_start = reinterpret_cast<int*>(s_scan + kThreads / 32 + 1);  // b, head, tile, unit, abort
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* empty = full + C::kStages;
  volatile int* abort_flag = s_start + 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int page = p.a.b.page, rec = kv4_rec_bytes(page, D);

  // ---- the CTA's run of units: a scan over the items' sizes
  const int items = p.a.b.n_seqs * p.heads;
  const int per = (items + kThreads - 1) / kThreads;
  const int i0 = min(items, (int)threadIdx.x * per), i1 = min(items, i0 + per);
  long long mine = 0;
  for (int i = i0; i < i1; ++i) {
    int units, tiles;
    item_size<ROWS>(p, i / p.heads, i % p.heads, &units, &tiles);
    mine += units_cost(units) * tiles;
  }
  long long incl = mine;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long x = __shfl_up_sync(0xFFFFFFFFu, incl, m);
    if (lane >= m) incl += x;
  }
  if (lane == 31) s_scan[warp] = incl;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 8);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  long long before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  const int ctas = (int)(total < (long long)gridDim.x ? total : (long long)gridDim.x);
  const int cta = blockIdx.x;
  if (threadIdx.x == 0) p.parts[cta].parts = 0;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (cta >= ctas) return;
  const long long u0 = total * cta / ctas, u1 = total * (cta + 1) / ctas;
  if (u0 >= before && u0 < before + mine) {
    long long x = before;
    for (int i = i0; i < i1; ++i) {
      int units, tiles;
      item_size<ROWS>(p, i / p.heads, i % p.heads, &units, &tiles);
      if (u0 < x + units_cost(units) * tiles) {
        s_start[0] = i / p.heads;
        s_start[1] = i % p.heads;
        s_start[2] = (int)((u0 - x) / units_cost(units));
        s_start[3] = (int)((u0 - x) % units_cost(units));
        break;
      }
      x += units_cost(units) * tiles;
    }
  }
  __syncthreads();
  Walk w;
  w.b = s_start[0], w.head = s_start[1], w.tile = s_start[2], w.cost = s_start[3];
  w.left = w.cost + u1 - u0;
  item_size<ROWS>(p, w.b, w.head, &w.units, &w.tiles);

  float* ks = reinterpret_cast<float*>(smem + C::kOffScale) + warp * 2 * kTile * NG;
  float* vs = ks + kTile * NG;
  auto fail = [&]() {
    *abort_flag = 1;
    if (p.a.b.status) atomicCAS(p.a.b.status, 0, SBSA_ERR_TIMEOUT);
  };

  if (warp >= kWarps) {
    regs_lower<C::kRegsCopy>();
    if (warp > kWarps) return;
    // ================================================================ copies
    const int pages = kUnit / page;
    int n = 0;  // stages filled
    bool ok = true;
    while (w.left > 0 && ok) {
      const Seq s = seq_of(p, w.b);
      const int begin = w.begin(), end = w.end();
      // tokens that the tile's last row sees
      const long long last = min((long long)(w.tile + 1) * ROWS, (long long)s.rows * p.group) - 1;
      const int limit = s.len - s.rows + (int)(last / p.group) + 1;
      const int32_t* list = nullptr;
      int count = 0;
      if (p.a.list_heads) {
        const long long row = (long long)w.b * p.heads + w.head;
        list = p.a.idx + row * p.a.max_blocks;
        count = clamp_int(p.a.cnt[row], 0, p.a.max_blocks);
      }
      const int32_t* table = p.a.b.table + (long long)w.b * p.a.b.max_pages;
      // 32 pages at a time: lane x looks up page x (its number, or -1, and the position of its
      // first token), so that a memory round trip serves 32 * page / 128 units
      auto look = [&](int first, int* pos) {
        long long at = (long long)(first + lane) * page;
        *pos = INT_MAX - kUnit;
        if (list) {
          const int e = (int)(at / p.a.block);
          if (e >= count) return -1;
          const int j = list[e];
          if (j < 0 || j > (s.len - 1) / p.a.block || s.len == 0) {
            kv4_record(p.a.b.status);
            return -1;
          }
          at = j * p.a.block + at % p.a.block;
        }
        if (at >= limit) return -1;
        const int pg = table[at / page];
        if (pg < 0 || pg >= p.a.b.n_pages) {
          kv4_record(p.a.b.status);
          return -1;
        }
        *pos = (int)at;
        return pg;
      };
      const uint8_t* heads = p.a.cache + (long long)(w.head / p.kv_div) * 2 * rec;
      int chunk = begin * pages, pos = 0, pg = begin < end ? look(chunk, &pos) : -1;
      for (int u = begin; u < end; ++u) {
        if (u * pages - chunk + pages > 32) {
          chunk = u * pages;
          pg = look(chunk, &pos);
        }
        const int st = n % C::kStages;
        bool good = true;
        if (lane == 0 && n >= C::kStages)
          good = mbar_wait_bounded(&empty[st], (n / C::kStages - 1) & 1, abort_flag, kTimeoutNs);
        ok = __shfl_sync(0xFFFFFFFFu, good, 0);
        if (!ok) break;
        const int x = lane - (u * pages - chunk);  // this lane's page within the unit
        const bool in = x >= 0 && x < pages;
        if (in) s_meta[st * 8 + x] = pos;
        const int bytes = 2 * rec * __popc(__ballot_sync(0xFFFFFFFFu, in && pg >= 0));
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&full[st], bytes);
        __syncwarp();
        if (in && pg >= 0)
          bulk_load(smem + st * C::kStageBytes + x * 2 * rec,
                    heads + (long long)pg * p.a.b.hkv * 2 * rec, 2 * rec, &full[st]);
        ++n;
      }
      next_item<ROWS>(p, w);
    }
    if (!ok && lane == 0) {
      if (!*abort_flag) fail();
      volatile int never = 0;  // copies still on their way into shared memory
      for (int i = max(0, n - C::kStages); i < n; ++i)
        mbar_wait_bounded(&full[i % C::kStages], (i / C::kStages) & 1, &never, kTimeoutNs);
    }
    return;
  }

  // ==================================================================== products
  regs_raise<C::kRegs>();
  const int r = lane >> 2, q = lane & 3;
  // Column n of S is token n ^ (n >> 2) of 8: with it neither the keys', the
  // values' nor the pairs' reads meet a bank twice.  A lane's logits are those of
  // columns 2q and 2q + 1, its key rows' that of column r.
  const int tok_k = r ^ (r >> 2);
  const int tok_a = (2 * q) ^ (q >> 1), tok_b = (2 * q + 1) ^ (q >> 1);
  // this warp's next tile (8 to a stage), and its stage's number and place in the ring
  int tile = warp, stage = 0, st = 0, phase = 0;
  int base_n = 0;                    // the number of the item's first stage
  bool ok = true;
  while (w.left > 0) {
    const Seq s = seq_of(p, w.b);
    const int begin = w.begin(), end = w.end();
    if (begin >= end) break;  // the run ends in the item's fixed cost: the next CTA begins it
    const long long row0 = (long long)w.tile * ROWS;

    // ---- the query rows as fragments: register pairs (0, 4), (1, 5)/16, (2, 6), (3, 7)/16 of
    // each 8 channels, as the levels come out of a word
    uint32_t aq[PARTS][NG][2][4];
    // sum(q_g) 2^-24 in three bf16 parts, against the lows of two groups a lane: with 4 groups
    // k-pairs q = 0, 1 hold the first part of groups (0, 1) and (2, 3), 2 and 3 the second, 8 behind
    // them the third; with 2 groups q = 0, 1, 2 hold the three parts
    uint32_t al[4] = {0, 0, 0, 0};
    float f[NT];
    int lim[NT];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (x >= NT) {
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int pt = 0; pt < PARTS; ++pt)
            aq[pt][g][0][1] = aq[pt][g][0][3] = aq[pt][g][1][1] = aq[pt][g][1][3] = 0;
        continue;
      }
      long long t;
      int h, i;
      const bool have = row_of(p, s, w.head, row0 + x * 8 + r, &t, &h, &i);
      float v[NG][8], qs[NG];
      float mx = 0.f;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (have) {
          load_q8(static_cast<const T*>(p.a.q.ptr) + t * p.a.q.token + h * p.a.q.head + g * 32 + q * 8,
                  v[g]);
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c) v[g][c] = 0.f;
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) mx = fmaxf(mx, fabsf(v[g][c]));
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
      const int e = clamp_int(137 - (int)(__float_as_uint(mx) >> 23), -90, 100);
      const float up = __uint_as_float((uint32_t)(e + 127) << 23);
      f[x & (NT - 1)] = p.scale_log2 * __uint_as_float((uint32_t)(24 - e + 127) << 23);
      // rows that see nothing (before the sequence, beyond max_new) mask all; rows past the
      // tile's last mask nothing, so that they never send the warp to the masked path
      lim[x & (NT - 1)] = INT_MAX;
      if (have) {
        const int visible = s.len - s.rows + i + 1;
        lim[x & (NT - 1)] = i < p.a.max_new ? max(visible, 0) : 0;
        if ((visible < 1 || i >= p.a.max_new) && q == 0) kv4_record(p.a.b.status);
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          v[g][c] *= up;
          sum += v[g][c];
        }
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float sc = (j & 1) ? 0.0625f : 1.f;
          const float lo = v[g][j] * sc, hi = v[g][j + 4] * sc;
          const uint32_t h0 = pack_half2(lo, hi);
          aq[0][g][j >> 1][(j & 1) * 2 + x] = h0;
          if constexpr (PARTS == 2) {
            const __half2 back = *reinterpret_cast<const __half2*>(&h0);
            aq[PARTS - 1][g][j >> 1][(j & 1) * 2 + x] =
                pack_half2(lo - __low2float(back), hi - __high2float(back));
          }
        }
        qs[g] = sum * 0x1p-24f;
      }
      if constexpr (NG == 4) {
        float u = (q & 1) ? qs[2] : qs[0], w2 = (q & 1) ? qs[3] : qs[1];
        const uint32_t p0 = take_bf16(u, w2), p1 = take_bf16(u, w2), p2 = take_bf16(u, w2);
        al[x] = q < 2 ? p0 : p1;
        al[2 + x] = q < 2 ? p2 : 0;
      } else {
        float u = qs[0], w2 = qs[1];
        const uint32_t p0 = take_bf16(u, w2), p1 = take_bf16(u, w2), p2 = take_bf16(u, w2);
        al[x] = q == 0 ? p0 : q == 1 ? p1 : q == 2 ? p2 : 0;
      }
    }
    int lim_min = lim[0], lim_max = lim[0] == INT_MAX ? 0 : lim[0];
    if constexpr (NT == 2) {
      lim_min = min(lim_min, lim[NT - 1]);
      lim_max = max(lim_max, lim[NT - 1] == INT_MAX ? 0 : lim[NT - 1]);
    }
    lim_min = __reduce_min_sync(0xFFFFFFFFu, lim_min);
    lim_max = __reduce_max_sync(0xFFFFFFFFu, lim_max);

    // outputs; and rows 0 to NG - 1 the lows' sums of the groups, row 4 the weights' sum
    // rows' references: ms for the logits, me (an exponent as bf16 holds it) for the magnitude of the
    // values, common to all rows; weights are 2^(logit - m), m = ms + (me - 127) - kHead
    float o[NT][NG][2][4], ol[NT][4], m[NT], ms[NT];
    uint32_t me = 0, big = 0;
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      m[x] = ms[x] = -FLT_MAX;
#pragma unroll
      for (int c = 0; c < 4; ++c) ol[x][c] = 0.f;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[x][g][j][c] = 0.f;
      }
    }

    // ---- one step: 16 tokens.  kMask: some row does not see all of them.
    auto step = [&](const unsigned char* base, int row, int pos, auto mask_tag) {
      constexpr bool kMask = decltype(mask_tag)::value;
      const unsigned char* kl = base + row * (D / 2);
      const unsigned char* kp = base + page * (D / 2) + row * (D / 8);
      const unsigned char* vl = kl + rec;
      const unsigned char* vp = kp + rec;
      // each lane unpacks the scales of half a token (4 groups) or a whole one, for all lanes
      // to read, and looks at the largest magnitude of its values' scales and lows
      uint32_t top = 0;
      {
        const Words<NG / 2> e = lds_words<NG / 2>(vp + lane * (D / 16));
        const Words<NG / 2> k = lds_words<NG / 2>(kp + lane * (D / 16));
        const bool in = !kMask || pos + (lane >> 1) < lim_max;
#pragma unroll
        for (int g = 0; g < NG / 2; ++g) {
          top = __vmaxu2(top, e.w[g] & 0x7FFF7FFFu);
          ks[lane * (NG / 2) + g] = scale_of(k.w[g]);
          vs[lane * (NG / 2) + g] = in ? scale_of(e.w[g]) : 0.f;
        }
        if (!in) top = 0;
      }
      __syncwarp();
      // ---- logits (without the row's factor f)
      float sv[NT][4];  // tokens a, b of the first 8, then of the second
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const Words<NG> wk = lds_words<NG>(kl + (hf * 8 + tok_k) * (D / 2) + q * (D / 8));
        const Words<2> pl = lds_words<2>(kp + (hf * 8 + tok_k) * (D / 8) + (NG == 4 ? (q & 1) * 8 : 0));
        const Words<NG> sa = lds_words<NG>(ks + (hf * 8 + tok_a) * NG);
        const Words<NG> sb = lds_words<NG>(ks + (hf * 8 + tok_b) * NG);
        const uint32_t lows = __byte_perm(pl.w[0], pl.w[1], 0x7632);
        float acc[4];
        mma_bf16_first(acc, al, lows, lows);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float d[4];
          const uint32_t x = wk.w[g], y = x >> 8;
          mma_f16_first(d, aq[0][g][0], x & 0x000F000Fu, x & 0x00F000F0u);
          mma_f16(d, aq[0][g][1], y & 0x000F000Fu, y & 0x00F000F0u);
          if constexpr (PARTS == 2) {
            mma_f16(d, aq[PARTS - 1][g][0], x & 0x000F000Fu, x & 0x00F000F0u);
            mma_f16(d, aq[PARTS - 1][g][1], y & 0x000F000Fu, y & 0x00F000F0u);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            acc[2 * nt] = fmaf(__uint_as_float(sa.w[g]), d[2 * nt], acc[2 * nt]);
            acc[2 * nt + 1] = fmaf(__uint_as_float(sb.w[g]), d[2 * nt + 1], acc[2 * nt + 1]);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          sv[nt][2 * hf] = acc[2 * nt];
          sv[nt][2 * hf + 1] = acc[2 * nt + 1];
          if constexpr (kMask) {
            if (pos + hf * 8 + tok_a >= lim[nt]) sv[nt][2 * hf] = -INFINITY;
            if (pos + hf * 8 + tok_b >= lim[nt]) sv[nt][2 * hf + 1] = -INFINITY;
          }
        }
      }
      // ---- the references, moved only when they have to
      bool need = __vmaxu2(top, big) != big;
      float mx[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mx[nt] = fmaxf(fmaxf(sv[nt][0], sv[nt][1]), fmaxf(sv[nt][2], sv[nt][3])) * f[nt];
        need |= mx[nt] > ms[nt] + kLazy;
      }
      if (__any_sync(0xFFFFFFFFu, need)) {
        uint32_t e = max((top & 0xFFFFu) < 0x7F80u ? top & 0xFFFFu : 0u,
                         (top >> 16) < 0x7F80u ? top >> 16 : 0u);
        if (top >= 0x7F800000u || (top & 0xFFFFu) >= 0x7F80u) {  // a NaN hides its lane's others
          e = 0;
          const Words<NG / 2> w2 = lds_words<NG / 2>(vp + lane * (D / 16));
#pragma unroll
          for (int g = 0; g < NG / 2; ++g) {
            const uint32_t lo = w2.w[g] & 0x7FFFu, hi = (w2.w[g] >> 16) & 0x7FFFu;
            e = max(e, lo < 0x7F80u ? lo : 0u);
            e = max(e, hi < 0x7F80u ? hi : 0u);
          }
        }
        e = max(__reduce_max_sync(0xFFFFFFFFu, e) >> 7, 47u);
        const float de = e > me ? (float)((int)e - (int)me) : 0.f;
        if (e > me) {
          me = e;
          const uint32_t lim16 = min(((e + (int)kLazy) << 7) | 0x7Fu, 0x7F7Fu);
          big = lim16 | (lim16 << 16);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float mn = mx[nt];
          mn = fmaxf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, 1));
          mn = fmaxf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, 2));
          mn = fmaxf(mn, ms[nt]);
          const float alpha = exp2f(ms[nt] - mn - de);
          ms[nt] = mn;
          m[nt] = mn + ((float)((int)me - 127) - kHead);
          const float a0 = __shfl_sync(0xFFFFFFFFu, alpha, 8 * q);
          const float a1 = __shfl_sync(0xFFFFFFFFu, alpha, 8 * q + 4);
          ol[nt][0] *= a0;
          ol[nt][1] *= a1;
#pragma unroll
          for (int g = 0; g < NG; ++g) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              o[nt][g][j][0] *= a0;
              o[nt][g][j][1] *= a1;
              o[nt][g][j][2] *= a0;
              o[nt][g][j][3] *= a1;
            }
          }
        }
      }
      // ---- weights
      float pw[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          pw[nt][c] = ex2_approx(fmaf(sv[nt][c], f[nt], -m[nt]));
          if constexpr (PARTS == 1)  // cut to tf32: one value for the sums and the products
            pw[nt][c] = __uint_as_float(__float_as_uint(pw[nt][c]) & 0xFFFFE000u);
        }
      // ---- lows of the values and the weights' sum: the lows as they are (row g of the first
      // operand), ones (row 4), against the weights in tf32 (in two parts of fp32 rows)
      {
        const unsigned char* lp = vp + (r & (NG - 1)) * 4;
        uint32_t lw[4] = {*reinterpret_cast<const uint32_t*>(lp + tok_a * (D / 8)),
                          *reinterpret_cast<const uint32_t*>(lp + tok_b * (D / 8)),
                          *reinterpret_cast<const uint32_t*>(lp + (8 + tok_a) * (D / 8)),
                          *reinterpret_cast<const uint32_t*>(lp + (8 + tok_b) * (D / 8))};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          lw[c] &= 0xFFFF0000u;
          if constexpr (kMask) {
            // nothing from behind the last token; a NaN reaches the rows that see it through its
            // scale below, and must not meet the weight 0 of a row that does not
            const bool in = pos + (c >> 1) * 8 + ((c & 1) ? tok_b : tok_a) < lim_max;
            if (!in || (lw[c] & 0x7F800000u) == 0x7F800000u) lw[c] = 0;
          }
          if (r == 4) lw[c] = 0x3F800000u;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint32_t x[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) x[c] = __float_as_uint(pw[nt][c]) & 0xFFFFE000u;
          mma_tf32(ol[nt], lw[0], lw[1], x[0], x[1]);
          mma_tf32(ol[nt], lw[2], lw[3], x[2], x[3]);
          if constexpr (PARTS == 2) {
#pragma unroll
            for (int c = 0; c < 4; ++c) x[c] = __float_as_uint(pw[nt][c] - __uint_as_float(x[c]));
            mma_tf32(ol[nt], lw[0], lw[1], x[0], x[1]);
            mma_tf32(ol[nt], lw[2], lw[3], x[2], x[3]);
          }
        }
      }
      // ---- values
      const unsigned char* vl2 = vl + (r ^ (NG == 4 ? (q & 1) * 4 : 0)) * (D / 16);
      const Words<NG / 2> va0 = lds_words<NG / 2>(vl2 + tok_a * (D / 2));
      const Words<NG / 2> vb0 = lds_words<NG / 2>(vl2 + tok_b * (D / 2));
      const Words<NG / 2> va1 = lds_words<NG / 2>(vl2 + (8 + tok_a) * (D / 2));
      const Words<NG / 2> vb1 = lds_words<NG / 2>(vl2 + (8 + tok_b) * (D / 2));
      const Words<NG> sc[4] = {lds_words<NG>(vs + tok_a * NG), lds_words<NG>(vs + tok_b * NG),
                               lds_words<NG>(vs + (8 + tok_a) * NG), lds_words<NG>(vs + (8 + tok_b) * NG)};
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint32_t sel = (g & 1) ? 0x7632u : 0x5410u;
        const uint32_t x0 = __byte_perm(va0.w[g >> 1], vb0.w[g >> 1], sel), y0 = x0 >> 8;
        const uint32_t x1 = __byte_perm(va1.w[g >> 1], vb1.w[g >> 1], sel), y1 = x1 >> 8;
        const uint32_t f0[4] = {x0 & 0x000F000Fu, x0 & 0x00F000F0u, x1 & 0x000F000Fu, x1 & 0x00F000F0u};
        const uint32_t f1[4] = {y0 & 0x000F000Fu, y0 & 0x00F000F0u, y1 & 0x000F000Fu, y1 & 0x00F000F0u};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float pv[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            pv[c] = pw[nt][c] * __uint_as_float(sc[c].w[g]);
            if constexpr (kMask)  // 0 * NaN in a hidden place
              if (pos + (c >> 1) * 8 + ((c & 1) ? tok_b : tok_a) >= lim[nt]) pv[c] = 0.f;
          }
          const uint32_t b0 = pack_half2(pv[0], pv[1]), b1 = pack_half2(pv[2], pv[3]);
          mma_f16(o[nt][g][0], f0, b0, b1);
          mma_f16(o[nt][g][1], f1, b0, b1);
          if constexpr (PARTS == 2) {
            const __half2 h0 = *reinterpret_cast<const __half2*>(&b0);
            const __half2 h1 = *reinterpret_cast<const __half2*>(&b1);
            const uint32_t c0 = pack_half2(pv[0] - __low2float(h0), pv[1] - __high2float(h0));
            const uint32_t c1 = pack_half2(pv[2] - __low2float(h1), pv[3] - __high2float(h1));
            mma_f16(o[nt][g][0], f0, c0, c1);
            mma_f16(o[nt][g][1], f1, c0, c1);
          }
        }
      }
    };

    const int page_log = __ffs(page) - 1;
    for (; (tile >> 3) - base_n < end - begin; tile += W) {
      st += (tile >> 3) - stage;
      stage = tile >> 3;
      if (st >= C::kStages) {
        st -= C::kStages;
        phase ^= 1;
      }
      if (ok) ok = mbar_wait_bounded(&full[st], phase, abort_flag, kTimeoutNs);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (ok) {
        const int pg = (tile & 7) * kTile >> page_log, row = (tile & 7) * kTile & (page - 1);
        const int pos = s_meta[st * 8 + pg] + row;
        const unsigned char* base = smem + st * C::kStageBytes + pg * 2 * rec;
        if (pos + kTile <= lim_min)
          step(base, row, pos, std::false_type{});
        else if (pos < lim_max)
          step(base, row, pos, std::true_type{});
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
      }
    }
    base_n += end - begin;
    if (!ok && lane == 0 && !*abort_flag) fail();

    // ---- join the 8 warps: each leaves its rows' outputs and sums in shared memory
    consumers_sync<kWarps * 32>();  // the previous item's have been read
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float* dst = s_out + (warp * ROWS + nt * 8 + 2 * q + c) * C::kOutStride + g * 32 + r * 4;
          *reinterpret_cast<float4*>(dst) =
              make_float4(o[nt][g][0][c] * 0x1p24f, o[nt][g][0][2 + c] * 0x1p20f,
                          o[nt][g][1][c] * 0x1p24f, o[nt][g][1][2 + c] * 0x1p20f);
        }
      }
      // lane (r, q) has row r of the sums for heads 2q and 2q + 1
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float* st = s_stat + (warp * ROWS + nt * 8 + 2 * q + c) * C::kStat;
        if (r == 4) st[1] = ol[nt][c];
        if (r < NG) st[2 + r] = ol[nt][c];
      }
      if (q == 0) s_stat[(warp * ROWS + nt * 8 + r) * C::kStat] = m[nt];
    }
    consumers_sync<kWarps * 32>();
    const bool whole = begin == 0 && end == w.units;
    const int slot = 2 * cta + (begin == 0 ? 1 : 0);
    constexpr int kPerRow = D / 4;  // threads of a row, 4 channels each
    for (int x = threadIdx.x; x < ROWS * kPerRow; x += kWarps * 32) {
      const int row = x / kPerRow, c = x % kPerRow * 4;
      float top = -FLT_MAX;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) top = fmaxf(top, s_stat[(i * ROWS + row) * C::kStat]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        const float* st = s_stat + (i * ROWS + row) * C::kStat;
        const float4 v = *reinterpret_cast<const float4*>(s_out + (i * ROWS + row) * C::kOutStride + c);
        const float fac = exp2f(st[0] - top), lw = st[2 + c / 32];
        sum = fmaf(fac, st[1], sum);
        acc.x = fmaf(fac, v.x + lw, acc.x);
        acc.y = fmaf(fac, v.y + lw, acc.y);
        acc.z = fmaf(fac, v.z + lw, acc.z);
        acc.w = fmaf(fac, v.w + lw, acc.w);
      }
      if (whole) {
        long long t;
        int h, i;
        if (row_of(p, s, w.head, row0 + row, &t, &h, &i)) {
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          store4(static_cast<T*>(p.a.o) + t * p.a.o_token + h * p.a.o_head + c,
                 make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
        }
      } else {
        float* dst = p.slots + (long long)slot * slot_floats(D);
        *reinterpret_cast<float4*>(dst + row * D + c) = acc;
        if (c == 0) {
          dst[16 * D + row] = top;
          dst[16 * D + 16 + row] = sum;
        }
      }
    }
    if (!whole && begin == 0 && threadIdx.x == 0) {
      // the item goes on in the CTAs up to the one that owns its last unit
      const long long last = u1 - w.left + units_cost(w.units) - 1;
      const int owner = (int)(((last + 1) * ctas + total - 1) / total) - 1;
      p.parts[cta] = Part{owner - cta + 1, w.b, w.head, w.tile};
    }
    next_item<ROWS>(p, w);
  }
}

// Joins the parts of the item that begins in CTA blockIdx.x and goes on in
// the next ones; one CTA a row, one thread a channel.
template <int D, int NT, typename T>
__global__ void __launch_bounds__(D) kv4_join_kernel(const __grid_constant__ Params p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Part part = p.parts[blockIdx.x];
  if (part.parts < 2) return;
  const int row = blockIdx.y, c = threadIdx.x;
  const Seq s = seq_of(p, part.seq);
  long long t;
  int h, i;
  if (!row_of(p, s, part.head, (long long)part.tile * 8 * NT + row, &t, &h, &i)) return;
  auto slot = [&](int k) {
    return p.slots + (long long)(k == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + k)) * slot_floats(D);
  };
  float top = -FLT_MAX;
  for (int k = 0; k < part.parts; ++k) top = fmaxf(top, slot(k)[16 * D + row]);
  float acc = 0.f, sum = 0.f;
#pragma unroll 4
  for (int k = 0; k < part.parts; ++k) {
    const float* x = slot(k);
    const float fac = exp2f(x[16 * D + row] - top);
    sum = fmaf(fac, x[16 * D + 16 + row], sum);
    acc = fmaf(fac, x[row * D + c], acc);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  T* dst = static_cast<T*>(p.a.o) + t * p.a.o_token + h * p.a.o_head + c;
  if constexpr (sizeof(T) == 4)
    *dst = acc * inv;
  else
    *dst = __float2bfloat16(acc * inv);
}

template <int D, int NT, int W, typename T>
int launch(const Params& p, cudaStream_t stream) {
  using C = Cfg<D, NT, W>;
  auto kern = kv4_attend_kernel<D, NT, W, T>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
    return SBSA_ERR_CUDA;
  int grid = sm_count();
  if (grid <= 0) return SBSA_ERR_CUDA;
  grid = grid < kMaxCtas ? grid : kMaxCtas;
  kern<<<grid, C::kThreads, C::kSmem, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return SBSA_ERR_CUDA;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid, 8 * NT);
  cfg.blockDim = dim3(D);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, NT, T>, p) == cudaSuccess ? SBSA_OK : SBSA_ERR_CUDA;
}

}  // namespace

size_t kv4_attend_workspace(int d) {
  return kMaxCtas * (2 * slot_floats(d) * sizeof(float) + sizeof(Part));
}

int launch_kv4_attend(const Kv4AttendArgs& a, cudaStream_t stream) {
  Params p{};
  p.a = a;
  p.heads = a.list_heads ? a.list_heads : a.b.hkv;
  p.group = a.hq / p.heads;
  p.kv_div = p.heads / a.b.hkv;
  p.scale_log2 = a.sm_scale * 1.4426950408889634f;
  p.slots = static_cast<float*>(a.workspace);
  p.parts = reinterpret_cast<Part*>(p.slots + (size_t)kMaxCtas * 2 * slot_floats(a.d));
  // 16 rows share a read of the cache where a sequence has more than 8
  const bool two = (long long)p.group * a.max_new > 8;
  if (a.dtype == SBSA_FP32)
    return a.d == 64 ? launch<64, 1, 8, float>(p, stream) : launch<128, 1, 8, float>(p, stream);
  if (a.d == 64)
    return two ? launch<64, 2, 8, __nv_bfloat16>(p, stream) : launch<64, 1, 12, __nv_bfloat16>(p, stream);
  return two ? launch<128, 2, 8, __nv_bfloat16>(p, stream) : launch<128, 1, 12, __nv_bfloat16>(p, stream);
}

}  // namespace sbsa
