// Attention over the 4-bit key-value cache for few rows: single tokens and
// drafts, and any number of rows in fp32.
//
// Mathematics.  With a key's group g of 32 channels as low + scale * n, a
// row's logit is  sum_g scale[t, g] (q_g . n[t, g]) + low[t, g] sum(q_g),  and
// its output  sum_t P[t] scale[t, g] n[t, c] + sum_t P[t] low[t, g]  over
// sum_t P[t]: the products take the levels n, and scales and lows enter per (row,
// token, group) in fp32.  A 4-bit level in the low bits of a 16-bit word is the
// fp16 denormal n 2^-24, exactly; at bit 4 it is 16 n 2^-24.  So a fragment
// register of two levels costs one AND (and half a shift), no conversion: the powers
// of two are folded into q and the output.  (The values' levels are taken less 8.)
//
// Bound: HBM, 5/4 d bytes a token and kv head.  At 6.5 TB/s an SM has about
// 110 cycles for 16 tokens (d = 128, 2560 bytes), and the work on them is
// about 370 warp instructions (93 issue cycles) at 8 rows and takes 155 cycles (524288 tokens of 8
// kv heads, 64 query heads: 163 us, 4.1 TB/s, among other calls for a second; in bursts of 12 ms,
// before the power limit lowers the clocks, 152, and without the arithmetic 122): levels must be
// unpacked with next to nothing, which rules out a copy in fp16 through shared
// memory for tcgen05 (its writes and reads alone would exceed the shared memory's
// bandwidth).  The products therefore run on mma.sync m16n8k16, whose
// operands are registers: S^T = K Q^T with 16 tokens as M and 8 query rows as N, and
// O^T = V^T P^T with 16 channels as M; in between the scaled weights are transposed
// (movmatrix), so that a lane holds scales and lows of two tokens, not four.
//
// The rows of one kv head (or listed query head) of a sequence, in tiles of
// kRows, are an item; an item's tokens fall into units of 128 (one stage).  The
// units of all items form one sequence, cut into equal runs, one for each CTA, so
// that ragged batches and single long contexts both fill the GPU.  A CTA walks its
// run: one warp copies whole pages (bulk copies, a ring of stages), 8 warps take
// 16 tokens of each stage.  At the end of an item's run the 8 warps join their
// partial results.  Of an item shared by several CTAs each leaves its part in the
// workspace, and the one that has its last unit joins them when it is done with its own
// run: it waits only for CTAs before it, which wait for nobody before they have left their
// parts; after a failure (a wait that ran out) nothing is joined, and the words that say what
// is there are left clean (kv4_ready.h).  (A second kernel for the joins cost a launch on the
// host, and on the GPU: 33 listed blocks of 8 sequences 24.6 us, 23.0 without; 524288 tokens
// 164, 159 at the time.)  Everything is in a fixed order: results do not change between runs.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <climits>
#include <type_traits>

#include "internal.h"
#include "kv4_ready.h"
#include "kv4_split.cuh"
#include "ptx.cuh"
#include "tma_map.h"

namespace sbsa {
namespace {

constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr int kUnit = kSplitUnit;  // tokens of a stage
// What an item costs a CTA besides its units (rows, joining, output), in units.
constexpr int kItemCost = 6;
// Weights are 2^(S - M), M = (reference of the logits) + (reference of the
// values' exponents) - kHead; each reference moves only when it is outgrown by more
// than kLazy, so the fp16 weights times a scale stay below 2^(kHead + 2 kLazy + 1) = 2^15.
constexpr float kHead = 6.f, kLazy = 4.f;

// 8 computing warps take the tiles of 16 TT tokens in turn; with two of them a
// scheduler the latency of a tile's chain (levels, products, weights, products) is what
// they wait for, so they take two tiles of 16 at once (one: 524288 tokens 185 us, two 153;
// drafts 78 and 73).  The copying warp and its
// three idle neighbours are a warpgroup whose registers the computing warps take
// over: 256 * 224 + 128 * 56 = 384 * 168, what the block is launched with.
constexpr int kWarps = 8;
constexpr int kThreads = (kWarps + 4) * 32;
constexpr int kRegs = 224, kRegsCopy = 56;

template <int D, int NT>
struct Cfg {
  static constexpr int kSub = 2;                  // TT
  static constexpr int kTile = 16 * kSub;         // tokens of a warp's step
  static constexpr int kTiles = kUnit / kTile;    // of a stage
  static constexpr int kRows = 8 * NT;
  static constexpr int kGroups = D / 32;
  static constexpr int kStageBytes = kUnit * (D / 8) * 10;
  static constexpr int kStages = D == 64 ? 10 : 7;
  static constexpr int kOutStride = D + 4;  // floats; spreads the heads over the banks
  static constexpr int kOffOut = kStages * kStageBytes;
  static constexpr int kOffStat = kOffOut + kWarps * kRows * kOutStride * 4;
  // per warp and row: M, l, and the lows' sums of the groups
  static constexpr int kStat = 2 + kGroups;
  static constexpr int kOffMeta = kOffStat + kWarps * kRows * kStat * 4;
  static constexpr int kOffScan = kOffMeta + kStages * 8 * 4;
  static constexpr int kOffBar = kOffScan + kScanBytes<kThreads>;
  static constexpr int kSmem = kOffBar + 2 * kStages * 8 + 16;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static_assert(kOffBar % 8 == 0 && kOffScan % 8 == 0, "alignment");
};

constexpr int kSlotRows = 16;

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
// Transpose of an 8 x 8 matrix of 16-bit elements (row lane / 4, columns 2 (lane % 4) and the next).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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

// Two levels (the bits in MASK, times 16 in the upper one) less N.  As fp16 denormals, in units
// of 2^-24, they cost an AND and an exact subtraction; but the tensor cores align products by
// the operands' exponents, and a denormal's leading zeros are then missing at the other end:
// 18 bits are left of a sum.  That is enough for bf16 rows.  For fp32 rows (kExact) they are made
// normal numbers: OR into the mantissa of 1024 before the subtraction.
template <bool kExact, uint32_t MASK, int N>
__device__ __forceinline__ uint32_t less(uint32_t x) {
  uint32_t y = x & MASK;
  if (!kExact && N == 0) return y;
  if (kExact) y |= 0x64006400u;
  const __half n = __ushort_as_half((unsigned short)((kExact ? 0x6400 : 0) + N));
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&y), __half2half2(n));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ float scale_of(uint32_t pair) { return __uint_as_float(pair << 16); }
__device__ __forceinline__ float low_of(uint32_t pair) {
  return __uint_as_float(pair & 0xFFFF0000u);
}
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

// Tiles of 16 tokens: the page's keys, the tile's first token there, its position.
template <int TT>
struct Tiles {
  const unsigned char* base[TT];
  int row[TT], pos[TT];
};

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
// A word of kv4_ready.h in the workspace.
struct ReadyWord {
  uint64_t* at;
  __device__ uint64_t load() const {
    uint64_t x;
    asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(x) : "l"(at) : "memory");
    return x;
  }
  __device__ uint64_t exchange(uint64_t x) const {
    uint64_t old;
    asm volatile("atom.exch.acq_rel.gpu.global.b64 %0, [%1], %2;" : "=l"(old) : "l"(at), "l"(x) : "memory");
    return old;
  }
  __device__ void store(uint64_t x) const {
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(at), "l"(x) : "memory");
  }
};

template <int THREADS>
__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// T: type of q and o.  fp32 rows enter the products as two fp16 parts (22
// bits), and so do their weights; a bf16 row is one fp16 part exactly (its
// elements are scaled by a power of two so that the largest is near 2^10) and
// the weights are rounded to fp16 once, 2^-11 of each.
template <int D, int NT, typename T>
__global__ void __launch_bounds__(kThreads, 1) kv4_attend_kernel(const __grid_constant__ SplitParams p) {
  using C = Cfg<D, NT>;
  constexpr int NG = C::kGroups;
  constexpr int ROWS = C::kRows;
  constexpr int PARTS = sizeof(T) == 4 ? 2 : 1;
  constexpr int TT = C::kSub;
  constexpr bool kExact = PARTS == 2;
  constexpr int kUnitLog2 = kExact ? 0 : 24;  // levels enter the products in units of 2^-kUnitLog2
  extern __shared__ __align__(128) unsigned char smem[];
  float* s_out = reinterpret_cast<float*>(smem + C::kOffOut);
  float* s_stat = reinterpret_cast<float*>(smem + C::kOffStat);
  int* s_meta = reinterpret_cast<int*>(smem + C::kOffMeta);  // [stage][page]: first token's position
  long long* s_scan = reinterpret_cast<long long*>(smem + C::kOffScan);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* empty = full + C::kStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + C::kStages);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int page = p.a.b.page, rec = kv4_rec_bytes(page, D);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], C::kTiles);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  Run run;
  if (!split_run<ROWS, kItemCost, kThreads>(p, s_scan, &run)) return;
  SplitWalk<ROWS, kItemCost> w(p, run);
  const int cta = blockIdx.x;

  auto fail = [&]() {
    *abort_flag = 1;
    if (p.a.b.status) atomicCAS(p.a.b.status, 0, SBSA_ERR_TIMEOUT);
  };

  if (warp >= kWarps) {
    regs_lower<kRegsCopy>();
    if (warp > kWarps) return;
    // ================================================================ copies
    const int page_log = __ffs(page) - 1, block_log = __ffs(p.a.block) - 1;  // powers of two
    const int pages = kUnit >> page_log;
    int n = 0;  // stages filled
    bool ok = true;
    for (; w.more() && ok; w.next(p)) {
      const Seq s = w.seq;
      const int begin = w.begin(), end = w.end();
      const int limit = w.limit(), len = s.len(p);
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
        long long at = (long long)(first + lane) << page_log;
        *pos = INT_MAX - kUnit;
        if (list) {
          const int e = (int)(at >> block_log);
          if (e >= count) return -1;
          const int j = list[e];
          if (j < 0 || j > (len - 1) >> block_log || len == 0) {
            kv4_record(p.a.b.status);
            return -1;
          }
          at = (j << block_log) + (at & (p.a.block - 1));
        }
        if (at >= limit) return -1;
        const int pg = table[at >> page_log];
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
  regs_raise<kRegs>();
  const int r = lane >> 2, q = lane & 3;
  // Row r of the first product is token r ^ (r >> 2) of 8: with it neither the keys' nor the values'
  // reads meet a bank twice.  A lane has the keys and weights of tokens tok and tok + 8 of a tile, and
  // the values of the tokens of rows 2q and 2q + 1.
  const int tok = r ^ (r >> 2);
  const int tok_a = (2 * q) ^ (q >> 1), tok_b = (2 * q + 1) ^ (q >> 1);
  // this warp's next tile, and its stage's number and place in the ring
  int tile = warp, stage = 0, st = 0, phase = 0;
  int base_n = 0;                    // the number of the item's first stage
  const int page_log = __ffs(page) - 1;
  bool ok = true;
  // The 8 warps' partial rows, in shared memory, together: to o, or to a slot.
  auto merge = [&](const Seq& s, int head, uint32_t row0, int slot) {
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
      if (slot < 0) {
        long long t;
        int h, i;
        if (row_of(p, s, head, row0 + row, &t, &h, &i)) {
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          store4(static_cast<T*>(p.a.o) + t * p.a.o_token + h * p.a.o_head + c,
                 make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
        }
      } else {
        float* dst = p.slots + (long long)slot * slot_floats(kSlotRows, D);
        *reinterpret_cast<float4*>(dst + row * D + c) = acc;
        if (c == 0) {
          dst[kSlotRows * D + row] = top;
          dst[kSlotRows * (D + 1) + row] = sum;
        }
      }
    }
  };
  // the item that ends in this CTA but begins in an earlier one
  Seq join_seq{};
  int join_head = 0, join_first = -1;
  uint32_t join_row0 = 0;
  for (; w.more(); w.next(p)) {
    const Seq s = w.seq;
    const int begin = w.begin(), end = w.end();
    const uint32_t row0 = (uint32_t)w.tile * ROWS;

    // ---- the query rows as fragments: elements (0, 4), (1, 5)/16, (2, 6), (3, 7)/16 of each 8
    // channels, as the levels come out of a word
    uint32_t bq[NT][PARTS][NG][2][2];
    // sum(q_g) (in the products' unit) in three bf16 parts, against the lows of two groups a lane: with 4 groups
    // k-pairs q = 0, 1 hold the first part of groups (0, 1) and (2, 3), 2 and 3 the second, 8 behind
    // them the third; with 2 groups q = 0, 1, 2 hold the three parts
    uint32_t bl[NT][2];
    // of rows 2q and 2q + 1: the factor of the logits, and the first token that is not seen
    float f[NT][2];
    int lim[NT][2];
    int lim_min = INT_MAX, lim_max = 0;
#pragma unroll
    for (int x = 0; x < NT; ++x) {
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
      // (positive: -inf * 0, a masked logit's, would be NaN)
      const float fr = fmaxf(p.scale_log2 * __uint_as_float((uint32_t)(kUnitLog2 - e + 127) << 23), 0x1p-126f);
      // rows that see nothing (out of the sequence's range, beyond max_new) mask all; rows past the
      // tile's last mask nothing, so that they never send the warp to the masked path
      int lr = INT_MAX;
      if (have) {
        lr = i < p.a.max_new ? s.visible(p, i) : 0;
        if (lr == 0 && q == 0) kv4_record(p.a.b.status);
        lim_min = min(lim_min, lr);
        lim_max = max(lim_max, lr);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        f[x][c] = __shfl_sync(0xFFFFFFFFu, fr, 8 * q + 4 * c);
        lim[x][c] = __shfl_sync(0xFFFFFFFFu, lr, 8 * q + 4 * c);
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
        qs[g] = sum * (kUnitLog2 ? 0x1p-24f : 1.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float sc = (j & 1) ? 0.0625f : 1.f;
          const float lo = v[g][j] * sc, hi = v[g][j + 4] * sc;
          const uint32_t h0 = pack_half2(lo, hi);
          bq[x][0][g][j >> 1][j & 1] = h0;
          if constexpr (PARTS == 2) {
            const __half2 back = *reinterpret_cast<const __half2*>(&h0);
            bq[x][PARTS - 1][g][j >> 1][j & 1] =
                pack_half2(lo - __low2float(back), hi - __high2float(back));
          }
        }
      }
      if constexpr (NG == 4) {
        float u = (q & 1) ? qs[2] : qs[0], w2 = (q & 1) ? qs[3] : qs[1];
        const uint32_t p0 = take_bf16(u, w2), p1 = take_bf16(u, w2), p2 = take_bf16(u, w2);
        bl[x][0] = q < 2 ? p0 : p1;
        bl[x][1] = q < 2 ? p2 : 0;
      } else {
        float u = qs[0], w2 = qs[1];
        const uint32_t p0 = take_bf16(u, w2), p1 = take_bf16(u, w2), p2 = take_bf16(u, w2);
        bl[x][0] = q == 0 ? p0 : q == 1 ? p1 : q == 2 ? p2 : 0;
        bl[x][1] = 0;
      }
    }
    lim_min = __reduce_min_sync(0xFFFFFFFFu, lim_min);
    lim_max = __reduce_max_sync(0xFFFFFFFFu, lim_max);
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (lim[x][c] == INT_MAX) lim[x][c] = lim_max;

    // rows' references: ms for the logits, me (an exponent as bf16 holds it) for the magnitude of the
    // values, common to all rows; weights are 2^(logit - m), m = ms + (me - 127) - kHead.
    // o: outputs; ol: the sums of this lane's tokens' low + 8 scale, l: of their weights
    float o[NT][NG][2][4], ol[NT][NG][2], l[NT][2], m[NT][2], ms[NT][2];
    uint32_t me = 0, big = 0;
#pragma unroll
    for (int x = 0; x < NT; ++x) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        m[x][c] = ms[x][c] = -FLT_MAX;
        l[x][c] = 0.f;
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        ol[x][g][0] = ol[x][g][1] = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[x][g][j][c] = 0.f;
      }
    }

    // ---- one step: TT tiles of 16 tokens; base and row: the page's keys and the tile's first
    // token there.  kMask: some row does not see all of them.
    auto step = [&](const Tiles<TT>& at, auto mask_tag) {
      constexpr bool kMask = decltype(mask_tag)::value;
      uint32_t top = 0;  // the largest magnitude of a scale or low that this lane looks at
      float sv[TT][NT][4];  // logits (without f): token tok for rows 2q, 2q + 1, then token tok + 8
      Words<NG> pv[TT][2];
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) {
        const unsigned char* kl = at.base[tt] + at.row[tt] * (D / 2);
        const unsigned char* kp = at.base[tt] + page * (D / 2) + at.row[tt] * (D / 8);
        const unsigned char* vp = kp + rec;
        const Words<NG> w0 = lds_words<NG>(kl + tok * (D / 2) + q * (D / 8));
        const Words<NG> w1 = lds_words<NG>(kl + (8 + tok) * (D / 2) + q * (D / 8));
        const Words<NG> p0 = lds_words<NG>(kp + tok * (D / 8));
        const Words<NG> p1 = lds_words<NG>(kp + (8 + tok) * (D / 8));
        pv[tt][0] = lds_words<NG>(vp + tok * (D / 8));
        pv[tt][1] = lds_words<NG>(vp + (8 + tok) * (D / 8));
        const Words<NG / 2> e = lds_words<NG / 2>(vp + lane * (D / 16));
        const bool in = !kMask || at.pos[tt] + (lane >> 1) < lim_max;
#pragma unroll
        for (int g = 0; g < NG / 2; ++g)
          if (in) top = __vmaxu2(top, e.w[g] & 0x7FFF7FFFu);
        uint32_t a[4];
        a[0] = __byte_perm(p0.w[0], p0.w[1], 0x7632);
        a[1] = __byte_perm(p1.w[0], p1.w[1], 0x7632);
        if constexpr (NG == 4) {
          if (q & 1) {
            a[0] = __byte_perm(p0.w[NG - 2], p0.w[NG - 1], 0x7632);
            a[1] = __byte_perm(p1.w[NG - 2], p1.w[NG - 1], 0x7632);
          }
        }
        a[2] = a[0];
        a[3] = a[1];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_bf16_first(sv[tt][nt], a, bl[nt][0], bl[nt][1]);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const uint32_t x0 = w0.w[g], x1 = w1.w[g], y0 = x0 >> 8, y1 = x1 >> 8;
          const uint32_t f0[4] = {less<kExact, 0x000F000Fu, 0>(x0), less<kExact, 0x000F000Fu, 0>(x1),
                                  less<kExact, 0x00F000F0u, 0>(x0), less<kExact, 0x00F000F0u, 0>(x1)};
          const uint32_t f1[4] = {less<kExact, 0x000F000Fu, 0>(y0), less<kExact, 0x000F000Fu, 0>(y1),
                                  less<kExact, 0x00F000F0u, 0>(y0), less<kExact, 0x00F000F0u, 0>(y1)};
          const float s0 = scale_of(p0.w[g]), s1 = scale_of(p1.w[g]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float d[4];
            mma_f16_first(d, f0, bq[nt][0][g][0][0], bq[nt][0][g][0][1]);
            mma_f16(d, f1, bq[nt][0][g][1][0], bq[nt][0][g][1][1]);
            if constexpr (PARTS == 2) {
              mma_f16(d, f0, bq[nt][PARTS - 1][g][0][0], bq[nt][PARTS - 1][g][0][1]);
              mma_f16(d, f1, bq[nt][PARTS - 1][g][1][0], bq[nt][PARTS - 1][g][1][1]);
            }
            sv[tt][nt][0] = fmaf(s0, d[0], sv[tt][nt][0]);
            sv[tt][nt][1] = fmaf(s0, d[1], sv[tt][nt][1]);
            sv[tt][nt][2] = fmaf(s1, d[2], sv[tt][nt][2]);
            sv[tt][nt][3] = fmaf(s1, d[3], sv[tt][nt][3]);
          }
        }
        if constexpr (kMask) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (at.pos[tt] + tok + (c >> 1) * 8 >= lim[nt][c & 1]) sv[tt][nt][c] = -INFINITY;
        }
      }
      // ---- the references, moved only when they have to
      bool need = __vmaxu2(top, big) != big;
      float mx[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float x = fmaxf(sv[0][nt][c], sv[0][nt][2 + c]);
          if constexpr (TT == 2) x = fmaxf(x, fmaxf(sv[TT - 1][nt][c], sv[TT - 1][nt][2 + c]));
          mx[nt][c] = x * f[nt][c];
          need |= mx[nt][c] > ms[nt][c] + kLazy;
        }
      if (__any_sync(0xFFFFFFFFu, need)) {
        uint32_t e = 0;
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
          const Words<NG / 2> w2 =
              lds_words<NG / 2>(at.base[tt] + rec + page * (D / 2) + at.row[tt] * (D / 8) + lane * (D / 16));
          if (kMask && at.pos[tt] + (lane >> 1) >= lim_max) continue;
#pragma unroll
          for (int g = 0; g < NG / 2; ++g) {  // NaN groups say nothing
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
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float mn = mx[nt][c];
            mn = fmaxf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, 4));
            mn = fmaxf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, 8));
            mn = fmaxf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, 16));
            mn = fmaxf(mn, ms[nt][c]);
            const float alpha = exp2f(ms[nt][c] - mn - de);
            ms[nt][c] = mn;
            m[nt][c] = mn + ((float)((int)me - 127) - kHead);
            l[nt][c] *= alpha;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
              ol[nt][g][c] *= alpha;
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                o[nt][g][j][c] *= alpha;
                o[nt][g][j][2 + c] *= alpha;
              }
            }
          }
      }
      // ---- weights and values
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) {
        const unsigned char* vl =
            at.base[tt] + rec + at.row[tt] * (D / 2) + (r ^ (NG == 4 ? (q & 1) * 4 : 0)) * (D / 16);
        const Words<NG / 2> va0 = lds_words<NG / 2>(vl + tok_a * (D / 2));
        const Words<NG / 2> vb0 = lds_words<NG / 2>(vl + tok_b * (D / 2));
        const Words<NG / 2> va1 = lds_words<NG / 2>(vl + (8 + tok_a) * (D / 2));
        const Words<NG / 2> vb1 = lds_words<NG / 2>(vl + (8 + tok_b) * (D / 2));
        float pw[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            pw[nt][c] = ex2_approx(fmaf(sv[tt][nt][c], f[nt][c & 1], -m[nt][c & 1]));
            l[nt][c & 1] += pw[nt][c];
          }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const uint32_t sel = (g & 1) ? 0x7632u : 0x5410u;
          const uint32_t x0 = __byte_perm(va0.w[g >> 1], vb0.w[g >> 1], sel), y0 = x0 >> 8;
          const uint32_t x1 = __byte_perm(va1.w[g >> 1], vb1.w[g >> 1], sel), y1 = x1 >> 8;
          // level - 8, and the lows' sums below take low + 8 scale: the levels alone would make
          // sums that only grow, which the tensor cores cut off at every step and the lows then
          // cancel (over 500,000 tokens 5e-6 of the values, three times the output's rounding)
          const uint32_t f0[4] = {less<kExact, 0x000F000Fu, 8>(x0), less<kExact, 0x00F000F0u, 128>(x0),
                                  less<kExact, 0x000F000Fu, 8>(x1), less<kExact, 0x00F000F0u, 128>(x1)};
          const uint32_t f1[4] = {less<kExact, 0x000F000Fu, 8>(y0), less<kExact, 0x00F000F0u, 128>(y0),
                                  less<kExact, 0x000F000Fu, 8>(y1), less<kExact, 0x00F000F0u, 128>(y1)};
          const float sc[2] = {scale_of(pv[tt][0].w[g]), scale_of(pv[tt][1].w[g])};
          const float lw[2] = {fmaf(8.f, sc[0], low_of(pv[tt][0].w[g])),
                               fmaf(8.f, sc[1], low_of(pv[tt][1].w[g]))};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float x[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              x[c] = pw[nt][c] * sc[c >> 1];
              if constexpr (kMask) {  // 0 * NaN in a hidden place
                const bool hidden = at.pos[tt] + tok + (c >> 1) * 8 >= lim[nt][c & 1];
                if (hidden) x[c] = 0.f;
                if (!hidden) ol[nt][g][c & 1] = fmaf(pw[nt][c], lw[c >> 1], ol[nt][g][c & 1]);
              } else {
                ol[nt][g][c & 1] = fmaf(pw[nt][c], lw[c >> 1], ol[nt][g][c & 1]);
              }
            }
            const uint32_t h0 = pack_half2(x[0], x[1]), h1 = pack_half2(x[2], x[3]);
            const uint32_t b0 = transpose8(h0), b1 = transpose8(h1);
            mma_f16(o[nt][g][0], f0, b0, b1);
            mma_f16(o[nt][g][1], f1, b0, b1);
            if constexpr (PARTS == 2) {
              const __half2 k0 = *reinterpret_cast<const __half2*>(&h0);
              const __half2 k1 = *reinterpret_cast<const __half2*>(&h1);
              const uint32_t c0 = transpose8(pack_half2(x[0] - __low2float(k0), x[1] - __high2float(k0)));
              const uint32_t c1 = transpose8(pack_half2(x[2] - __low2float(k1), x[3] - __high2float(k1)));
              mma_f16(o[nt][g][0], f0, c0, c1);
              mma_f16(o[nt][g][1], f1, c0, c1);
            }
          }
        }
      }
    };

    for (; tile / C::kTiles - base_n < end - begin; tile += kWarps) {
      st += tile / C::kTiles - stage;
      stage = tile / C::kTiles;
      if (st >= C::kStages) {
        st -= C::kStages;
        phase ^= 1;
      }
      if (ok) ok = mbar_wait_bounded(&full[st], phase, abort_flag, kTimeoutNs);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (ok) {
        Tiles<TT> x;
        bool all = true, some = false;
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
          const int at = tile % C::kTiles * C::kTile + tt * 16, pg = at >> page_log;
          x.row[tt] = at & (page - 1);
          x.pos[tt] = s_meta[st * 8 + pg] + x.row[tt];
          x.base[tt] = smem + st * C::kStageBytes + pg * 2 * rec;
          all = all && x.pos[tt] + 16 <= lim_min;
          some = some || x.pos[tt] < lim_max;
        }
        if (all)
          step(x, std::false_type{});
        else if (some)
          step(x, std::true_type{});
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
      }
    }
    base_n += end - begin;
    if (!ok && lane == 0 && !*abort_flag) fail();

    constexpr float kUnit = kExact ? 1.f : 0x1p24f;
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
              make_float4(o[nt][g][0][c] * kUnit, o[nt][g][0][2 + c] * (kUnit / 16),
                          o[nt][g][1][c] * kUnit, o[nt][g][1][2 + c] * (kUnit / 16));
        }
      }
      // the sums over the lanes' tokens
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x[NG + 1];
        x[0] = l[nt][c];
#pragma unroll
        for (int g = 0; g < NG; ++g) x[1 + g] = ol[nt][g][c];
        float* dst = s_stat + (warp * ROWS + nt * 8 + 2 * q + c) * C::kStat;
#pragma unroll
        for (int g = 0; g <= NG; ++g) {
          x[g] += __shfl_xor_sync(0xFFFFFFFFu, x[g], 4);
          x[g] += __shfl_xor_sync(0xFFFFFFFFu, x[g], 8);
          x[g] += __shfl_xor_sync(0xFFFFFFFFu, x[g], 16);
          if (r == 0) dst[1 + g] = x[g];
        }
        if (r == 0) dst[0] = m[nt][c];
      }
    }
    consumers_sync<kWarps * 32>();
    const int slot = 2 * cta + (begin == 0 ? 1 : 0);
    const bool whole = w.whole();
    merge(s, w.head, row0, whole ? -1 : slot);
    if (!whole) {
      __threadfence();
      if (end == w.unit_count) {  // joined at the end of the run
        join_seq = s, join_head = w.head, join_row0 = row0, join_first = w.first_cta(run);
      } else {
        consumers_sync<kWarps * 32>();
        if (threadIdx.x == 0) ready_publish(ReadyWord{p.ready + slot}, p.call, *abort_flag != 0);
      }
    }
  }

  // ==================================================================== joining
  if (join_first < 0) return;
  const int others = cta - join_first;
  auto slot_of = [&](int k) { return k == 0 ? 2 * join_first + 1 : 2 * (join_first + k); };
  if ((int)threadIdx.x < others) {
    const ReadyWord word{p.ready + slot_of(threadIdx.x)};
    const uint64_t t0 = global_timer_ns();
    Ready found = kReadyNot;
    while (ok && (found = ready_look(word, p.call)) == kReadyNot)
      ok = !*abort_flag && global_timer_ns() - t0 <= kTimeoutNs;
    ready_leave(word, p.call, found == kReadyNot);
    ok = found == kReadyPart;
  }
  if (bar_red_or(1, kWarps * 32, !ok)) {
    if (threadIdx.x == 0 && !*abort_flag) fail();
    return;
  }
  // the warps take the parts (the last one is this CTA's) in turn, and join like after an item
  constexpr int kPerRow = D / 4;              // lanes of a row, 4 channels each
  constexpr int kRowsWarp = 32 / kPerRow;     // rows of a warp's pass
  constexpr int kPasses = ROWS / kRowsWarp;
  float4 acc[kPasses];
  float sum[kPasses], top[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    sum[i] = 0.f;
    top[i] = -FLT_MAX;
  }
  const int c = lane % kPerRow * 4, row_w = lane / kPerRow;
  for (int k = warp; k <= others; k += kWarps) {
    const float* x = p.slots + (size_t)slot_of(k) * slot_floats(kSlotRows, D);
    float4 v[kPasses];
    float m[kPasses], l[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int row = i * kRowsWarp + row_w;
      v[i] = __ldcg(reinterpret_cast<const float4*>(x + row * D + c));
      m[i] = __ldcg(x + kSlotRows * D + row);
      l[i] = __ldcg(x + kSlotRows * (D + 1) + row);
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const float mn = fmaxf(top[i], m[i]);
      const float fa = exp2f(top[i] - mn), fb = exp2f(m[i] - mn);
      top[i] = mn;
      sum[i] = fmaf(sum[i], fa, l[i] * fb);
      acc[i].x = fmaf(acc[i].x, fa, v[i].x * fb);
      acc[i].y = fmaf(acc[i].y, fa, v[i].y * fb);
      acc[i].z = fmaf(acc[i].z, fa, v[i].z * fb);
      acc[i].w = fmaf(acc[i].w, fa, v[i].w * fb);
    }
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int row = i * kRowsWarp + row_w;
    *reinterpret_cast<float4*>(s_out + (warp * ROWS + row) * C::kOutStride + c) = acc[i];
    float* st = s_stat + (warp * ROWS + row) * C::kStat;
    if (c == 0) {
      st[0] = top[i];
      st[1] = sum[i];
#pragma unroll
      for (int g = 0; g < NG; ++g) st[2 + g] = 0.f;
    }
  }
  consumers_sync<kWarps * 32>();
  merge(join_seq, join_head, join_row0, -1);
}

template <int D, int NT, typename T>
int launch(const SplitParams& p, cudaStream_t stream) {
  using C = Cfg<D, NT>;
  auto kern = kv4_attend_kernel<D, NT, T>;
  static SplitGrid ctas;
  const int grid = ctas.get(reinterpret_cast<const void*>(kern), C::kSmem);
  if (grid <= 0) return SBSA_ERR_CUDA;
  kern<<<grid, kThreads, C::kSmem, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return SBSA_ERR_CUDA;
  return SBSA_OK;
}

}  // namespace

size_t kv4_few_workspace(const Kv4AttendArgs& a) {
  return split_possible(a) ? split_workspace(kSlotRows, a.d) : 0;
}

int launch_kv4_few(const Kv4AttendArgs& a, cudaStream_t stream) {
  SplitParams p = split_params(a, kSlotRows);
  p.call = call_number();
  // 16 rows share a read of the cache where a sequence has more than 8
  const bool two = (long long)p.group * a.max_new > 8;
  if (a.dtype == SBSA_FP32)
    return a.d == 64 ? launch<64, 1, float>(p, stream) : launch<128, 1, float>(p, stream);
  if (a.d == 64)
    return two ? launch<64, 2, __nv_bfloat16>(p, stream) : launch<64, 1, __nv_bfloat16>(p, stream);
  return two ? launch<128, 2, __nv_bfloat16>(p, stream) : launch<128, 1, __nv_bfloat16>(p, stream);
}

}  // namespace sbsa
