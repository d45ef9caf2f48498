// Attention over the 4-bit key-value cache for many rows (chunks of prompts),
// bf16, on tcgen05.
//
// Mathematics.  Keys and values are taken back to fp16 once a tile of 128 tokens
// and used for 256 rows (two query tiles A and B of 128: tokens by query heads of a
// kv head): S = Q K^T, exact online softmax, O += P V.  In fp16 a value stands for
// (low' + scale' n), with low' and scale' scaled by a power of two so that scale' stays
// below 2^-8 and low' below 2^14: a level in the low bits of a half is the fp16 denormal
// n 2^-24, and one fused multiply-add by scale' 2^24 (2^20 where the level stands at bit
// 4) gives the value, rounded once, 2^-11 of it.  Where low' or the value is an fp16
// denormal itself, each is off by up to 2^-25, together 2^-15 of the largest scale that the
// power of two goes by (or 2^-37 of the largest low, when that is above 2^22 scales): for keys
// it is that of the tile's 128 tokens, all groups; for values each group has its own, the
// largest of the item's tokens so far.  q's rows are scaled to fp16 exactly.  The powers of
// two go into the logits' factor and, for the values, into the rescaling of O's columns.
//
// Bound: the tensor cores and the exponentials alike.  A tile of 128 tokens against 256
// rows is 2 * 2 * 2^21 multiply-adds, 2096 cycles at 4000 a cycle, its 2^15 exponentials
// 2048 cycles at 16 a cycle.  Neither is reached: 4096 new of 32768 tokens, 32 query heads on 8,
// 2.26 ms among other calls for a second (912 TFLOP/s, 0.66 of what cuBLAS holds that long: the
// power limit lowers the clocks); in bursts of 12 ms 2.07 ms (998 TFLOP/s, 0.60 of cuBLAS's burst).
// The parts below were measured in short runs on the form that took 2.00 to 2.05 (one unit for
// all groups of the values): about 4,400 cycles a token tile, softmax
// 2,700 of them and 1,500 of waiting for the products, unpacking 3,300 and 1,100 of waiting.  No
// single role is what the others wait for: without the exponentials 2.00 ms, without the unpacking
// loops 1.86, with a quarter of the products 1.91.  (S in halves of 64 tokens, so that softmax and
// products of a query tile overlap, takes 48 products a token tile instead of 32, which read 192
// bytes a cycle of shared memory: 3.3 ms, with an issuing thread for each query tile 2.1.)
// Four roles at a time share the instruction caches, so their loops are kept short (unroll 1 where
// it stands): all unrolled, 2.5 of the 12 warp cycles that an issued instruction cost were spent
// waiting for instructions (then 0.44 of 8.4, now 0.65) and the same call took 2.78 ms; with the
// unpacking loops short 2.25.  The softmax reads S twice out of TMEM, 64 columns at a time, for the
// same reason, and then needs so few registers that hardly anything spills (2.05).  How the
// compiler lays the roles out is worth up to 5 % of it either way.
//
// One CTA an SM, 16 warps:
//   0-3, 4-7  softmax of tile A, of tile B: a thread has a row; S out of TMEM, P (fp16)
//             back over its first half; the reference maximum moves (and O is
//             rescaled in TMEM) only when it is outgrown by 2^8.  They write their
//             tile's Q into shared memory and O to global memory.
//   8-11      a thread has a token of the tile: takes its levels from a ring of three
//             half tiles (keys or values) and writes its K and V rows into the swizzled layout
//             of the products' operands (two buffers each; the channels in the order in
//             which they come out of the words, which Q and the output follow).
//   12        issues the products: [PV_A(j-1), S_A(j)], [PV_B(j-1), S_B(j)], ...; one
//             commit each announces S, that the O of the tile is at rest, and (B's) that
//             K(j) and V(j-1) are free again.
//   13        copies whole pages into the ring (bulk copies).
// The items and their cut over the CTAs: kv4_split.cuh.  Every wait is bounded (2 s).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <climits>

#include "internal.h"
#include "kv4_split.cuh"
#include "ptx.cuh"

namespace sbsa {
namespace {

constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr int kRows = 256;  // of an item: two tiles of 128
constexpr int kItemCost = 5;
constexpr int kThreads = 512;
// What the block is launched with, 512 * 128, divided anew.  The issuing thread's loop spills below 96
// (88: 150 bytes, 80: 230, 72: 500), which shows in every token tile.
constexpr int kRegsSoftmax = 144, kRegsUnpack = 128, kRegsIssue = 96;
static_assert(256 * kRegsSoftmax + 128 * (kRegsUnpack + kRegsIssue) <= kThreads * 128 && kRegsSoftmax >= 128 &&
                  kRegsUnpack <= 128 && kRegsIssue <= 128,
              "the softmax warps' share is raised from 128, the others' are lowered");
constexpr float kRescaleLog2 = 8.0f;
// Weights are 2^(logit - m + kHeadLog2), m a reference that the logits outgrow by 2^8 at most: below
// 2^15 in fp16, and those down to 2^-21 of the largest are normal numbers.
constexpr float kHeadLog2 = 7.0f;
constexpr float kLeastFactor = 0x1p-126f, kMostFactor = 0x1p80f;  // (|S'| is below 2^32)

constexpr int kHalves = 3;

template <int D>
struct MC {
  static constexpr int NG = D / 32;
  static constexpr int kTileBytes = 128 * D * 2;   // of Q, K or V
  static constexpr int kOffQ = 0;                  // Q[2]
  static constexpr int kOffK = 2 * kTileBytes;     // K[2]
  static constexpr int kOffV = 4 * kTileBytes;     // V[2]
  static constexpr int kHalfBytes = 128 * (D / 8) * 5;  // levels and pairs of 128 keys (or values)
  static constexpr int kOffRing = 6 * kTileBytes;       // [kHalves]
  static constexpr int kOffInfo = kOffRing + kHalves * kHalfBytes;  // Info[4]
  static constexpr int kInfoBytes = 32;
  static constexpr int kOffNan = kOffInfo + 4 * kInfoBytes;  // int[4 items][4 groups]
  static constexpr int kOffMax = kOffNan + 64;               // uint32[2 parities][4 warps][2]
  static constexpr int kOffPages = kOffMax + 64;             // int[kHalves][8]: the pages' numbers
  static constexpr int kOffScan = kOffPages + kHalves * 32;
  static constexpr int kOffBar = kOffScan + kScanBytes<kThreads>;
  // q_full[2] k_full[2] v_full[2] s_bar[2][2] o_bar[2][2] p_full[2] p_half[2] drain c_full[3]
  // c_free[3]
  static constexpr int kBars = 2 + 2 + 2 + 4 + 4 + 2 + 2 + 1 + 2 * kHalves;
  static constexpr int kOffMisc = kOffBar + kBars * 8;
  static constexpr int kSmem = kOffMisc + 16 + 1024;
  static constexpr uint32_t kDescS = make_idesc(0, 128, 128, false, false);
  static constexpr uint32_t kDescO = make_idesc(0, 128, D, false, true);
  static constexpr int kTmO = 256;  // TMEM: S_A, S_B (128 columns each), O_A, O_B (D each)
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static_assert(kOffScan % 8 == 0 && kOffBar % 8 == 0, "alignment");
};

// What the softmax has to know of a tile of tokens.
struct Info {
  float k_unit[2];   // logits are S' * both (powers of two) * the row's factor
  uint32_t v_exp;    // O's units after this tile: a byte e for each group, 2^(e - 118)
  uint32_t on[4];    // tokens whose page is in the cache
  int pad;
};
static_assert(sizeof(Info) == 32, "Info");

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// What a group's power of two has to reach: the larger of its scale and 2^-22 of its low, as bf16
// holds it; 0 for a NaN group.
__device__ __forceinline__ uint32_t reach(uint32_t pair) {
  const int scale = pair & 0x7FFFu, low = (pair >> 16) & 0x7FFFu;
  return scale >= 0x7F80 || low >= 0x7F80 ? 0u : (uint32_t)max(scale, low - (22 << 7));
}
// The power of two that byte g of v_exp stands for.
__device__ __forceinline__ int unit_exp(uint32_t bytes, int g) {
  return (int)((bytes >> (8 * g)) & 255u) - 118;
}

__device__ __forceinline__ uint32_t h2(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }
__device__ __forceinline__ __half2 as_h2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }

// Eight channels of a word of levels as fp16 values, in the order 0 4 1 5 2 6 3 7:
// the halves hold channels i and i + 4, with scale (2^24, and 2^20 for the odd i) and low.
__device__ __forceinline__ uint4 unpack8(uint32_t x, __half2 se, __half2 so, __half2 lo) {
  const uint32_t y = x >> 8;
  uint4 r;
  r.x = h2(__hfma2(as_h2(x & 0x000F000Fu), se, lo));
  r.y = h2(__hfma2(as_h2(x & 0x00F000F0u), so, lo));
  r.z = h2(__hfma2(as_h2(y & 0x000F000Fu), se, lo));
  r.w = h2(__hfma2(as_h2(y & 0x00F000F0u), so, lo));
  return r;
}

// Pairs of fp32 values in one 64-bit register.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Offset of chunk c (8 elements) of row `row` in a tile of 128 rows.
__device__ __forceinline__ int chunk_at(int row, int c) {
  return (c >> 3) * (128 * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
}

// Group of place y of O (or k + y, k a multiple of 16).
template <int NG>
__device__ __forceinline__ constexpr int group_of(int y) {
  return NG == 4 ? 2 * ((y >> 3) & 1) + (y & 1) : (y & 1);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv4_many_kernel(const __grid_constant__ SplitParams p) {
  using C = MC<D>;
  constexpr int NG = C::NG;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* q_full = bar;          // [tile]
  uint64_t* k_full = bar + 2;      // [token tile & 1]
  uint64_t* v_full = bar + 4;
  uint64_t* s_bar = bar + 6;       // [tile * 2 + (token tile & 1)]: S(j) and PV(j - 1) done
  uint64_t* o_bar = bar + 10;      // [tile * 2 + (item & 1)]: the item's last PV done
  uint64_t* p_full = bar + 14;     // [tile]
  uint64_t* p_half = bar + 16;     // [tile]: the weights of the first 64 tokens
  uint64_t* drain = bar + 18;
  uint64_t* c_full = bar + 19;     // [half tile % kHalves]
  uint64_t* c_free = c_full + kHalves;
  int* s_pages = reinterpret_cast<int*>(smem + C::kOffPages);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  Info* info = reinterpret_cast<Info*>(smem + C::kOffInfo);
  int* nan_pos = reinterpret_cast<int*>(smem + C::kOffNan);
  uint32_t* s_max = reinterpret_cast<uint32_t*>(smem + C::kOffMax);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 128);
      mbar_init(&k_full[i], 128);
      mbar_init(&v_full[i], 128);
      mbar_init(&p_full[i], 128);
      mbar_init(&p_half[i], 128);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_bar[i], 1);
      mbar_init(&o_bar[i], 1);
    }
    for (int i = 0; i < kHalves; ++i) {
      mbar_init(&c_full[i], 1);
      mbar_init(&c_free[i], 128);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (threadIdx.x == 0) p.parts[blockIdx.x].parts = 0;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the joining kernel may start up
  Run run;
  if (!split_run<kRows, kItemCost, kThreads>(p, reinterpret_cast<long long*>(smem + C::kOffScan), &run))
    return;
  if (warp == 12) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int cta = blockIdx.x;
  SplitWalk<kRows, kItemCost> w(p, run);

  auto fail = [&]() {
    *abort_flag = 1;
    if (p.a.b.status) atomicCAS(p.a.b.status, 0, SBSA_ERR_TIMEOUT);
  };
  auto wait = [&](uint64_t* b, uint32_t parity) {
    return mbar_wait_bounded(b, parity, abort_flag, kTimeoutNs);
  };
  // rows of the item (past the last sequence row: none) and whether it has a tile B
  auto item_rows = [&]() {
    return (int)min((uint32_t)kRows, (uint32_t)w.seq.rows * (uint32_t)p.group - (uint32_t)w.tile * kRows);
  };

  if (warp < 8) {
    // ================================================================ softmax
    regs_raise<kRegsSoftmax>();
    const int x = warp >> 2;  // which tile
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lanes + x * 128;
    const uint32_t o_col = tmem + lanes + C::kTmO + x * D;
    int n = 0, item = 0;  // token tiles and items so far
    bool ok = true;
    for (; w.more() && ok; w.next(p), ++item) {
      const int begin = w.begin(), end = w.end();
      const int rows = item_rows();
      if (x == 1 && rows <= 128) {
        // no tile B: its warps keep in step with its barriers (a wait for a phase that is more
        // than one away from the current one would take one for the other)
        for (int j = begin; ok && j < end; ++j, ++n) {
          ok = __all_sync(0xFFFFFFFFu, wait(&s_bar[2 + (n & 1)], (n >> 1) & 1));
          if (ok) mbar_arrive(&p_full[1]);
        }
        if (ok) ok = __all_sync(0xFFFFFFFFu, wait(&o_bar[2 + (item & 1)], (item >> 1) & 1));
        continue;
      }
      long long t = 0;
      int h = 0, i = 0;
      const bool have = row_of(p, w.seq, w.head, (uint32_t)w.tile * kRows + x * 128 + row, &t, &h, &i);
      // ---- Q: the row in fp16, scaled by a power of two to a largest element near 2^10
      int lim = w.limit();  // rows past the last see all, so that they never mask
      if (have) {
        lim = i < p.a.max_new ? w.seq.visible(p, i) : 0;
        if (lim == 0) kv4_record(p.a.b.status);
      }
      float f;
      {
        uint4 u[D / 8];
        float mx = 0.f;
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const __nv_bfloat16*>(p.a.q.ptr) + t * p.a.q.token + h * p.a.q.head);
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          u[c] = have ? src[c] : make_uint4(0, 0, 0, 0);
          const uint32_t v[4] = {u[c].x, u[c].y, u[c].z, u[c].w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(v[k] << 16)),
                                 fabsf(__uint_as_float(v[k] & 0xFFFF0000u))));
        }
        const int e = clamp_int(137 - (int)(__float_as_uint(mx) >> 23), -90, 100);
        const float up = __uint_as_float((uint32_t)(e + 127) << 23);
        f = p.scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23);
        unsigned char* dst = smem + C::kOffQ + x * C::kTileBytes;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {  // 8 channels 32 g + 8 q: chunk q NG + g
          const uint32_t v[4] = {u[c].x, u[c].y, u[c].z, u[c].w};
          float z[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            z[2 * k] = __uint_as_float(v[k] << 16) * up;
            z[2 * k + 1] = __uint_as_float(v[k] & 0xFFFF0000u) * up;
          }
          uint4 o;
          o.x = h2(__floats2half2_rn(z[0], z[4]));
          o.y = h2(__floats2half2_rn(z[1], z[5]));
          o.z = h2(__floats2half2_rn(z[2], z[6]));
          o.w = h2(__floats2half2_rn(z[3], z[7]));
          *reinterpret_cast<uint4*>(dst + chunk_at(row, (c & 3) * NG + (c >> 2))) = o;
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();  // O of the item before has been read
      mbar_arrive(&q_full[x]);

      float m = -FLT_MAX, l = 0.f;
      uint32_t v_exp = 0;
      for (int j = begin; j < end; ++j, ++n) {
        ok = __all_sync(0xFFFFFFFFu, wait(&s_bar[x * 2 + (n & 1)], (n >> 1) & 1));
        if (!ok) break;
        tc_fence_after();
        const Info& in = info[n & 3];
        // A zero row's f and a tile of zero keys make a c below fp32's least value, and -inf * 0, a masked
        // score's, would be NaN: c stays positive (S' is 0 there or the logit next to it) and finite.
        const float c = fminf(fmaxf(f * in.k_unit[0] * in.k_unit[1], kLeastFactor), kMostFactor);
        const uint32_t ve = in.v_exp;
        const uint32_t on = in.on[0] & in.on[1] & in.on[2] & in.on[3];
        const bool mask = __any_sync(0xFFFFFFFFu, j * 128 + 128 > lim) || on != 0xFFFFFFFFu;
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        // the maximum (a masked S goes back into TMEM)
#pragma unroll 1
        for (int k = 0; k < 128; k += 64) {
          float s[64];
#pragma unroll
          for (int y = 0; y < 64; y += 32)
            tmem_ld32(s_col + k + y, *reinterpret_cast<float(*)[32]>(s + y));
          tmem_wait_ld();
          if (mask) {
#pragma unroll
            for (int z = 0; z < 64; z += 32) {
              const int left = lim - j * 128 - k - z;  // of these 32 tokens the row sees so many
              uint32_t bits = left >= 32 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << left) - 1u;
              bits &= in.on[(k + z) >> 5];
#pragma unroll
              for (int y = 0; y < 32; ++y)
                if (!((bits >> y) & 1u)) s[z + y] = -INFINITY;
            }
#pragma unroll
            for (int y = 0; y < 64; y += 16)
              tmem_st16(s_col + k + y, *reinterpret_cast<float(*)[16]>(s + y));
            tmem_wait_st();
          }
#pragma unroll
          for (int y = 0; y < 64; y += 4) {
            mx[0] = fmaxf(mx[0], s[y]);
            mx[1] = fmaxf(mx[1], s[y + 1]);
            mx[2] = fmaxf(mx[2], s[y + 2]);
            mx[3] = fmaxf(mx[3], s[y + 3]);
          }
        }
        const float mn = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c);
        if (j == begin) {
          m = mn;
          v_exp = ve;
        } else if (__any_sync(0xFFFFFFFFu, mn > m + kRescaleLog2) || ve != v_exp) {
          // (S(j)'s commit says that O holds PV(j - 1))
          const float alpha = exp2f(m - mn);
          l *= alpha;
          m = mn;
          float ao[NG];
#pragma unroll
          for (int g = 0; g < NG; ++g) ao[g] = alpha * exp2f((float)(unit_exp(v_exp, g) - unit_exp(ve, g)));
          v_exp = ve;
#pragma unroll 1
          for (int k = 0; k < D; k += 16) {
            float o[16];
            tmem_ld16(o_col + k, o);
            tmem_wait_ld();
#pragma unroll
            for (int y = 0; y < 16; ++y) o[y] *= ao[group_of<NG>(y)];
            tmem_st16(o_col + k, o);
          }
        }
        // (two at a time: packed fp32 operations halve what is issued for all but the exponentials)
        const uint64_t c2 = pack2(c, c), m2 = pack2(kHeadLog2 - m, kHeadLog2 - m);
        uint64_t sum = pack2(0.f, 0.f);
        // the weights; PV of the first 64 tokens may begin while the others are at work
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          float s[64];
          tmem_ld32(s_col + half * 64, *reinterpret_cast<float(*)[32]>(s));
          tmem_ld32(s_col + half * 64 + 32, *reinterpret_cast<float(*)[32]>(s + 32));
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t pk[16];
#pragma unroll
            for (int y = 0; y < 32; y += 2) {
              float p0, p1;
              unpack2(fma2(pack2(s[k * 32 + y], s[k * 32 + y + 1]), c2, m2), p0, p1);
              p0 = ex2_approx(p0);
              p1 = ex2_approx(p1);
              sum = add2(sum, pack2(p0, p1));
              pk[y >> 1] = h2(__floats2half2_rn(p0, p1));
            }
            tmem_st16u(s_col + half * 32 + k * 16, pk);
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(half ? &p_full[x] : &p_half[x]);
        }
        float sum0, sum1;
        unpack2(sum, sum0, sum1);
        l += sum0 + sum1;
      }
      if (!ok) break;
      // ---- O
      ok = __all_sync(0xFFFFFFFFu, wait(&o_bar[x * 2 + (item & 1)], (item >> 1) & 1));
      if (!ok) break;
      tc_fence_after();
      const bool whole = w.whole();
      const int* np = nan_pos + (item & 3) * 4;
      float* slot = p.slots + (size_t)(2 * cta + (begin == 0 ? 1 : 0)) * slot_floats(kRows, D);
      const int sr = x * 128 + row;
      // 1 / l and the powers of two of the values' units, these in two steps (each within fp32's range)
      float u0[NG], u1[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int e = unit_exp(v_exp, g);
        u0[g] = pow2(e >> 1) * (whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f);
        u1[g] = pow2(e - (e >> 1));
      }
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.a.o) + t * p.a.o_token + h * p.a.o_head;
#pragma unroll 1
      for (int k = 0; k < D; k += 32) {
        float o[32];
        tmem_ld32(o_col + k, o);
        tmem_wait_ld();
#pragma unroll
        for (int y = 0; y < 32; ++y) {
          const int g = group_of<NG>(y);
          o[y] = lim > np[g] ? NAN : o[y] * u0[g] * u1[g];
        }
        if (!whole) {
#pragma unroll
          for (int y = 0; y < 32; y += 4)
            *reinterpret_cast<float4*>(slot + (size_t)sr * D + k + y) =
                make_float4(o[y], o[y + 1], o[y + 2], o[y + 3]);
        } else if (have) {
          // 32 places are 32 / NG channels of each group, beginning at 4 r of the first chunk
          constexpr int kPer = 32 / NG;
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int y = 0; y < kPer; y += 8) {
              uint32_t b[4];
#pragma unroll
              for (int z = 0; z < 8; z += 2) {
                // channel y + z of these: chunk of r = (y + z) / 4, place 2 (channel % 4) + (g & 1)
                const int c0 = y + z;
                const int at = NG == 4 ? (c0 >> 2) * 16 + (g >> 1) * 8 + 2 * (c0 & 3) + (g & 1)
                                       : (c0 >> 2) * 8 + 2 * (c0 & 3) + g;
                const __nv_bfloat162 v = __floats2bfloat162_rn(o[at], o[at + 2]);
                b[z >> 1] = *reinterpret_cast<const uint32_t*>(&v);
              }
              *reinterpret_cast<uint4*>(dst + 32 * g + k / NG + y) = make_uint4(b[0], b[1], b[2], b[3]);
            }
        }
      }
      if (!whole) {
        slot[(size_t)kRows * D + sr] = m;
        slot[(size_t)kRows * (D + 1) + sr] = l;
        if (begin == 0 && threadIdx.x == 0) p.parts[cta] = w.part(run, cta);
      }
      tc_fence_before();
    }
    if (!ok && lane == 0 && !*abort_flag) fail();
  } else if (warp < 12) {
    // ================================================================ tokens
    regs_lower<kRegsUnpack>();
    const int tok = threadIdx.x - 256;
    const int page = p.a.b.page, page_log = __ffs(page) - 1, rec = kv4_rec_bytes(page, D);
    constexpr int kWords = D / 32;  // 16-byte pieces of a row of levels
    const int off = tok & (page - 1);
    const int turn = NG == 4 ? ((off >> 1) & 1) * 2 : 0;  // pieces of a value's row change places
    // With 4 pieces neighbouring pairs of tokens begin at different ones, so that no bank is met
    // twice.  A piece's words are chunks 4 piece to 4 piece + 3 of the token's row, at
    // place(piece) + word[k] (chunk_at).
    const int first = NG == 4 ? (tok >> 1) & 3 : 0;
    auto place = [&](int piece) {
      return (piece >> 1) * (128 * 128) + ((((piece & 1) << 2) ^ (tok & 4)) << 4);
    };
    int word[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) word[k] = tok * 128 + ((k ^ (tok & 3)) << 4);
    const unsigned char* ring = smem + C::kOffRing + (tok >> page_log) * rec;
    int n = 0, item = 0;
    int ended[2] = {0, 0};  // by buffer: 1 + the item that ended with its last token tile, else 0
    int kh = 0, kph = 0;    // ring place and phase of the keys of tile n; the values' follow them
    // out: all 128 threads know of a failure, and leave together (none may be missing at a barrier)
    bool ok = true, out = false;
    for (; w.more() && !out; w.next(p), ++item) {
      const int begin = w.begin(), end = w.end();
      uint32_t ve = 0x2F2F2F2Fu;  // the values' units so far, a byte a group (at least 2^-80)
      if (tok < 4) nan_pos[(item & 3) * 4 + tok] = INT_MAX;
      for (int j = begin; j < end; ++j, ++n) {
        const int vh = kh + 1 == kHalves ? 0 : kh + 1, vph = kh + 1 == kHalves ? kph ^ 1 : kph;
        if (ok) ok = wait(&c_full[kh], kph);
        if (ok) ok = wait(&c_full[vh], vph);
        const unsigned char* kc = ring + kh * C::kHalfBytes;
        const unsigned char* vc = ring + vh * C::kHalfBytes;
        // the page's number: -1 behind the last token, -2 where it is not in the cache
        const int pg = ok ? s_pages[kh * 8 + (tok >> page_log)] : -1;
        uint4 kp = make_uint4(0, 0, 0, 0), vp = kp;
        if (pg >= 0 && j * 128 + tok < w.limit()) {
          const unsigned char* a = kc + page * (D / 2) + off * (D / 8);
          const unsigned char* b = vc + page * (D / 2) + off * (D / 8);
          if constexpr (NG == 4) {
            kp = *reinterpret_cast<const uint4*>(a);
            vp = *reinterpret_cast<const uint4*>(b);
          } else {
            const uint2 a2 = *reinterpret_cast<const uint2*>(a), b2 = *reinterpret_cast<const uint2*>(b);
            kp.x = a2.x, kp.y = a2.y, vp.x = b2.x, vp.y = b2.y;
          }
        }
        // ---- the tile's units: one for its keys, one for the values of each group
        uint32_t ka = 0, va = 0;
        const uint32_t pk[4] = {kp.x, kp.y, kp.z, kp.w}, pv[4] = {vp.x, vp.y, vp.z, vp.w};
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          ka = max(ka, reach(pk[g]));
          va |= __reduce_max_sync(0xFFFFFFFFu, reach(pv[g]) >> 7) << (8 * g);
        }
        ka = __reduce_max_sync(0xFFFFFFFFu, ka >> 7);
        uint32_t* mx = s_max + (n & 1) * 8;
        if (lane == 0) {
          mx[(warp - 8) * 2] = ka;
          mx[(warp - 8) * 2 + 1] = va;
        }
        out = bar_red_or(1, 128, !ok);
        if (out) break;
        const uint32_t ke = max(max(max(mx[0], mx[2]), max(mx[4], mx[6])), 47u);
        ve = __vmaxu4(ve, __vmaxu4(__vmaxu4(mx[1], mx[3]), __vmaxu4(mx[5], mx[7])));
        const int kn = (int)ke - 118;  // scales below 2^-8: times 2^-(e + 9), e = ke - 127
        const uint32_t on = __ballot_sync(0xFFFFFFFFu, pg != -2);
        if (pg == -2) kv4_record(p.a.b.status);
        // ---- K(n), once S(n - 2) has been taken of its buffer
        if (ok && n >= 2) ok = wait(&s_bar[2 + (n & 1)], ((n - 2) >> 1) & 1);
        if (ok) {
          Info& in = info[n & 3];
          if (tok == 0) {
            // in two factors: 2^kn alone, or with a small f, may leave fp32's range
            in.k_unit[0] = pow2(kn >> 1);
            in.k_unit[1] = pow2(kn - (kn >> 1));
            in.v_exp = ve;
          }
          if (lane == 0) in.on[warp - 8] = on;
          unsigned char* dst = smem + C::kOffK + (n & 1) * C::kTileBytes;
          // 2^(24 - kn), in two factors (either may leave fp32's range alone)
          const float a0 = pow2((24 - kn) >> 1), a1 = pow2(24 - kn - ((24 - kn) >> 1));
          __half2 se[NG], so[NG], lo[NG];
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const float sc = __uint_as_float(pk[g] << 16) * a0 * a1;
            const float lw = __uint_as_float(pk[g] & 0xFFFF0000u) * a0 * a1 * 0x1p-24f;
            se[g] = __float2half2_rn(sc);
            so[g] = __float2half2_rn(sc * 0.0625f);
            lo[g] = __float2half2_rn(lw);
          }
#pragma unroll 1
          for (int i = 0; i < kWords; ++i) {  // d = 128: piece q, words g; d = 64: two pieces of two
            const int piece = (i + first) & (kWords - 1);
            const uint4 u = reinterpret_cast<const uint4*>(kc + off * (D / 2))[piece];
            const uint32_t wd[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              *reinterpret_cast<uint4*>(dst + place(piece) + word[k]) =
                  unpack8(wd[k], se[k % NG], so[k % NG], lo[k % NG]);
          }
          mbar_arrive(&c_free[kh]);
          fence_proxy_async_smem();
          mbar_arrive(&k_full[n & 1]);
        }
        // ---- V(n), once PV(n - 2) has: with S(n - 1) in the same item, or the item's last PV
        if (ok && n >= 2) {
          const int it = ended[n & 1];
          ok = it ? wait(&o_bar[2 + ((it - 1) & 1)], ((it - 1) >> 1) & 1)
                  : wait(&s_bar[2 + ((n - 1) & 1)], ((n - 1) >> 1) & 1);
        }
        if (ok) {
          unsigned char* dst = smem + C::kOffV + (n & 1) * C::kTileBytes;
          float sc[NG], lw[NG];
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const int e = 24 - unit_exp(ve, g);
            const float a0 = pow2(e >> 1), a1 = pow2(e - (e >> 1));
            sc[g] = __uint_as_float(pv[g] << 16) * a0 * a1;
            lw[g] = __uint_as_float(pv[g] & 0xFFFF0000u) * a0 * a1 * 0x1p-24f;
            // a NaN group stands as 0 in the products (rows that do not see the token must not
            // meet it); the rows that do get their NaN at the end
            if ((pv[g] & 0x7F80u) == 0x7F80u || (pv[g] & 0x7F800000u) == 0x7F800000u) {
              sc[g] = lw[g] = 0.f;
              atomicMin(&nan_pos[(item & 3) * 4 + g], j * 128 + tok);
            }
          }
          __half2 se[NG / 2], so[NG / 2], lo[NG / 2];
#pragma unroll
          for (int g = 0; g < NG / 2; ++g) {
            se[g] = __floats2half2_rn(sc[2 * g], sc[2 * g + 1]);
            so[g] = __floats2half2_rn(sc[2 * g] * 0.0625f, sc[2 * g + 1] * 0.0625f);
            lo[g] = __floats2half2_rn(lw[2 * g], lw[2 * g + 1]);
          }
#pragma unroll 1
          for (int i = 0; i < kWords; ++i) {
            const int piece = (i + first) & (kWords - 1);
            const uint4 u = reinterpret_cast<const uint4*>(vc + off * (D / 2))[piece ^ turn];
            const uint32_t wd[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              *reinterpret_cast<uint4*>(dst + place(piece) + word[k]) =
                  unpack8(wd[k], se[k % (NG / 2)], so[k % (NG / 2)], lo[k % (NG / 2)]);
          }
          mbar_arrive(&c_free[vh]);
          fence_proxy_async_smem();
          mbar_arrive(&v_full[n & 1]);
        }
        ended[n & 1] = j == end - 1 ? item + 1 : 0;
        kh = vh + 1 == kHalves ? 0 : vh + 1;
        kph = vh + 1 == kHalves ? vph ^ 1 : vph;
      }
    }
    if ((!ok || out) && lane == 0 && !*abort_flag) fail();
  } else {
    regs_lower<kRegsIssue>();
    if (warp == 12 && lane == 0) {
      // ================================================================ products
      const uint64_t q0 = smem_desc(smem_u32(smem + C::kOffQ), 16, 1024);
      const uint64_t k0 = smem_desc(smem_u32(smem + C::kOffK), 16, 1024);
      const uint64_t v0 = smem_desc(smem_u32(smem + C::kOffV), 128 * 128, 1024);
      int n = 0, item = 0;
      int pc[2] = {0, 0}, hc[2] = {0, 0}, qc[2] = {0, 0};  // phases of p_full, p_half, q_full
      bool ok = true;
      // S of query tile x and token tile t
      auto issue_s = [&](int x, int t) {
        const uint64_t a = q0 + (uint64_t)(x * (C::kTileBytes >> 4));
        const uint64_t b = k0 + (uint64_t)((t & 1) * (C::kTileBytes >> 4));
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t at = (uint64_t)(((k / 4) * (128 * 128) + (k % 4) * 32) >> 4);
          umma_f16_ss(tmem + x * 128, a + at, b + at, C::kDescS, k > 0 ? 1u : 0u);
        }
      };
      // O += P V, the first or the second 64 tokens
      auto issue_pv = [&](int x, int t, bool first, int half) {
        const uint64_t b = v0 + (uint64_t)((t & 1) * (C::kTileBytes >> 4));
#pragma unroll
        for (int k = half * 4; k < half * 4 + 4; ++k)
          umma_f16_ts(tmem + C::kTmO + x * D, tmem + x * 128 + k * 8, b + (uint64_t)(k * 128), C::kDescO,
                      k > 0 || !first ? 1u : 0u);
      };
      for (; w.more() && ok; w.next(p), ++item) {
        const int begin = w.begin(), end = w.end();
        const int tiles = item_rows() > 128 ? 2 : 1;
        for (int j = begin; ok && j <= end; ++j) {
          // for each query tile: PV(j - 1), then S(j); token tile j is number n
          for (int x = 0; ok && x < 2; ++x) {
            if (j > begin) {
              if (x == 0) ok = wait(&v_full[(n - 1) & 1], ((n - 1) >> 1) & 1);
              if (ok && x < tiles) {
                ok = wait(&p_half[x], hc[x] & 1);
                ++hc[x];
                if (!ok) break;
                tc_fence_after();
                issue_pv(x, n - 1, j - 1 == begin, 0);
              }
              if (ok) ok = wait(&p_full[x], pc[x] & 1);
              ++pc[x];
              if (!ok) break;
            }
            if (x < tiles) {
              tc_fence_after();
              if (j > begin) issue_pv(x, n - 1, j - 1 == begin, 1);
              if (j < end) {
                if (j == begin) {
                  ok = wait(&q_full[x], qc[x] & 1);
                  ++qc[x];
                }
                if (ok && x == 0) ok = wait(&k_full[n & 1], (n >> 1) & 1);
                if (!ok) break;
                tc_fence_after();
                issue_s(x, n);
              }
            }
            // tile B's barriers tell when buffers are free, with or without a tile B
            umma_commit(j < end ? &s_bar[x * 2 + (n & 1)] : &o_bar[x * 2 + (item & 1)]);
          }
          if (j < end) ++n;
        }
      }
      if (!ok) {
        if (!*abort_flag) fail();
      }
      // nothing in flight when TMEM goes
      umma_commit(drain);
      volatile int never = 0;
      mbar_wait_bounded(drain, 0, &never, kTimeoutNs);
    }
    if (warp == 13) {
      // ================================================================ copies
      const int page = p.a.b.page, page_log = __ffs(page) - 1, rec = kv4_rec_bytes(page, D);
      const int pages = 128 >> page_log;
      int c = 0;  // halves so far
      bool ok = true;
      for (; w.more() && ok; w.next(p)) {
        const int begin = w.begin(), end = w.end(), limit = w.limit();
        const int32_t* table = p.a.b.table + (long long)w.b * p.a.b.max_pages;
        const uint8_t* heads = p.a.cache + (long long)w.head * 2 * rec;
        // 32 pages looked up at a time, one a lane
        auto look = [&](int first) {
          const long long pos = (long long)(first + lane) << page_log;
          if (pos >= limit) return -1;
          const int pg = table[pos >> page_log];
          return pg < 0 || pg >= p.a.b.n_pages ? -2 : pg;
        };
        int chunk = begin * pages, pg = look(chunk);
        for (int j = begin; ok && j < end; ++j) {
          if (j * pages - chunk + pages > 32) {
            chunk = j * pages;
            pg = look(chunk);
          }
          const int x = lane - (j * pages - chunk);  // this lane's page within the tile
          const bool in = x >= 0 && x < pages, on = in && pg >= 0;
          const int bytes = rec * __popc(__ballot_sync(0xFFFFFFFFu, on));
          for (int side = 0; side < 2; ++side, ++c) {
            const int st = c % kHalves;
            bool good = true;
            if (lane == 0 && c >= kHalves) good = wait(&c_free[st], (c / kHalves - 1) & 1);
            ok = __shfl_sync(0xFFFFFFFFu, good, 0);
            if (!ok) break;
            if (in) s_pages[st * 8 + x] = pg;
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(&c_full[st], bytes);
            __syncwarp();
            if (on)
              bulk_load(smem + C::kOffRing + st * C::kHalfBytes + x * rec,
                        heads + (long long)pg * p.a.b.hkv * 2 * rec + side * rec, rec, &c_full[st]);
          }
        }
      }
      if (!ok && lane == 0) {
        if (!*abort_flag) fail();
        volatile int never = 0;  // copies still on their way into shared memory
        for (int i = max(0, c - kHalves); i < c; ++i)
          mbar_wait_bounded(&c_full[i % kHalves], (i / kHalves) & 1, &never, kTimeoutNs);
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
int launch(const SplitParams& p, cudaStream_t stream) {
  using C = MC<D>;
  auto kern = kv4_many_kernel<D>;
  static SplitGrid ctas;
  const int grid = ctas.get(reinterpret_cast<const void*>(kern), C::kSmem);
  if (grid <= 0) return SBSA_ERR_CUDA;
  kern<<<grid, kThreads, C::kSmem, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return SBSA_ERR_CUDA;
  return launch_join<D, kRows>(p, grid, stream);
}

}  // namespace

size_t kv4_many_workspace(const Kv4AttendArgs& a) { return split_workspace(kRows, a.d); }

int launch_kv4_many(const Kv4AttendArgs& a, cudaStream_t stream) {
  const SplitParams p = split_params(a, kRows);
  return a.d == 64 ? launch<64>(p, stream) : launch<128>(p, stream);
}

}  // namespace sbsa
