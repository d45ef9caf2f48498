// How attention over the 4-bit cache is shared out over the CTAs, and how the
// parts of what several CTAs share are joined.
//
// The rows of one kv head (or listed query head) of a sequence, in tiles of
// ROWS, are items; an item's tokens fall into units of 128.  Item after item,
// each costs COST (rows, joining, output) and then one for each unit; the whole is
// cut into equal runs, one for each CTA, so that ragged batches and single long
// contexts both fill the GPU.  Each CTA finds its run by a scan over the items'
// sizes: nothing is read by the host, and the cuts depend on the sizes alone.
#pragma once
#include <atomic>
#include <cfloat>
#include <chrono>

#include "kv4.cuh"
#include "tma_map.h"

namespace sbsa {
namespace {

constexpr int kSplitUnit = 128;
constexpr int kMaxCtas = 160;

__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                            *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }

struct Part {  // the item whose first part a CTA holds, and its number of parts (0: none)
  int parts, seq, head, tile;
};

// A slot holds the partial rows of one item: [rows][d] outputs, their references
// and their weights' sums.
constexpr size_t slot_floats(int rows, int d) { return (size_t)rows * (d + 2); }

inline size_t split_workspace(int rows, int d) {
  return kMaxCtas * (2 * (slot_floats(rows, d) * sizeof(float) + sizeof(uint64_t)) + sizeof(Part));
}

struct SplitParams {
  Kv4AttendArgs a;
  int heads;         // items per sequence and row tile: kv heads, or listed query heads
  int group;         // query heads of an item
  int kv_div;        // item head / kv_div = kv head
  int capacity;      // tokens that a row of the page table can name
  float scale_log2;  // sm_scale * log2(e)
  float* slots;      // two a CTA: of the item that begins before its run, and of the one that
                     // goes on behind it
  Part* parts;       // one a CTA
  uint64_t* ready;   // one a slot (kv4_ready.h)
  uint64_t call;
};

// A number that no other call has (and that memory which no call has written does not hold by
// chance); it ends in binary 01.
inline uint64_t call_number() {
  static std::atomic<uint64_t> next{
      (uint64_t)std::chrono::steady_clock::now().time_since_epoch().count()};
  uint64_t z = (next.fetch_add(1) + 1) * 0x9E3779B97F4A7C15ull;  // splitmix64 (Steele, Lea, Flood)
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return ((z ^ (z >> 31)) & ~3ull) | 1;
}

inline SplitParams split_params(const Kv4AttendArgs& a, int slot_rows) {
  SplitParams p{};
  p.a = a;
  p.heads = a.list_heads ? a.list_heads : a.b.hkv;
  p.group = a.hq / p.heads;
  p.kv_div = p.heads / a.b.hkv;
  p.capacity = a.b.max_pages * a.b.page;  // below 2^31 - 2^16: checked with the parameters
  p.scale_log2 = a.sm_scale * 1.4426950408889634f;
  p.slots = static_cast<float*>(a.workspace);
  p.parts = reinterpret_cast<Part*>(p.slots + kMaxCtas * 2 * slot_floats(slot_rows, a.d));
  p.ready = reinterpret_cast<uint64_t*>(p.parts + kMaxCtas);
  return p;
}

// What a launch has to know of the current device, asked once a device and kernel (the
// questions cost as much as a launch): the CTAs of the grid, 0 on an error.
struct SplitGrid {
  std::atomic<int> ctas[64] = {};
  int get(const void* kernel, int smem_bytes) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = ctas[dev].load(std::memory_order_relaxed);
    if (n) return n;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes) !=
        cudaSuccess)
      return 0;
    n = sm_count();
    n = n < kMaxCtas ? n : kMaxCtas;
    ctas[dev].store(n, std::memory_order_relaxed);
    return n;
  }
};

// Whether an item can have more than one unit, and so more than one CTA: else there
// is nothing to join, and no workspace.
inline bool split_possible(const Kv4AttendArgs& a) {
  if (a.list_heads) return (long long)a.max_blocks * a.block > kSplitUnit;
  return (long long)a.b.max_pages * a.b.page > kSplitUnit;
}

// A sequence as an item sees it: its first row and number of rows, and the first row's position.
// (The position of a row fits 31 bits; 1 more than it are the tokens that the row sees.)
struct Seq {
  int first, rows, ahead;

  // Tokens that row i sees: 0 before the sequence's first token and behind the last one that the
  // table can name.
  __device__ int visible(const SplitParams& p, int i) const {
    const int n = ahead + i + 1;
    return n < 1 || n > p.capacity ? 0 : n;
  }
  // Tokens of the sequence, as far as the table can name them.
  __device__ int len(const SplitParams& p) const { return clamp_int(ahead + rows, 0, p.capacity); }
};

__device__ __forceinline__ Seq seq_of(const SplitParams& p, int b) {
  // the rows that the tensors have; positions go by cu and the length as they are given
  const int to = p.a.b.cu[b + 1];
  Seq s;
  s.first = clamp_int(p.a.b.cu[b], 0, p.a.b.n_tokens);
  s.rows = clamp_int(to, s.first, p.a.b.n_tokens) - s.first;
  // (31 bits hold it for a sequence with rows: to > first >= 0; a negative length is as good as none)
  s.ahead = (int)((uint32_t)max(p.a.b.lens[b], 0) - (uint32_t)to + (uint32_t)s.first);
  return s;
}

// Reports a sequence that is longer than the table, or whose rows the tensors do not have.
__device__ __forceinline__ void check_seq(const SplitParams& p, int b) {
  const int from = p.a.b.cu[b], to = p.a.b.cu[b + 1];
  kv4_named(p.a.b, p.a.b.lens[b]);
  if (from < 0 || to < from || to > p.a.b.n_tokens) kv4_record(p.a.b.status);
}

// Row `row` of the item head: the token row, its number in the sequence and the
// query head; false past the last.
__device__ __forceinline__ bool row_of(const SplitParams& p, const Seq& s, int head, uint32_t row,
                                       long long* t, int* h, int* i) {
  const uint32_t group = p.group, n = row / group;
  *i = (int)n;
  if (n >= (uint32_t)s.rows) return false;
  *t = s.first + (int)n;
  *h = head * p.group + (int)(row - n * group);
  return true;
}

// The kernel for many rows is not called with lists.
template <int ROWS>
constexpr bool kTakesLists = ROWS <= 16;

// The items of one (sequence, head).  (Rows times heads fit 31 bits: checked on the host.)
template <int ROWS>
struct Items {
  Seq seq;
  int tiles;
  int listed;  // units of the listed blocks, -1 without lists

  __device__ Items() {}
  __device__ Items(const SplitParams& p, int b, int head) {
    seq = seq_of(p, b);
    tiles = (int)(((uint32_t)seq.rows * (uint32_t)p.group + ROWS - 1) / ROWS);
    listed = -1;
    if (kTakesLists<ROWS> && p.a.list_heads) {
      const int n = clamp_int(p.a.cnt[(long long)b * p.heads + head], 0, p.a.max_blocks);
      listed = (n * p.a.block + kSplitUnit - 1) / kSplitUnit;
    }
  }
  // Tokens that no row of the tile sees more of: those of its last row, as far as there are any.
  __device__ int limit(const SplitParams& p, int tile) const {
    const uint32_t rows = min((uint32_t)(tile + 1) * ROWS, (uint32_t)seq.rows * (uint32_t)p.group);
    return clamp_int(seq.ahead + (int)((rows - 1) / (uint32_t)p.group) + 1, 0, p.capacity);
  }
  // Units of a tile; one that sees nothing still takes one (it writes zeros).
  __device__ int units(const SplitParams& p, int tile) const {
    const int n = kTakesLists<ROWS> && listed >= 0 ? listed : (limit(p, tile) + kSplitUnit - 1) / kSplitUnit;
    return n < 1 ? 1 : n;
  }
  template <int COST>
  __device__ long long cost(const SplitParams& p) const {
    long long c = (long long)tiles * COST;
    for (int i = 0; i < tiles; ++i) c += units(p, i);
    return c;
  }
};

// A CTA's run: where it begins, and the cut of the whole.
struct Run {
  int b, head, tile, cost;  // first item, and how much of its cost lies before the run
  int ctas;
  long long total, begin, end;
};

template <int THREADS>
constexpr int kScanBytes = (THREADS / 32 + 2) * 8 + 16;

// All threads of the CTA together, with kScanBytes of shared memory; false when
// the CTA has no run.  Ends with the CTA in step (earlier writes to shared memory are
// visible).
template <int ROWS, int COST, int THREADS>
__device__ __forceinline__ bool split_run(const SplitParams& p, long long* s_scan, Run* run) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* s_start = reinterpret_cast<int*>(s_scan + THREADS / 32);
  const int items = p.a.b.n_seqs * p.heads;
  const int per = (items + THREADS - 1) / THREADS;
  const int i0 = min(items, (int)threadIdx.x * per), i1 = min(items, i0 + per);
  long long mine = 0;
  for (int i = i0; i < i1; ++i) {
    mine += Items<ROWS>(p, i / p.heads, i % p.heads).template cost<COST>(p);
    if (blockIdx.x == 0 && i % p.heads == 0) check_seq(p, i / p.heads);
  }
  long long incl = mine;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long x = __shfl_up_sync(0xFFFFFFFFu, incl, m);
    if (lane >= m) incl += x;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  long long before = incl - mine, total = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  const int ctas = (int)(total < (long long)gridDim.x ? total : (long long)gridDim.x);
  const int cta = blockIdx.x;
  if (cta >= ctas) return false;
  run->ctas = ctas;
  run->total = total;
  run->begin = total * cta / ctas;
  run->end = total * (cta + 1) / ctas;
  if (run->begin >= before && run->begin < before + mine) {
    long long x = run->begin - before;
    for (int i = i0; i < i1; ++i) {
      const Items<ROWS> it(p, i / p.heads, i % p.heads);
      int t = 0;
      for (; t < it.tiles; ++t) {
        const long long c = COST + it.units(p, t);
        if (x < c) break;
        x -= c;
      }
      if (t < it.tiles) {
        s_start[0] = i / p.heads;
        s_start[1] = i % p.heads;
        s_start[2] = t;
        s_start[3] = (int)x;
        break;
      }
    }
  }
  __syncthreads();
  run->b = s_start[0], run->head = s_start[1], run->tile = s_start[2], run->cost = s_start[3];
  return true;
}

// Walks the items of a run.  Units [begin, end) of the current item are the
// CTA's; a run that ends within an item's COST leaves it to the next CTA.
template <int ROWS, int COST>
struct SplitWalk : Items<ROWS> {
  int b, head, tile, unit_count;
  int item_limit;
  long long before, left;  // cost from the item's start to the run's begin and end

  __device__ SplitWalk(const SplitParams& p, const Run& r) : Items<ROWS>(p, r.b, r.head) {
    b = r.b, head = r.head, tile = r.tile;
    before = r.cost;
    left = r.cost + r.end - r.begin;
    set(p);
  }
  __device__ void set(const SplitParams& p) {
    unit_count = this->units(p, tile);
    item_limit = Items<ROWS>::limit(p, tile);
  }
  __device__ int limit() const { return item_limit; }
  __device__ int begin() const { return before > COST ? (int)before - COST : 0; }
  __device__ int end() const {
    const long long e = left - COST;
    return e < 0 ? 0 : e < unit_count ? (int)e : unit_count;
  }
  __device__ bool whole() const { return begin() == 0 && end() == unit_count; }
  __device__ bool more() const { return left > COST; }
  __device__ void next(const SplitParams& p) {
    left -= COST + unit_count;
    before = 0;
    if (left <= COST) return;
    if (++tile == this->tiles) {
      tile = 0;
      do {
        if (++head == p.heads) {
          head = 0;
          if (++b == p.a.b.n_seqs) {
            left = 0;
            return;
          }
        }
        static_cast<Items<ROWS>&>(*this) = Items<ROWS>(p, b, head);
      } while (this->tiles == 0);
    }
    set(p);
  }
  // The CTA that owns the item's first unit.
  __device__ int first_cta(const Run& r) const {
    const long long first = r.end - left + COST;
    return (int)(((first + 1) * r.ctas + r.total - 1) / r.total) - 1;
  }
  // The CTA's entry of p.parts for an item that begins here and goes on in the next
  // CTAs, up to the one that owns its last unit.
  __device__ Part part(const Run& r, int cta) const {
    const long long last = r.end - left + COST + unit_count - 1;
    const int owner = (int)(((last + 1) * r.ctas + r.total - 1) / r.total) - 1;
    return Part{owner - cta + 1, b, head, tile};
  }
};

// Joins the parts of the item that begins in CTA blockIdx.x and goes on in the next
// ones (kv4_many.cu).  A thread takes 4 places of a slot's row.
constexpr int kJoinThreads = 256;

template <int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) kv4_join_kernel(const __grid_constant__ SplitParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Part part = p.parts[blockIdx.x];
  if (part.parts < 2) return;
  const int x = blockIdx.y * kJoinThreads + threadIdx.x;
  const int c = x % (D / 4) * 4, row = x / (D / 4);
  if (row >= ROWS) return;
  const Seq s = seq_of(p, part.seq);
  long long t;
  int h, i;
  if (!row_of(p, s, part.head, (uint32_t)part.tile * ROWS + row, &t, &h, &i)) return;
  auto slot = [&](int k) {
    return p.slots + (size_t)(k == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + k)) *
                         slot_floats(ROWS, D);
  };
  float top = -FLT_MAX;
#pragma unroll 4
  for (int k = 0; k < part.parts; ++k) top = fmaxf(top, slot(k)[ROWS * D + row]);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
#pragma unroll 4
  for (int k = 0; k < part.parts; ++k) {
    const float* y = slot(k);
    const float4 v = *reinterpret_cast<const float4*>(y + row * D + c);
    const float fac = exp2f(y[ROWS * D + row] - top);
    sum = fmaf(fac, y[ROWS * (D + 1) + row], sum);
    acc.x = fmaf(fac, v.x, acc.x);
    acc.y = fmaf(fac, v.y, acc.y);
    acc.z = fmaf(fac, v.z, acc.z);
    acc.w = fmaf(fac, v.w, acc.w);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.a.o) + t * p.a.o_token + h * p.a.o_head;
  // places c to c + 3: channels u and u + 1 of two neighbouring groups
  const int u = D == 128 ? 64 * ((c >> 3) & 1) + 4 * (c >> 4) + ((c & 7) >> 1)
                         : 4 * (c >> 3) + ((c & 7) >> 1);
  *reinterpret_cast<__nv_bfloat162*>(dst + u) = __floats2bfloat162_rn(acc.x, acc.z);
  *reinterpret_cast<__nv_bfloat162*>(dst + u + 32) = __floats2bfloat162_rn(acc.y, acc.w);
}

// Behind the attending kernel, which lets it start up early.
template <int D, int ROWS>
int launch_join(const SplitParams& p, int grid, cudaStream_t stream) {
  if (!split_possible(p.a)) return SBSA_OK;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid, (ROWS * (D / 4) + kJoinThreads - 1) / kJoinThreads);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, ROWS>, p) == cudaSuccess
             ? SBSA_OK
             : SBSA_ERR_CUDA;
}

}  // namespace
}  // namespace sbsa
