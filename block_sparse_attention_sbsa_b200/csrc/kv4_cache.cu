// The 4-bit key-value cache: quantising new tokens into their pages, and
// reading tokens back.  Format and layout: include/sbsa.h.
//
// Both kernels move bytes: append reads 2 d (bf16) or 4 d (fp32) bytes and
// writes 5/8 d for each token, kv head and side (key or value), read the
// reverse; HBM bounds them, with the arithmetic close behind (a 128k prompt of 8
// heads is 268 M elements: at 10 instructions each 60 us of issue against 107 us of
// traffic).  So what is done per group is done once: in append a thread has a whole
// group of 32 channels (extremes without shuffles, in packed bf16 with NaN passing
// through), rounds to levels by adding 1.5 * 2^23 and gathers 8 levels by
// multiply-adds on the sums' bits; in read a level is taken to fp32 by OR into the
// mantissa of 2^23, the place in the word going into the scale.  A CTA takes a tile of
// tokens of one kv head and side.  append collects the tile's rows in shared memory and
// writes them to the pages 16 bytes a thread, token after token, whatever the order of the
// inputs.  Measured among other calls for a second: the 128k prompt 136 us (5.2 TB/s, 0.79 of a
// copy), a 32k context read in 32.8 us (5.4 TB/s, 0.82); in bursts of 12 ms, before the power limit
// lowers the clocks, 120 us (256 with a thread for 8 channels) and 31 (49 with 4 bytes a thread).
#include <cuda_runtime.h>

#include "kv4.cuh"

namespace sbsa {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float nan_max(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float nan_min(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The 32 channels of a group, as they lie in memory.
template <typename T>
struct Group;

template <>
struct Group<float> {
  float4 v[8];
  __device__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = reinterpret_cast<const float4*>(p)[i];
  }
  __device__ float2 pair(int i) const {  // channels 2 i, 2 i + 1
    return i & 1 ? make_float2(v[i >> 1].z, v[i >> 1].w) : make_float2(v[i >> 1].x, v[i >> 1].y);
  }
  __device__ void extremes(float* mn, float* mx) const {
    float a = v[0].x, b = v[0].x;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 x = pair(i);
      a = nan_min(a, nan_min(x.x, x.y));
      b = nan_max(b, nan_max(x.x, x.y));
    }
    *mn = a;
    *mx = b;
  }
};

template <>
struct Group<__nv_bfloat16> {
  uint4 v[4];
  __device__ void load(const __nv_bfloat16* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ uint32_t word(int i) const {
    const uint4& u = v[i >> 2];
    return (i & 3) == 0 ? u.x : (i & 3) == 1 ? u.y : (i & 3) == 2 ? u.z : u.w;
  }
  __device__ float2 pair(int i) const {
    const uint32_t w = word(i);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  __device__ static __nv_bfloat162 two(uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); }
  __device__ void extremes(float* mn, float* mx) const {
    __nv_bfloat162 a = two(word(0)), b = a;
#pragma unroll
    for (int i = 1; i < 16; ++i) {
      a = __hmin2_nan(a, two(word(i)));
      b = __hmax2_nan(b, two(word(i)));
    }
    *mn = nan_min(__low2float(a), __high2float(a));
    *mx = nan_max(__low2float(b), __high2float(b));
  }
};

// Levels 8 q to 8 q + 7 of a group in w[q], and its pair (scale low, low high).
struct Quantised {
  uint32_t w[4], pair;
};

template <typename T>
__device__ __forceinline__ Quantised quantise(const Group<T>& x) {
  float mn, mx;
  x.extremes(&mn, &mx);
  mn = __fadd_rn(mn, 0.f);  // -0 becomes +0
  uint32_t bits = __float_as_uint(mn);
  if (bits >> 31) bits += 0xFFFFu;
  bits &= 0xFFFF0000u;  // rounded down to bf16
  const float low = __uint_as_float(bits);
  const float span = __fsub_rn(mx, low);  // NaN or infinite with any such element
  const float step = __fmul_rn(span, 1.0f / 15.0f);
  const uint32_t up = (__float_as_uint(step) + 0xFFFFu) & 0xFFFF0000u;  // rounded up
  const float scale = span < 0x1p-100f ? 0.f : __uint_as_float(up);
  const bool finite = isfinite(span) && isfinite(__uint_as_float(up));
  const float inv = scale > 0.f ? __frcp_rn(scale) : 0.f;
  Quantised r;
  r.pair = finite ? (__float_as_uint(scale) >> 16) | bits : 0x7FC07FC0u;
  // x - low <= span <= 15.00001 scale, so the nearest level is at most 15; the sum with
  // 1.5 * 2^23 has the bits 0x4B400000 + level
  constexpr uint32_t kBias = 0x4B400000u * 0x11111111u;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t acc = 0;
#pragma unroll
    for (int i = 3; i >= 0; --i) {
      const float2 e = x.pair(4 * q + i);
      const float a = __fadd_rn(__fmul_rn(__fsub_rn(e.x, low), inv), 12582912.f);
      const float b = __fadd_rn(__fmul_rn(__fsub_rn(e.y, low), inv), 12582912.f);
      acc = acc * 16u + __float_as_uint(b);
      acc = acc * 16u + __float_as_uint(a);
    }
    r.w[q] = finite ? acc - kBias : 0u;
  }
  return r;
}

// What 8 levels of a group stand for: low + scale * level.  Scale has 8 significant
// bits and level 4, so the product is exact and there is one rounding.  A level at bit 4 i
// of a half word becomes level * 16^i in fp32; scale[i] is scale / 16^i.
struct Unpacker {
  float scale[4], low;
  __device__ explicit Unpacker(uint32_t pair) {
    scale[0] = __uint_as_float(pair << 16);
    scale[1] = scale[0] * 0x1p-4f;
    scale[2] = scale[0] * 0x1p-8f;
    scale[3] = scale[0] * 0x1p-12f;
    low = __uint_as_float(pair & 0xFFFF0000u);
  }
  __device__ float one(uint32_t w, int i) const {  // level i of 8
    const uint32_t half = i < 4 ? w : w >> 16;
    const float f = __uint_as_float((half & (15u << (4 * (i & 3)))) | 0x4B000000u) - 8388608.f;
    return fmaf(scale[i & 3], f, low);
  }
};

__device__ __forceinline__ void store8(float* p, const Unpacker& u, uint32_t w) {
  reinterpret_cast<float4*>(p)[0] = make_float4(u.one(w, 0), u.one(w, 1), u.one(w, 2), u.one(w, 3));
  reinterpret_cast<float4*>(p)[1] = make_float4(u.one(w, 4), u.one(w, 5), u.one(w, 6), u.one(w, 7));
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const Unpacker& u, uint32_t w) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(u.one(w, 2 * i), u.one(w, 2 * i + 1));
    o[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
}

// A tile's rows: page and token of the page of each, page -1 where the row
// has no place, -2 where it belongs to no sequence.
template <int TOKENS>
struct Places {
  int page[TOKENS];
  int off[TOKENS];
};

template <int TOKENS>
__device__ __forceinline__ void find_places(const Kv4Batch& b, int t0, Places<TOKENS>& pl) {
  // (a thread that looks up none)
  if (threadIdx.x == kThreads - 1 && t0 == 0 && blockIdx.y == 0) kv4_check_rows(b);
  static_assert(TOKENS < kThreads, "a thread to spare");
  for (int i = threadIdx.x; i < TOKENS; i += kThreads) {
    int page = -2, off = 0;
    if (t0 + i < b.n_tokens) {
      bool in_seq;
      if (!kv4_place(b, t0 + i, &in_seq, &page, &off)) page = in_seq ? -1 : -2;
    }
    pl.page[i] = page;
    pl.off[i] = off;
  }
}

template <int D>
struct Append {
  static constexpr int kGroups = D / 32;
  static constexpr int kTokens = kThreads / kGroups;  // a thread a group
  // bytes of a collected row: levels, pairs, and what keeps the rows' banks apart
  static constexpr int kRow = D == 128 ? 80 : 48;
  static constexpr int kPieces = D / 32;              // of 16 bytes, of a row's levels
};

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const __grid_constant__ Kv4AppendArgs a) {
  using C = Append<D>;
  constexpr int NG = C::kGroups;
  __shared__ Places<C::kTokens> pl;
  __shared__ __align__(16) unsigned char s_rows[C::kTokens * C::kRow];
  const int t0 = blockIdx.x * C::kTokens;
  const int h = blockIdx.y;
  const bool values = blockIdx.z != 0;
  const int i = threadIdx.x / NG, g = threadIdx.x % NG;
  const Kv4Rows& rows = values ? a.v : a.k;
  // (rows of no sequence may be read: they are there)
  Group<T> x{};
  const bool in = t0 + i < a.b.n_tokens;
  if (in)
    x.load(static_cast<const T*>(rows.ptr) + (long long)(t0 + i) * rows.token + (long long)h * rows.head +
           g * 32);
  find_places(a.b, t0, pl);
  const Quantised z = quantise(x);
  __syncthreads();
  const int page = pl.page[i], off = pl.off[i];
  unsigned char* row = s_rows + i * C::kRow;
  if (values) {
    // channels 4 r to 4 r + 3: half r & 1 of word r / 2, to place r (r ^ 4)
    const int turn = NG == 4 ? ((off >> 1) & 1) << 2 : 0;
#pragma unroll
    for (int r = 0; r < 8; ++r)
      *reinterpret_cast<uint16_t*>(row + (r ^ turn) * (D / 16) + 2 * g) = (uint16_t)(z.w[r >> 1] >> (16 * (r & 1)));
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) *reinterpret_cast<uint32_t*>(row + q * (D / 8) + 4 * g) = z.w[q];
  }
  *reinterpret_cast<uint32_t*>(row + D / 2 + 4 * g) = z.pair;
  T* stored = static_cast<T*>(values ? a.v_stored : a.k_stored);
  if (stored && page >= 0) {
    T* dst = stored + ((long long)h * a.b.n_tokens + t0 + i) * D + g * 32;
    const Unpacker u(z.pair);
#pragma unroll
    for (int q = 0; q < 4; ++q) store8(dst + 8 * q, u, z.w[q]);
  }
  __syncthreads();
  const int rec = kv4_rec_bytes(a.b.page, D);
  uint8_t* side = a.cache + ((long long)h * 2 + (values ? 1 : 0)) * rec;
#pragma unroll
  for (int y = threadIdx.x; y < C::kTokens * C::kPieces; y += kThreads) {
    const int tok = y / C::kPieces, piece = y % C::kPieces, pg = pl.page[tok];
    if (pg < 0) continue;
    *reinterpret_cast<uint4*>(side + (long long)pg * a.b.hkv * 2 * rec + pl.off[tok] * (D / 2) + piece * 16) =
        *reinterpret_cast<const uint4*>(s_rows + tok * C::kRow + piece * 16);
  }
  if (threadIdx.x < C::kTokens) {
    const int tok = threadIdx.x, pg = pl.page[tok];
    if (pg >= 0) {
      uint8_t* dst = side + (long long)pg * a.b.hkv * 2 * rec + a.b.page * (D / 2) + pl.off[tok] * (D / 8);
      const unsigned char* src = s_rows + tok * C::kRow + D / 2;
      if constexpr (NG == 4)
        *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
      else
        *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(src);
    }
  }
}

// Read: 4 threads a token, thread q the channels 32 g + 8 q to 32 g + 8 q + 7 of every
// group: for keys the q-th quarter of its levels, for values places 2 q and 2 q + 1 of 8, a
// quarter too (the other half's with the halves exchanged).
constexpr int kReadTokens = 128;

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const __grid_constant__ Kv4ReadArgs a) {
  constexpr int NG = D / 32;
  __shared__ Places<kReadTokens> pl;
  const int t0 = blockIdx.x * kReadTokens;
  const int h = blockIdx.y;
  const bool values = blockIdx.z != 0;
  T* out = static_cast<T*>(values ? a.v_out : a.k_out);
  if (!out) return;
  find_places(a.b, t0, pl);
  __syncthreads();
  const int q = threadIdx.x & 3;
  const int rec = kv4_rec_bytes(a.b.page, D);
  const uint8_t* side = a.cache + ((long long)h * 2 + (values ? 1 : 0)) * rec;
  constexpr int kPasses = kReadTokens * 4 / kThreads;
  uint32_t lev[kPasses][NG], pair[kPasses][NG];
#pragma unroll
  for (int x = 0; x < kPasses; ++x) {
    const int i = x * (kThreads / 4) + threadIdx.x / 4;
    const int page = pl.page[i], off = pl.off[i];
#pragma unroll
    for (int g = 0; g < NG; ++g) lev[x][g] = pair[x][g] = 0;
    if (page >= 0) {
      const uint8_t* src = side + (long long)page * a.b.hkv * 2 * rec;
      const int at = values && NG == 4 ? q ^ (off & 2) : q;
      const uint8_t* l = src + off * (D / 2) + at * (D / 8);
      const uint8_t* p = src + a.b.page * (D / 2) + off * (D / 8);
      if constexpr (NG == 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(l), w = *reinterpret_cast<const uint4*>(p);
        lev[x][0] = u.x, lev[x][1] = u.y, lev[x][NG - 2] = u.z, lev[x][NG - 1] = u.w;
        pair[x][0] = w.x, pair[x][1] = w.y, pair[x][NG - 2] = w.z, pair[x][NG - 1] = w.w;
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(l), w = *reinterpret_cast<const uint2*>(p);
        lev[x][0] = u.x, lev[x][1] = u.y;
        pair[x][0] = w.x, pair[x][1] = w.y;
      }
    }
  }
#pragma unroll
  for (int x = 0; x < kPasses; ++x) {
    const int i = x * (kThreads / 4) + threadIdx.x / 4;
    if (pl.page[i] == -2) continue;
    uint32_t w[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      // a value's words hold two groups' halves for places 2 q, then for 2 q + 1
      w[g] = !values ? lev[x][g]
                     : __byte_perm(lev[x][g >> 1], lev[x][(NG >> 1) + (g >> 1)], (g & 1) ? 0x7632 : 0x5410);
    }
    T* dst = out + ((long long)h * a.b.n_tokens + t0 + i) * D + q * 8;
#pragma unroll
    for (int g = 0; g < NG; ++g) store8(dst + 32 * g, Unpacker(pair[x][g]), w[g]);
  }
}

template <typename Args>
cudaError_t launch(void (*k64b)(Args), void (*k128b)(Args), void (*k64f)(Args),
                   void (*k128f)(Args), int tokens, const Args& a, cudaStream_t stream) {
  const dim3 grid((a.b.n_tokens + tokens - 1) / tokens, a.b.hkv, 2);
  auto k = a.dtype == SBSA_BF16 ? (a.d == 64 ? k64b : k128b) : (a.d == 64 ? k64f : k128f);
  k<<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendArgs& a, cudaStream_t stream) {
  return launch<Kv4AppendArgs>(kv4_append_kernel<64, __nv_bfloat16>,
                               kv4_append_kernel<128, __nv_bfloat16>, kv4_append_kernel<64, float>,
                               kv4_append_kernel<128, float>,
                               a.d == 64 ? Append<64>::kTokens : Append<128>::kTokens, a, stream);
}

cudaError_t launch_kv4_read(const Kv4ReadArgs& a, cudaStream_t stream) {
  return launch<Kv4ReadArgs>(kv4_read_kernel<64, __nv_bfloat16>, kv4_read_kernel<128, __nv_bfloat16>,
                             kv4_read_kernel<64, float>, kv4_read_kernel<128, float>, kReadTokens, a,
                             stream);
}

}  // namespace sbsa
