// The 4-bit key-value cache: quantising new tokens into their pages, and
// reading tokens back.  Format and layout: include/sbsa.h.
//
// Both kernels move bytes: append reads 2 d (bf16) or 4 d (fp32) bytes and
// writes 5/8 d for each token, kv head and side (key or value), read the
// reverse; HBM bounds them.  A lane takes 8 channels, so the 4 lanes of a
// group find its extremes in two shuffles, and in both layouts a lane's 8
// levels are one 32-bit word (keys) or two 16-bit halves (values) of the row.
// A CTA takes kTokens rows of one kv head and side: its levels and pairs land
// in contiguous parts of the pages, whatever the order of the inputs.
#include <cuda_runtime.h>

#include "kv4.cuh"

namespace sbsa {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 64;

struct F8 {
  float x[8];
};

__device__ __forceinline__ F8 load8(const float* p) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

__device__ __forceinline__ F8 load8(const __nv_bfloat16* p) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  F8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.x[2 * i] = __uint_as_float(w[i] << 16);
    r.x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  return r;
}

__device__ __forceinline__ void store8(float* p, const F8& v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v.x[0], v.x[1], v.x[2], v.x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v.x[4], v.x[5], v.x[6], v.x[7]);
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const F8& v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x[2 * i], v.x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// The 8 levels of a lane, channel i in bits 4 i of `w`: the lane's word of a
// key row, or its two halves of a value row (see include/sbsa.h).
template <int D>
__device__ __forceinline__ void put_levels(uint8_t* row, bool values, int off, int g, int q,
                                           uint32_t w) {
  if (!values) {
    *reinterpret_cast<uint32_t*>(row + q * (D / 8) + 4 * g) = w;
    return;
  }
  const int turn = D == 128 ? ((off >> 1) & 1) << 2 : 0;
  *reinterpret_cast<uint16_t*>(row + ((2 * q) ^ turn) * (D / 16) + 2 * g) = (uint16_t)w;
  *reinterpret_cast<uint16_t*>(row + ((2 * q + 1) ^ turn) * (D / 16) + 2 * g) = (uint16_t)(w >> 16);
}

template <int D>
__device__ __forceinline__ uint32_t get_levels(const uint8_t* row, bool values, int off, int g,
                                               int q) {
  if (!values) return *reinterpret_cast<const uint32_t*>(row + q * (D / 8) + 4 * g);
  const int turn = D == 128 ? ((off >> 1) & 1) << 2 : 0;
  const uint32_t lo = *reinterpret_cast<const uint16_t*>(row + ((2 * q) ^ turn) * (D / 16) + 2 * g);
  const uint32_t hi =
      *reinterpret_cast<const uint16_t*>(row + ((2 * q + 1) ^ turn) * (D / 16) + 2 * g);
  return lo | (hi << 16);
}

// low + scale * level: scale has 8 significant bits and level 4, so the
// product is exact and there is one rounding.
__device__ __forceinline__ F8 stands_for(uint32_t levels, float scale, float low) {
  F8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    r.x[i] = __fadd_rn(low, __fmul_rn(scale, (float)((levels >> (4 * i)) & 15u)));
  return r;
}

struct Quantised {
  uint32_t levels, pair;  // pair: scale in the low half, low in the high half
  float scale, low;
};

// The group of 32 channels that 4 neighbouring lanes hold, 8 each.
__device__ __forceinline__ Quantised quantise(const F8& v) {
  float mn = v.x[0], mx = v.x[0];
  bool finite = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    mn = fminf(mn, v.x[i]);
    mx = fmaxf(mx, v.x[i]);
    finite &= isfinite(v.x[i]);
  }
#pragma unroll
  for (int m = 1; m <= 2; m <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, m));
    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, m));
    finite &= __shfl_xor_sync(0xFFFFFFFFu, (int)finite, m) != 0;
  }
  mn = __fadd_rn(mn, 0.f);  // -0 becomes +0
  uint32_t bits = __float_as_uint(mn);
  if (bits >> 31) bits += 0xFFFFu;
  bits &= 0xFFFF0000u;  // rounded down to bf16
  const float low = __uint_as_float(bits);
  const float span = __fsub_rn(mx, low);
  const float step = __fmul_rn(span, 1.0f / 15.0f);
  const uint32_t up = (__float_as_uint(step) + 0xFFFFu) & 0xFFFF0000u;  // rounded up
  float scale = span < 0x1p-100f ? 0.f : __uint_as_float(up);
  finite &= isfinite(span) && isfinite(__uint_as_float(up));
  const float inv = scale > 0.f ? __frcp_rn(scale) : 0.f;
  Quantised r;
  r.levels = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float n = fminf(rintf(__fmul_rn(__fsub_rn(v.x[i], low), inv)), 15.f);
    r.levels |= (uint32_t)(finite ? (int)n : 0) << (4 * i);
  }
  r.pair = finite ? (__float_as_uint(scale) >> 16) | bits : 0x7FC07FC0u;
  r.scale = finite ? scale : __uint_as_float(0x7FC00000u);
  r.low = finite ? low : __uint_as_float(0x7FC00000u);
  return r;
}

// A CTA's rows: page and token of the page of each, page -1 where the row
// has no place, -2 where it belongs to no sequence.
struct Places {
  int page[kTokens];
  int off[kTokens];
};

__device__ __forceinline__ void find_places(const Kv4Batch& b, int t0, Places& pl) {
  for (int i = threadIdx.x; i < kTokens; i += kThreads) {
    int page = -2, off = 0;
    if (t0 + i < b.n_tokens) {
      bool in_seq;
      if (!kv4_place(b, t0 + i, &in_seq, &page, &off)) page = in_seq ? -1 : -2;
    }
    pl.page[i] = page;
    pl.off[i] = off;
  }
  __syncthreads();
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const Kv4AppendArgs a) {
  __shared__ Places pl;
  constexpr int kLanes = D / 8;  // lanes of a row
  const int t0 = blockIdx.x * kTokens;
  const int h = blockIdx.y;
  const bool values = blockIdx.z != 0;
  find_places(a.b, t0, pl);
  const Kv4Rows& rows = values ? a.v : a.k;
  T* stored = static_cast<T*>(values ? a.v_stored : a.k_stored);
  const int lane = threadIdx.x % kLanes, g = lane >> 2, q = lane & 3;
  const int rec = kv4_rec_bytes(a.b.page, D);
  for (int i = threadIdx.x / kLanes; i < kTokens; i += kThreads / kLanes) {
    const bool on = pl.page[i] >= 0;
    const T* src = static_cast<const T*>(rows.ptr) + (long long)(t0 + i) * rows.token +
                   (long long)h * rows.head + lane * 8;
    F8 v{};
    if (on) v = load8(src);
    const Quantised z = quantise(v);
    if (!on) continue;
    const int off = pl.off[i];
    uint8_t* dst = a.cache + (((long long)pl.page[i] * a.b.hkv + h) * 2 + (values ? 1 : 0)) * rec;
    put_levels<D>(dst + off * (D / 2), values, off, g, q, z.levels);
    if (q == 0)
      *reinterpret_cast<uint32_t*>(dst + a.b.page * (D / 2) + off * (D / 8) + g * 4) = z.pair;
    if (stored)
      store8(stored + ((long long)h * a.b.n_tokens + t0 + i) * D + lane * 8,
             stands_for(z.levels, z.scale, z.low));
  }
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const Kv4ReadArgs a) {
  __shared__ Places pl;
  constexpr int kLanes = D / 8;
  const int t0 = blockIdx.x * kTokens;
  const int h = blockIdx.y;
  const bool values = blockIdx.z != 0;
  T* out = static_cast<T*>(values ? a.v_out : a.k_out);
  if (!out) return;
  find_places(a.b, t0, pl);
  const int lane = threadIdx.x % kLanes, g = lane >> 2, q = lane & 3;
  const int rec = kv4_rec_bytes(a.b.page, D);
  for (int i = threadIdx.x / kLanes; i < kTokens; i += kThreads / kLanes) {
    if (pl.page[i] == -2) continue;
    F8 v{};
    if (pl.page[i] >= 0) {
      const int off = pl.off[i];
      const uint8_t* src =
          a.cache + (((long long)pl.page[i] * a.b.hkv + h) * 2 + (values ? 1 : 0)) * rec;
      const uint32_t levels = get_levels<D>(src + off * (D / 2), values, off, g, q);
      const uint32_t pair =
          *reinterpret_cast<const uint32_t*>(src + a.b.page * (D / 2) + off * (D / 8) + g * 4);
      v = stands_for(levels, __uint_as_float(pair << 16), __uint_as_float(pair & 0xFFFF0000u));
    }
    store8(out + ((long long)h * a.b.n_tokens + t0 + i) * D + lane * 8, v);
  }
}

template <typename Args>
cudaError_t launch(void (*k64b)(Args), void (*k128b)(Args), void (*k64f)(Args),
                   void (*k128f)(Args), const Args& a, cudaStream_t stream) {
  const dim3 grid((a.b.n_tokens + kTokens - 1) / kTokens, a.b.hkv, 2);
  auto k = a.dtype == SBSA_BF16 ? (a.d == 64 ? k64b : k128b) : (a.d == 64 ? k64f : k128f);
  k<<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendArgs& a, cudaStream_t stream) {
  return launch<Kv4AppendArgs>(kv4_append_kernel<64, __nv_bfloat16>,
                               kv4_append_kernel<128, __nv_bfloat16>, kv4_append_kernel<64, float>,
                               kv4_append_kernel<128, float>, a, stream);
}

cudaError_t launch_kv4_read(const Kv4ReadArgs& a, cudaStream_t stream) {
  return launch<Kv4ReadArgs>(kv4_read_kernel<64, __nv_bfloat16>, kv4_read_kernel<128, __nv_bfloat16>,
                             kv4_read_kernel<64, float>, kv4_read_kernel<128, float>, a, stream);
}

}  // namespace sbsa
