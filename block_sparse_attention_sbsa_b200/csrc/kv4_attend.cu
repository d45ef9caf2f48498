// Attention over the 4-bit key-value cache: the direct form.  A CTA takes one
// row (token, query head); its warps share out the row's tokens, each with the
// running maximum and sum of its part, joined at the end.  All arithmetic is
// fp32 on the values that the cache stands for.
#include <cuda_runtime.h>

#include "kv4.cuh"

namespace sbsa {
namespace {

constexpr int kWarps = 8;

template <int D>
__device__ __forceinline__ float cached(const uint8_t* rec, bool values, int page, int off, int c) {
  const int g = c / 32, i = c % (values ? 4 : 8), lane = c % 32 / (values ? 4 : 8);
  int byte;
  if (values) {
    const int turn = D == 128 ? ((off >> 1) & 1) << 2 : 0;
    byte = (lane ^ turn) * (D / 16) + 2 * g + i / 2;
  } else {
    byte = lane * (D / 8) + 4 * g + i / 2;
  }
  const uint32_t level = (rec[off * (D / 2) + byte] >> (4 * (i & 1))) & 15u;
  const uint32_t pair =
      *reinterpret_cast<const uint32_t*>(rec + page * (D / 2) + off * (D / 8) + g * 4);
  return fmaf(__uint_as_float(pair << 16), (float)level, __uint_as_float(pair & 0xFFFF0000u));
}

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16(x); }

template <int D, typename T>
__global__ void __launch_bounds__(kWarps * 32) kv4_attend_kernel(const Kv4AttendArgs a) {
  __shared__ float acc[kWarps][D];
  __shared__ float top[kWarps], sum[kWarps];
  const int t = blockIdx.x, h = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = kv4_seq_of(a.b, t);
  if (s < 0) return;
  const int len = kv4_len(a.b, s);
  const long long pos = (long long)len - a.b.cu[s + 1] + t;
  const bool on = pos >= 0 && t - a.b.cu[s] < a.max_new;
  if (!on) kv4_record(a.b.status);
  const int g = h / (a.hq / a.b.hkv);
  float q[D / 32], o[D / 32] = {};
  for (int i = 0; i < D / 32; ++i)
    q[i] = as_float(static_cast<const T*>(a.q.ptr)[t * a.q.token + h * a.q.head + i * 32 + lane]);
  const int rec = kv4_rec_bytes(a.b.page, D);
  float m = -INFINITY, l = 0.f;
  const int32_t* list = nullptr;
  int n = on ? (int)pos + 1 : 0;
  if (on && a.list_heads) {
    const long long row = (long long)s * a.list_heads + h / (a.hq / a.list_heads);
    list = a.idx + row * a.max_blocks;
    n = clamp_int(a.cnt[row], 0, a.max_blocks) * a.block;
  }
  for (int i = warp; i < n; i += kWarps) {
    int u = i;
    if (list) {
      const int j = list[i / a.block];
      const bool in = j >= 0 && j <= (len - 1) / a.block;
      if (!in) kv4_record(a.b.status);
      if (!in) continue;
      u = j * a.block + i % a.block;
      if (u > pos) continue;
    }
    const int page = a.b.table[(long long)s * a.b.max_pages + u / a.b.page];
    if (page < 0 || page >= a.b.n_pages) {
      kv4_record(a.b.status);
      continue;
    }
    const uint8_t* keys = a.cache + ((long long)page * a.b.hkv + g) * 2 * rec;
    float x = 0.f;
    for (int j = 0; j < D / 32; ++j)
      x += q[j] * cached<D>(keys, false, a.b.page, u % a.b.page, j * 32 + lane);
    for (int w = 16; w; w >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, w);
    x *= a.sm_scale;
    const float m2 = fmaxf(m, x);
    const float scale = m == -INFINITY ? 0.f : expf(m - m2), p = expf(x - m2);
    l = l * scale + p;
    for (int j = 0; j < D / 32; ++j)
      o[j] = o[j] * scale + p * cached<D>(keys + rec, true, a.b.page, u % a.b.page, j * 32 + lane);
    m = m2;
  }
  for (int j = 0; j < D / 32; ++j) acc[warp][j * 32 + lane] = o[j];
  if (lane == 0) {
    top[warp] = m;
    sum[warp] = l;
  }
  __syncthreads();
  float mx = -INFINITY, total = 0.f;
  for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, top[w]);
  for (int w = 0; w < kWarps; ++w) total += sum[w] == 0.f ? 0.f : sum[w] * expf(top[w] - mx);
  for (int c = threadIdx.x; c < D; c += kWarps * 32) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w)
      x += sum[w] == 0.f ? 0.f : acc[w][c] * expf(top[w] - mx);
    put(static_cast<T*>(a.o) + t * a.o_token + h * a.o_head + c, total == 0.f ? 0.f : x / total);
  }
}

}  // namespace

size_t kv4_attend_workspace(int) { return 256; }

int launch_kv4_attend(const Kv4AttendArgs& a, cudaStream_t stream) {
  auto k = a.dtype == SBSA_BF16
               ? (a.d == 64 ? kv4_attend_kernel<64, __nv_bfloat16> : kv4_attend_kernel<128, __nv_bfloat16>)
               : (a.d == 64 ? kv4_attend_kernel<64, float> : kv4_attend_kernel<128, float>);
  k<<<dim3(a.b.n_tokens, a.hq), kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? SBSA_OK : SBSA_ERR_CUDA;
}

}  // namespace sbsa
