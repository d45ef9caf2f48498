// Device helpers shared by the kernels of the 4-bit key-value cache.
#pragma once
#include <cuda_bf16.h>

#include "kv4.h"

namespace sbsa {

__device__ __forceinline__ void kv4_record(int* status) {
  if (status) atomicCAS(status, 0, SBSA_ERR_DEVICE);
}

// Bytes of one page's keys (or values) of one kv head.
__host__ __device__ constexpr int kv4_rec_bytes(int page, int d) { return page * (d / 8) * 5; }

__device__ __forceinline__ int clamp_int(int x, int lo, int hi) {
  return x < lo ? lo : (x > hi ? hi : x);
}

// Tokens of a sequence whose length is given as n that its row of the page table can name.
__device__ __forceinline__ int kv4_named(const Kv4Batch& b, int n) {
  const int c = clamp_int(n, 0, b.max_pages * b.page);
  if (c != n) kv4_record(b.status);
  return c;
}

// The sequence that row t belongs to: the last one whose first row is not
// behind t; -1 when there is none or t lies behind its last row.
__device__ __forceinline__ int kv4_seq_of(const Kv4Batch& b, int t) {
  int lo = 0, hi = b.n_seqs + 1;  // the first i with cu[i] > t lies in [lo, hi]
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (b.cu[mid] > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo >= 1 && lo <= b.n_seqs ? lo - 1 : -1;
}

// Reports a batch that names rows before the tensors' first or behind their last.
__device__ __forceinline__ void kv4_check_rows(const Kv4Batch& b) {
  if (b.cu[0] < 0 || b.cu[b.n_seqs] > b.n_tokens) kv4_record(b.status);
}

// Page number and token of the page of row t; false (and recorded where it
// is an error) when row t has no place in the cache.  *in_seq tells whether
// the row belongs to a sequence at all.
__device__ __forceinline__ bool kv4_place(const Kv4Batch& b, int t, bool* in_seq, int* page,
                                          int* off) {
  const int s = kv4_seq_of(b, t);
  *in_seq = s >= 0;
  if (s < 0) return false;
  // positions go by the length as it is given, also where the table ends before it
  const int len = b.lens[s];
  const long long pos = (long long)len - b.cu[s + 1] + t;
  if (pos < 0 || pos >= kv4_named(b, len)) {
    kv4_record(b.status);
    return false;
  }
  const int page_log = __ffs(b.page) - 1;  // a power of two
  const int pg = b.table[(long long)s * b.max_pages + ((int)pos >> page_log)];
  if (pg < 0 || pg >= b.n_pages) {
    kv4_record(b.status);
    return false;
  }
  *page = pg;
  *off = (int)pos & (b.page - 1);
  return true;
}

}  // namespace sbsa
