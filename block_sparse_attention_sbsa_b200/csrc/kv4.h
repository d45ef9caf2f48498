// Internal interfaces of the 4-bit key-value cache (see include/sbsa.h for
// the format, the layout and the description of a batch).
#pragma once
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "sbsa.h"

namespace sbsa {

// A batch as every kernel of the cache takes it.
struct Kv4Batch {
  const int32_t* table;  // [n_seqs, max_pages]
  const int32_t* lens;   // [n_seqs]
  const int32_t* cu;     // [n_seqs + 1]
  int n_seqs, n_tokens, max_pages, n_pages, page, hkv;
  int* status;
};

struct Kv4Rows {
  const void* ptr;
  int64_t token, head;  // strides in elements
};

struct Kv4AppendArgs {
  Kv4Batch b;
  uint8_t* cache;
  Kv4Rows k, v;
  void *k_stored, *v_stored;  // contiguous [Hkv, n_tokens, d], or nullptr
  int d, dtype;
};
cudaError_t launch_kv4_append(const Kv4AppendArgs& a, cudaStream_t stream);

struct Kv4ReadArgs {
  Kv4Batch b;
  const uint8_t* cache;
  void *k_out, *v_out;  // contiguous [Hkv, n_tokens, d], or nullptr
  int d, dtype;
};
cudaError_t launch_kv4_read(const Kv4ReadArgs& a, cudaStream_t stream);

struct Kv4AttendArgs {
  Kv4Batch b;
  const uint8_t* cache;
  Kv4Rows q;
  void* o;
  int64_t o_token, o_head;
  const int32_t* idx;  // [n_seqs, list_heads, max_blocks], or nullptr
  const int32_t* cnt;
  int hq, d, dtype, max_new, list_heads, block, max_blocks;
  float sm_scale;
  void* workspace;
};
// The two kernels of the attention, and the bytes of their partial results: for few
// rows a sequence (all types, with lists), and for many (bf16, without lists).
// The launchers return an SBSA_* code.
size_t kv4_few_workspace(const Kv4AttendArgs& a);
int launch_kv4_few(const Kv4AttendArgs& a, cudaStream_t stream);
size_t kv4_many_workspace(const Kv4AttendArgs& a);
int launch_kv4_many(const Kv4AttendArgs& a, cudaStream_t stream);

}  // namespace sbsa
