// C-ABI entry points of the 4-bit key-value cache: argument checks (before
// any launch) and dispatch to the launchers.
#include <cmath>
#include <cstdint>

#include "internal.h"
#include "kv4.h"

namespace sbsa {
namespace {

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

// What all three operators check.
int validate_kv4(const sbsa_kv4_params* p) {
  if (!p) return SBSA_ERR_INVALID_ARG;
  if (p->n_kv_heads < 1 || p->head_dim < 1 || p->page_size < 1 || p->n_pages < 1 ||
      p->max_pages < 1 || p->n_seqs < 0 || p->n_tokens < 0)
    return SBSA_ERR_INVALID_ARG;
  if (p->dtype != SBSA_BF16 && p->dtype != SBSA_FP32) return SBSA_ERR_INVALID_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return SBSA_ERR_UNSUPPORTED;
  if (p->page_size != 16 && p->page_size != 32 && p->page_size != 64 && p->page_size != 128)
    return SBSA_ERR_UNSUPPORTED;
  if (p->n_kv_heads > 65535) return SBSA_ERR_UNSUPPORTED;
  // positions are 32-bit (with room for one tile behind the last token)
  if ((long long)p->max_pages * p->page_size > 0x7FFF0000LL) return SBSA_ERR_UNSUPPORTED;
  if (p->n_tokens > 0x7FFF0000 || p->n_seqs > 0x7FFF0000) return SBSA_ERR_UNSUPPORTED;
  return SBSA_OK;
}

int validate_attend(const sbsa_kv4_params* p) {
  int rc = validate_kv4(p);
  if (rc) return rc;
  if (p->n_q_heads < 1 || p->n_q_heads % p->n_kv_heads != 0) return SBSA_ERR_INVALID_ARG;
  if (p->max_new < 1) return SBSA_ERR_INVALID_ARG;
  if (!(p->sm_scale >= 0.f) || !std::isfinite(p->sm_scale)) return SBSA_ERR_INVALID_ARG;
  if (p->n_q_heads > 65535) return SBSA_ERR_UNSUPPORTED;
  // rows and (sequence, head) pairs are numbered in 32 bits
  if ((long long)p->n_tokens * p->n_q_heads > 0x7FFF0000LL ||
      (long long)p->n_seqs * p->n_q_heads > 0x7FFF0000LL)
    return SBSA_ERR_UNSUPPORTED;
  if (p->list_heads) {
    if (p->list_heads != p->n_kv_heads && p->list_heads != p->n_q_heads)
      return SBSA_ERR_INVALID_ARG;
    if (p->max_blocks < 1 || p->block_size < 1) return SBSA_ERR_INVALID_ARG;
    if (p->block_size != 64 && p->block_size != 128) return SBSA_ERR_UNSUPPORTED;
    if (p->block_size % p->page_size != 0) return SBSA_ERR_INVALID_ARG;
    if ((long long)p->max_blocks * p->block_size > 0x7FFF0000LL) return SBSA_ERR_UNSUPPORTED;
  }
  return SBSA_OK;
}

// Strides between tokens and heads: whole multiples of 16 bytes.
bool strides_ok(const sbsa_kv4_params* p, int64_t token, int64_t head) {
  const int64_t per16 = p->dtype == SBSA_BF16 ? 8 : 4;
  return token >= 0 && head >= 0 && token % per16 == 0 && head % per16 == 0;
}

bool batch_given(const int32_t* table, const int32_t* lens, const int32_t* cu) {
  return table && lens && cu;
}

Kv4Batch batch(const sbsa_kv4_params* p, const int32_t* table, const int32_t* lens,
               const int32_t* cu) {
  Kv4Batch b{};
  b.table = table;
  b.lens = lens;
  b.cu = cu;
  b.n_seqs = p->n_seqs;
  b.n_tokens = p->n_tokens;
  b.max_pages = p->max_pages;
  b.n_pages = p->n_pages;
  b.page = p->page_size;
  b.hkv = p->n_kv_heads;
  b.status = device_status_ptr();
  return b;
}

// Which kernel: the one for many rows reads the cache once for 256 rows, the other one for
// 16, but spends less on what it reads, so that it takes up to two reads (d = 128) or three
// (d = 64) to equal it.  12 sequences of 907 to 20011 tokens, 8 kv heads, all with the same number
// of rows (bursts of 10 ms, in a graph): d = 128, 32 rows few 81 us, many 111, 36 to 48 rows 115 and
// 111; d = 64, 40 and 48 rows 79 and 92, 52 rows 102 and 92.  The host knows max_new alone, so one
// chunk takes a batch's single tokens along: 47 of them over 211 to 16411 tokens with a chunk of 512
// over 8192, d = 128, are 334 us in one call (many), 190 in two.
bool many_rows(const sbsa_kv4_params* p) {
  return p->dtype == SBSA_BF16 && !p->list_heads &&
         (long long)p->max_new * (p->n_q_heads / p->n_kv_heads) > (p->head_dim == 64 ? 48 : 32);
}

// The sizes that the launchers go by (no pointers).
Kv4AttendArgs attend_sizes(const sbsa_kv4_params* p) {
  Kv4AttendArgs a{};
  a.b.n_seqs = p->n_seqs;
  a.b.n_tokens = p->n_tokens;
  a.b.max_pages = p->max_pages;
  a.b.n_pages = p->n_pages;
  a.b.page = p->page_size;
  a.b.hkv = p->n_kv_heads;
  a.hq = p->n_q_heads;
  a.d = p->head_dim;
  a.dtype = p->dtype;
  a.max_new = p->max_new;
  a.list_heads = p->list_heads;
  a.block = p->block_size;
  a.max_blocks = p->max_blocks;
  return a;
}

size_t attend_workspace(const sbsa_kv4_params* p) {
  const Kv4AttendArgs a = attend_sizes(p);
  return many_rows(p) ? kv4_many_workspace(a) : kv4_few_workspace(a);
}

int cuda_code(cudaError_t e) { return e == cudaSuccess ? SBSA_OK : SBSA_ERR_CUDA; }

}  // namespace
}  // namespace sbsa

using namespace sbsa;

extern "C" {

size_t sbsa_kv4_cache_bytes(const sbsa_kv4_params* p) {
  if (validate_kv4(p) != SBSA_OK) return 0;
  return (size_t)p->n_pages * p->n_kv_heads * 2 * p->page_size * (p->head_dim / 8) * 5;
}

int sbsa_kv4_append(const sbsa_kv4_params* p, void* cache, const int32_t* page_table,
                    const int32_t* seq_lens, const int32_t* cu_new, const void* k,
                    int64_t k_token_stride, int64_t k_head_stride, const void* v,
                    int64_t v_token_stride, int64_t v_head_stride, void* k_stored,
                    void* v_stored, void* stream) {
  int rc = validate_kv4(p);
  if (rc) return rc;
  if (!strides_ok(p, k_token_stride, k_head_stride) ||
      !strides_ok(p, v_token_stride, v_head_stride))
    return SBSA_ERR_INVALID_ARG;
  if (p->n_seqs == 0 || p->n_tokens == 0) return SBSA_OK;
  if (!cache || !batch_given(page_table, seq_lens, cu_new) || !k || !v)
    return SBSA_ERR_INVALID_ARG;
  if (!aligned16(cache) || !aligned16(k) || !aligned16(v) || !aligned16(k_stored) ||
      !aligned16(v_stored))
    return SBSA_ERR_INVALID_ARG;
  Kv4AppendArgs a{};
  a.b = batch(p, page_table, seq_lens, cu_new);
  a.cache = static_cast<uint8_t*>(cache);
  a.k = Kv4Rows{k, k_token_stride, k_head_stride};
  a.v = Kv4Rows{v, v_token_stride, v_head_stride};
  a.k_stored = k_stored;
  a.v_stored = v_stored;
  a.d = p->head_dim;
  a.dtype = p->dtype;
  return cuda_code(launch_kv4_append(a, static_cast<cudaStream_t>(stream)));
}

int sbsa_kv4_read(const sbsa_kv4_params* p, const void* cache, const int32_t* page_table,
                  const int32_t* seq_lens, const int32_t* cu_new, void* k_out, void* v_out,
                  void* stream) {
  int rc = validate_kv4(p);
  if (rc) return rc;
  if (p->n_seqs == 0 || p->n_tokens == 0 || (!k_out && !v_out)) return SBSA_OK;
  if (!cache || !batch_given(page_table, seq_lens, cu_new)) return SBSA_ERR_INVALID_ARG;
  if (!aligned16(cache) || !aligned16(k_out) || !aligned16(v_out)) return SBSA_ERR_INVALID_ARG;
  Kv4ReadArgs a{};
  a.b = batch(p, page_table, seq_lens, cu_new);
  a.cache = static_cast<const uint8_t*>(cache);
  a.k_out = k_out;
  a.v_out = v_out;
  a.d = p->head_dim;
  a.dtype = p->dtype;
  return cuda_code(launch_kv4_read(a, static_cast<cudaStream_t>(stream)));
}

size_t sbsa_kv4_attend_workspace_bytes(const sbsa_kv4_params* p) {
  if (validate_attend(p) != SBSA_OK) return 0;
  return attend_workspace(p);
}

int sbsa_kv4_attend(const sbsa_kv4_params* p, const void* cache, const int32_t* page_table,
                    const int32_t* seq_lens, const int32_t* cu_new, const void* q,
                    int64_t q_token_stride, int64_t q_head_stride, void* o,
                    int64_t o_token_stride, int64_t o_head_stride, const int32_t* idx,
                    const int32_t* cnt, void* workspace, size_t ws_bytes, void* stream) {
  int rc = validate_attend(p);
  if (rc) return rc;
  if (!strides_ok(p, q_token_stride, q_head_stride) ||
      !strides_ok(p, o_token_stride, o_head_stride))
    return SBSA_ERR_INVALID_ARG;
  if (p->n_seqs == 0 || p->n_tokens == 0) return SBSA_OK;
  if (!cache || !batch_given(page_table, seq_lens, cu_new) || !q || !o)
    return SBSA_ERR_INVALID_ARG;
  if (p->list_heads ? (!idx || !cnt) : (idx || cnt)) return SBSA_ERR_INVALID_ARG;
  if (!aligned16(cache) || !aligned16(q) || !aligned16(o)) return SBSA_ERR_INVALID_ARG;
  const size_t need = attend_workspace(p);
  if (need && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || ws_bytes < need))
    return SBSA_ERR_WORKSPACE;
  Kv4AttendArgs a = attend_sizes(p);
  a.b = batch(p, page_table, seq_lens, cu_new);
  a.cache = static_cast<const uint8_t*>(cache);
  a.q = Kv4Rows{q, q_token_stride, q_head_stride};
  a.o = o;
  a.o_token = o_token_stride;
  a.o_head = o_head_stride;
  a.idx = idx;
  a.cnt = cnt;
  a.sm_scale = p->sm_scale > 0.f ? p->sm_scale : 1.0f / std::sqrt((float)p->head_dim);
  a.workspace = workspace;
  auto launch = many_rows(p) ? launch_kv4_many : launch_kv4_few;
  return launch(a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
