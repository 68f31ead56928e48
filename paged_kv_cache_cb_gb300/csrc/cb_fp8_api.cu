// Entry points of the 8-bit KV cache (include/cbattn.h): argument checks and
// dispatch.  Host code only.
#include <algorithm>
#include <atomic>

#include "../../include/cbattn.h"
#include "cb_internal.h"

using namespace cb;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The cache arguments shared by every entry point; false: CB_EINVAL.
bool cache_of(Fp8Cache* c, const void* k, const void* v, const void* ke, const void* ve, int num_blocks, int n_kv_heads,
              int head_dim, int block_size) {
  if (num_blocks <= 0 || n_kv_heads <= 0 || (head_dim != 64 && head_dim != 128) || block_size != kBlockSize) return false;
  if ((long long)num_blocks * n_kv_heads * kBlockSize >= (1LL << 31) - kBlockSize) return false;
  if (!k || !v || !ke || !ve || !aligned16(k) || !aligned16(v) || !aligned16(ke) || !aligned16(ve)) return false;
  c->k = static_cast<uint8_t*>(const_cast<void*>(k));
  c->v = static_cast<uint8_t*>(const_cast<void*>(v));
  c->k_exps = static_cast<uint8_t*>(const_cast<void*>(ke));
  c->v_exps = static_cast<uint8_t*>(const_cast<void*>(ve));
  c->num_blocks = num_blocks;
  c->n_kv_heads = n_kv_heads;
  c->head_dim = head_dim;
  return true;
}

// No C++ exception (an allocation or a lock of the library's host state) leaves an entry point.
template <class F>
int guarded(F call) {
  try {
    return call();
  } catch (...) {
    return CB_ECUDA;
  }
}

struct NewRows {
  const void* k;
  const void* v;
  const int64_t* slots;
};

// A step's workspace: the single tokens' part, the chunks', the ready word.
size_t round_up(size_t x) { return (x + 255) / 256 * 256; }
size_t single_bytes(int head_dim) { return round_up(fp8_partials_bytes(kSingleRows, head_dim)); }
size_t ready_at(int head_dim) { return single_bytes(head_dim) + round_up(fp8_partials_bytes(kChunkRows, head_dim)); }

// A number that no other call of the process has (a recorded call keeps its own; its
// last kernel clears the word).
unsigned long long next_ticket() {
  static std::atomic<unsigned long long> n{0x6b1d3f5a00000001ull};
  return n.fetch_add(1, std::memory_order_relaxed);
}

int step_fp8(const NewRows* app, const void* q, const int32_t* cu_q_lens, const int32_t* ctx_lens,
             const int32_t* block_tables, int max_blocks_per_seq, int n_reqs, int n_tokens, int max_q_len,
             int max_kv_len, const void* k_cache, const void* v_cache, const void* k_exps, const void* v_exps,
             int num_blocks, void* out, float scale, int n_q_heads, int n_kv_heads, int head_dim, int block_size,
             int window, void* workspace, size_t workspace_bytes, void* stream) {
  if (!supported_shape(n_q_heads, n_kv_heads, head_dim, block_size) || window < 0) return CB_EINVAL;
  if (n_reqs < 0 || n_reqs > CB_MAX_REQS || n_tokens < 0 || max_q_len < 1 || max_kv_len < 1 ||
      max_blocks_per_seq < 1 || num_blocks <= 0 || !(scale > 0.f) || max_q_len > max_kv_len)
    return CB_EINVAL;
  if (n_reqs == 0 || n_tokens == 0) {
    set_last_launches(0);
    return CB_OK;
  }
  Fp8Step s{};
  if (!cache_of(&s.cache, k_cache, v_cache, k_exps, v_exps, num_blocks, n_kv_heads, head_dim, block_size))
    return CB_EINVAL;
  // the kernels count tiles of the step in 32 bits, with the empty places before them (single tokens: up to 6)
  const long long blocks = std::min<long long>(max_blocks_per_seq, ((long long)max_kv_len + kBlockSize - 1) / kBlockSize);
  const long long tok = kTileM / (n_q_heads / n_kv_heads), items = n_tokens / (2 * tok) + n_reqs;
  if ((blocks + 7) * n_reqs * n_kv_heads >= 1LL << 31 ||
      items * (((long long)max_kv_len + kTileN - 1) / kTileN + kChunkLead) * n_kv_heads >= 1LL << 31)
    return CB_EINVAL;
  if (!q || !cu_q_lens || !ctx_lens || !block_tables || !out || !workspace) return CB_EINVAL;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace)) return CB_EINVAL;
  if (app && (!app->k || !app->v || !app->slots || !aligned16(app->k) || !aligned16(app->v))) return CB_EINVAL;
  if (workspace_bytes < cb_paged_attention_fp8_workspace_size(n_reqs, n_tokens, max_q_len, max_kv_len, n_q_heads,
                                                              n_kv_heads, head_dim, block_size))
    return CB_EWORKSPACE;
  int sms = 0;
  if (!device_sms(&sms)) return CB_ECUDA;
  sms = sms < kMaxDecodeGrid ? sms : kMaxDecodeGrid;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int rc = CB_OK;
  s.err = stream_error_word(st, &rc);
  if (!s.err) return rc;
  s.q = static_cast<const uint16_t*>(q);
  s.cu_q_lens = cu_q_lens;
  s.ctx_lens = ctx_lens;
  s.block_tables = block_tables;
  s.out = static_cast<uint16_t*>(out);
  s.max_blocks_per_seq = max_blocks_per_seq;
  s.n_reqs = n_reqs;
  s.n_tokens = n_tokens;
  s.max_q_len = max_q_len;
  s.max_kv_len = max_kv_len;
  s.n_q_heads = n_q_heads;
  s.window = window;
  s.scale_log2 = scale * 1.4426950408889634f;
  if (max_q_len > 1) {
    s.ready = reinterpret_cast<unsigned long long*>(static_cast<uint8_t*>(workspace) + ready_at(head_dim));
    s.ticket = next_ticket();
  }
  if (app && launch_append_fp8(app->k, app->v, app->slots, n_tokens, s.cache, s.err, st) != cudaSuccess)
    return CB_ECUDA;
  int launches = app ? 1 : 0;
  // the single tokens, the chunks, then what both have cut into pieces
  const int group = n_q_heads / n_kv_heads;
  const bool tiles = fp8_decode_shape(head_dim, group), many = max_q_len > 1;
  const Fp8Partials singles = fp8_partials(workspace, kSingleRows);
  const Fp8Partials chunks = fp8_partials(static_cast<uint8_t*>(workspace) + single_bytes(head_dim), kChunkRows);
  if ((tiles ? launch_decode_fp8(s, singles, sms, app != nullptr, st)
             : launch_chunk_fp8(s, singles, true, sms, app != nullptr, st)) != cudaSuccess ||
      (many && launch_chunk_fp8(s, chunks, false, sms, true, st) != cudaSuccess) ||
      launch_join_fp8(s, singles, tiles ? fp8_head_group(n_kv_heads) * group : group, many ? &chunks : nullptr, sms, st) != cudaSuccess)
    return CB_ECUDA;
  launches += many ? 3 : 2;
  set_last_launches(launches);
  return CB_OK;
}

}  // namespace

extern "C" {

int cb_kv_append_fp8(const void* k_new, const void* v_new, const int64_t* slot_mapping, int n_tokens, void* k_cache,
                     void* v_cache, void* k_exps, void* v_exps, int num_blocks, int n_kv_heads, int head_dim,
                     int block_size, void* stream) {
  return guarded([&]() -> int {
    Fp8Cache c;
    if (n_tokens < 0 || !cache_of(&c, k_cache, v_cache, k_exps, v_exps, num_blocks, n_kv_heads, head_dim, block_size))
      return CB_EINVAL;
    if (n_tokens == 0) {
      set_last_launches(0);
      return CB_OK;
    }
    if (!k_new || !v_new || !slot_mapping || !aligned16(k_new) || !aligned16(v_new)) return CB_EINVAL;
    int rc = CB_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    unsigned int* err = stream_error_word(st, &rc);
    if (!err) return rc;
    if (launch_append_fp8(k_new, v_new, slot_mapping, n_tokens, c, err, st) != cudaSuccess) return CB_ECUDA;
    set_last_launches(1);
    return CB_OK;
  });
}

int cb_kv_gather_fp8(const int64_t* slot_mapping, int n_rows, const void* k_cache, const void* v_cache,
                     const void* k_exps, const void* v_exps, int num_blocks, void* k_out, void* v_out, int n_kv_heads,
                     int head_dim, int block_size, void* stream) {
  return guarded([&]() -> int {
    Fp8Cache c;
    if (n_rows < 0 || !cache_of(&c, k_cache, v_cache, k_exps, v_exps, num_blocks, n_kv_heads, head_dim, block_size))
      return CB_EINVAL;
    if (n_rows == 0) {
      set_last_launches(0);
      return CB_OK;
    }
    if (!k_out || !v_out || !slot_mapping || !aligned16(k_out) || !aligned16(v_out)) return CB_EINVAL;
    int rc = CB_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    unsigned int* err = stream_error_word(st, &rc);
    if (!err) return rc;
    if (launch_gather_fp8(slot_mapping, n_rows, c, k_out, v_out, err, st) != cudaSuccess) return CB_ECUDA;
    set_last_launches(1);
    return CB_OK;
  });
}

int cb_copy_blocks_fp8(const int32_t* pairs, int n_pairs, void* k_cache, void* v_cache, void* k_exps, void* v_exps,
                       int num_blocks, int n_kv_heads, int head_dim, int block_size, void* stream) {
  return guarded([&]() -> int {
    Fp8Cache c;
    if (n_pairs < 0 || n_pairs > 65535 ||
        !cache_of(&c, k_cache, v_cache, k_exps, v_exps, num_blocks, n_kv_heads, head_dim, block_size))
      return CB_EINVAL;
    if (n_pairs == 0) {
      set_last_launches(0);
      return CB_OK;
    }
    if (!pairs) return CB_EINVAL;
    int rc = CB_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    unsigned int* err = stream_error_word(st, &rc);
    if (!err) return rc;
    if (launch_copy_blocks_fp8(pairs, n_pairs, c, err, st) != cudaSuccess) return CB_ECUDA;
    set_last_launches(1);
    return CB_OK;
  });
}

size_t cb_paged_attention_fp8_workspace_size(int n_reqs, int n_tokens, int max_q_len, int max_kv_len, int n_q_heads,
                                             int n_kv_heads, int head_dim, int block_size) {
  if (n_reqs < 0 || n_reqs > CB_MAX_REQS || n_tokens < 0 || max_q_len < 1 || max_kv_len < 1 ||
      !supported_shape(n_q_heads, n_kv_heads, head_dim, block_size))
    return 0;
  return max_q_len > 1 ? ready_at(head_dim) + 16 : single_bytes(head_dim);
}

int cb_paged_attention_fp8(const void* q, const int32_t* cu_q_lens, const int32_t* ctx_lens,
                           const int32_t* block_tables, int max_blocks_per_seq, int n_reqs, int n_tokens, int max_q_len,
                           int max_kv_len, const void* k_cache, const void* v_cache, const void* k_exps,
                           const void* v_exps, int num_blocks, void* out, float scale, int n_q_heads, int n_kv_heads,
                           int head_dim, int block_size, int window, void* workspace, size_t workspace_bytes,
                           void* stream) {
  return guarded([&]() -> int {
    return step_fp8(nullptr, q, cu_q_lens, ctx_lens, block_tables, max_blocks_per_seq, n_reqs, n_tokens, max_q_len,
                    max_kv_len, k_cache, v_cache, k_exps, v_exps, num_blocks, out, scale, n_q_heads, n_kv_heads,
                    head_dim, block_size, window, workspace, workspace_bytes, stream);
  });
}

int cb_kv_append_paged_attention_fp8(const void* k_new, const void* v_new, const int64_t* slot_mapping, const void* q,
                                     const int32_t* cu_q_lens, const int32_t* ctx_lens, const int32_t* block_tables,
                                     int max_blocks_per_seq, int n_reqs, int n_tokens, int max_q_len, int max_kv_len,
                                     void* k_cache, void* v_cache, void* k_exps, void* v_exps, int num_blocks, void* out,
                                     float scale, int n_q_heads, int n_kv_heads, int head_dim, int block_size,
                                     int window, void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    const NewRows app{k_new, v_new, slot_mapping};
    return step_fp8(&app, q, cu_q_lens, ctx_lens, block_tables, max_blocks_per_seq, n_reqs, n_tokens, max_q_len,
                    max_kv_len, k_cache, v_cache, k_exps, v_exps, num_blocks, out, scale, n_q_heads, n_kv_heads,
                    head_dim, block_size, window, workspace, workspace_bytes, stream);
  });
}

}  // extern "C"
