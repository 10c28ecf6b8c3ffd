// Writing tokens into the paged caches and reading sequences back out of them
// (cache_io.cu).
#pragma once

#include <cuda_runtime.h>

#include "../../include/paged_kv.h"

namespace pkv {

struct CacheWriteParams {
  const void *key, *value;  // [num_tokens, num_kv_heads, head_size], elements of a head adjacent
  int64_t k_s0, k_s1, v_s0, v_s1;
  void *key_cache, *value_cache;
  int64_t kc_s0, kc_s1, vc_s0, vc_s1;
  const int64_t *slots;
  int64_t slot_stride, num_slots;
  int32_t *err;
  int32_t num_tokens, num_kv_heads, head_size, block_size;
  float k_scale, v_scale;
};

struct CacheReadParams {
  void *key, *value;  // [num_tokens, num_kv_heads, head_size], elements of a head adjacent
  int64_t k_s0, k_s1, v_s0, v_s1;
  const void *key_cache, *value_cache;
  int64_t kc_s0, kc_s1, vc_s0, vc_s1;
  const int32_t *bt;
  int64_t bt_s0, bt_s1;
  const int32_t *indptr, *cu, *starts;  // indptr, starts: optional
  int32_t *err;
  int32_t num_seqs, num_tokens, num_kv_heads, head_size, block_size, num_blocks;
  int32_t max_blocks_per_seq;
  float k_scale, v_scale;
};

// `vec`: every token row (of key and value) starts on a 16-byte boundary.
pkv_status_t launch_cache_write(const CacheWriteParams &p, pkv_dtype_t dtype, int32_t kv, bool vec,
                                cudaStream_t stream);
pkv_status_t launch_cache_read(const CacheReadParams &p, pkv_dtype_t dtype, int32_t kv, bool vec,
                               cudaStream_t stream);

}  // namespace pkv
