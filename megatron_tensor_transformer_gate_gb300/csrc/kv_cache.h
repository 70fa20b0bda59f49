// kv_cache.h — host launchers of the key-value cache and its attention (see
// tp_kv_cache in tp.h); arguments are checked by api.cu.  All return a
// cudaError_t value.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/tp.h"

namespace tp {

// Rows of K and V, [rows, n_kv, d], with a row a token.
struct KvRows {
  int64_t rows;
  void *k, *v;
  int64_t k_row, k_head, v_row, v_head;
  const int32_t* start;
};

// kv_cache.cu
int kv_cache_write(const tp_kv_cache& c, int dtype, const KvRows& r,
                   unsigned* status, void* stream);
int kv_cache_read(const tp_kv_cache& c, int dtype, const KvRows& r,
                  unsigned* status, void* stream);

// attn_decode.cu
struct DecodeArgs {
  int64_t rows;
  int n_q;
  float scale;
  const void* q;
  int64_t q_row, q_head;
  void* out;
  int64_t o_row, o_head;
  float* lse;
  void* ws;
  int bf16 = 0;   // q and out, else fp16 (set by attn_decode)
};
size_t attn_decode_ws_bytes(const tp_kv_cache& c, int64_t rows, int n_q);
int attn_decode(const tp_kv_cache& c, int dtype, const DecodeArgs& a,
                unsigned* status, void* stream);

}  // namespace tp
