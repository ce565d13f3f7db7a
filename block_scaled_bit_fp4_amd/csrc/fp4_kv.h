// fp4_kv.h -- what the kernels of the 4-bit KV cache share: the cache and
// batch as the kernels see them (already validated), and where a token of a
// sequence lies.
//
// One layer of the cache is four arrays: codes [pages][heads][page][D / 2]
// and scale bytes [pages][heads][page][D / B], for K and for V.  So one
// page of one head is contiguous (page * D / 2 code bytes), a token's row
// is D / 2 bytes, and sixteen consecutive tokens (a page holds a multiple
// of sixteen) are 8 * D contiguous bytes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

struct KvCacheArgs {
  uint8_t* k_codes;  // this layer's arrays
  uint8_t* k_scales;
  uint8_t* v_codes;
  uint8_t* v_scales;
  const float* k_scale;  // NVFP4: this layer's factor; null for the MX formats
  const float* v_scale;
  int64_t pages;
  int format, heads, dim, dim_log2;
  int page_log2;
  int rht;
  uint32_t signs;
};

struct KvBatchArgs {
  const int32_t* page_table;
  int64_t table_ld;
  const int32_t* kv_lens;
  const int32_t* cu_q;
  int batch, columns, max_q, max_kv;
  int64_t tokens;  // rows of the tensors that hold the new tokens
};

struct KvAppendLaunch {
  KvCacheArgs cache;
  KvBatchArgs batch;
  const void* k;
  const void* v;
  int64_t k_token, k_head, v_token, v_head;  // strides, elements
  int dtype;                                 // 0 bf16, 1 f32
};

struct KvGatherLaunch {
  KvCacheArgs cache;
  KvBatchArgs batch;
  void* k;
  void* v;
  int64_t token, head;  // strides of both outputs, elements
  int dtype;
};

struct KvAttentionLaunch {
  KvCacheArgs cache;
  KvBatchArgs batch;
  const void* q;
  int64_t q_token, q_head;
  int q_heads;
  float scale;
  int window, sinks;
  void* out;
  int out_dtype;
  int64_t out_token, out_head;
  float* lse;  // [tokens][q_heads] or null
  void* workspace;
};

// How an attention call is split: rows of a workgroup (new tokens of one
// sequence times the query heads of one key head), and pieces of the keys.
struct KvAttentionPlan {
  bool prompt;    // the kernel for many rows
  int rows;       // rows of a workgroup
  int row_tiles;  // of the longest sequence
  int splits;      // many rows: pieces of the keys
  int pieces;      // few rows: of every row tile's keys; 0: equal runs of all keys
  int64_t groups;  // workgroups
  size_t bytes;    // workspace
};

KvAttentionPlan fp4_plan_kv_attention(const KvCacheArgs& c, const KvBatchArgs& b, int q_heads,
                                      int window, int sinks);
hipError_t fp4_launch_kv_append(const KvAppendLaunch& q, hipStream_t s);
hipError_t fp4_launch_kv_gather(const KvGatherLaunch& q, hipStream_t s);
hipError_t fp4_launch_kv_attention(const KvAttentionLaunch& q, hipStream_t s);

#ifdef __HIPCC__
namespace fp4kv {

// One sequence of a batch.
struct KvSeq {
  int64_t first;  // row of its first new token in the caller's tensors
  int64_t pos;    // position of that token; negative if it has more new tokens than tokens
  int n;          // new tokens that this call covers
  int kv;         // tokens in the cache
};

// A length past the table's columns is cut, so that no entry past the row
// is read; new tokens past the caller's tensors, or past max_q (which the
// grid covers), are left out.
__device__ __forceinline__ KvSeq kv_seq(const KvBatchArgs& b, int seq, int page_log2) {
  KvSeq s;
  const int64_t cap = (int64_t)b.columns << page_log2;
  const int len = b.kv_lens[seq];
  s.kv = len < 0 ? 0 : (len > cap ? (int)cap : len);
  s.first = b.cu_q[seq];
  int64_t n = (int64_t)b.cu_q[seq + 1] - s.first;
  s.pos = (int64_t)len - n;
  if (s.first < 0) n = 0;
  if (n > b.tokens - s.first) n = b.tokens - s.first;
  if (n > b.max_q) n = b.max_q;
  s.n = n < 0 ? 0 : (int)n;
  return s;
}

}  // namespace fp4kv
#endif
