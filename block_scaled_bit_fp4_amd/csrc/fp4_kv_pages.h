// fp4_kv_pages.h -- internal interface of the page moves of a 4-bit cache.
// Arguments here are already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

// All layers of a cache: arrays [layers][pages][heads][page][row bytes].
struct KvPool {
  uint8_t* k_codes;
  uint8_t* k_scales;
  uint8_t* v_codes;
  uint8_t* v_scales;
  int64_t pages;
  int layers, heads, page_log2;
  int code_row, scale_row;  // bytes of one token and head
};

struct KvTables {
  int32_t* table;  // [sequences][table_ld >= columns]
  int64_t table_ld, sequences;
  int columns;
  int32_t* lens;
  int32_t* refs;
};

hipError_t fp4_launch_kv_copy(const KvPool& pool, const int32_t* src, const int32_t* dst,
                              const int32_t* tokens, int n, hipStream_t s);
// ws: 4 * n words
hipError_t fp4_launch_kv_fork(const KvPool& pool, const KvTables& t, const int32_t* parents,
                              const int32_t* children, int n, int32_t* failed, int32_t* ws,
                              hipStream_t s);
hipError_t fp4_launch_kv_free(const KvTables& t, int64_t pages, int page_log2, const int32_t* seqs,
                              int n, int window, int sinks, hipStream_t s);
// ws: 3 + pages words
hipError_t fp4_launch_kv_compact(const KvPool& pool, const KvTables& t, int32_t* place,
                                 int32_t* used, int32_t* ws, hipStream_t s);
