// Shared by the translation units of the paged key-value cache and the
// attention over it.  Not part of the public C ABI (include/loopq_kv.h).
#pragma once

#include "../../include/loopq_kv.h"
#include "loopq_internal.h"

namespace loopq {

constexpr int kKvMaxRows = 8192;       // fork keeps two ints per row in LDS
constexpr int kKvMaxPages = 1 << 22;   // 65536 64-bit words of used pages

// Scratch of reserve, fork and compact, carved from the caller's workspace.
struct KvScratch {
  uint64_t* bits;    // one bit per page, 64 pages a word
  uint32_t* prefix;  // set bits before each word
  int32_t* list;     // free pages by rank
  int32_t* row_a;    // per row
  int32_t* row_b;
  int32_t* src;      // pages to copy
  int32_t* dst;
  int32_t* head;     // {moves, failed, used pages}
};
size_t kv_scratch_bytes(int64_t rows, int64_t pages);
KvScratch kv_carve(void* ws, int64_t rows, int64_t pages);

struct KvTable {
  int32_t* table;
  int32_t* lens;
  int32_t* refs;
  int rows, width, pages;
};

hipError_t launch_kv_reserve(KvTable in, KvTable out, int page_size, const int32_t* grow, int32_t* info, KvScratch w,
                             hipStream_t s);
hipError_t launch_kv_fork(KvTable in, KvTable out, int page_size, void* pool, int64_t page_bytes, const int32_t* parent,
                          int32_t* info, KvScratch w, hipStream_t s);
hipError_t launch_kv_trim(KvTable in, KvTable out, int page_size, int window, int sinks, hipStream_t s);
hipError_t launch_kv_compact(KvTable in, KvTable out, void* pool, int64_t page_bytes, int32_t* page_map, int32_t* info,
                             KvScratch w, hipStream_t s);
hipError_t launch_kv_copy(const void* src_pool, int src_pages, const int32_t* src, void* dst_pool, int dst_pages,
                          const int32_t* dst, int count, int64_t page_bytes, hipStream_t s);

struct KvWriteArgs {
  uint16_t* pool;  // at the slab's keys of page 0
  int64_t page_stride;  // elements from a page to the next
  int64_t plane;        // elements from the slab's keys to its values
  KvTable t;
  const int32_t* cu;
  const void* k;
  const void* v;
  int64_t ldk, ldv;
  int bf16, tokens, heads, page_size, head_dim;
};
hipError_t launch_kv_write(const KvWriteArgs& a, hipStream_t s);

// One attention call.  Query t of row b sits at position p; key j is visible
// iff 0 <= j <= p, its page exists and window == 0 || p - j < window || j < sinks.
struct AttnArgs {
  const uint16_t* pool;  // bf16, at the slab's keys of page 0
  int64_t page_stride;   // elements from a page to the next
  int64_t plane;         // elements from keys to values
  int num_pages, page_shift;  // page_size = 1 << page_shift
  const int32_t* table;  // [rows][width]
  const int32_t* lens;   // [rows]
  int rows, width;
  const int32_t* cu;     // [rows + 1], or null: one query per row, its last token
  int queries;
  const void* q;
  void* out;
  int64_t ldq, ldo;
  int bf16;
  int heads, group;      // heads_q = heads * group
  int head_dim;
  float scale;
  int window, sinks;
  float* ws;
};
size_t attn_workspace_bytes(int64_t queries, int heads_q, int64_t rows, int head_dim);
hipError_t launch_attn(const AttnArgs& a, hipStream_t s);

}  // namespace loopq
