// C ABI of the paged key-value cache and the attention over it (declared in
// include/loopq_kv.h): host-side checks and dispatch on the caller's stream.
#include <math.h>

#include "arg_checks.h"

using namespace loopq;

namespace {

int32_t check_page_size(int n) {
  if (n <= 0) return LOOPQ_ERR_INVALID_ARG;
  return n < 8 || n > 256 || (n & (n - 1)) ? LOOPQ_ERR_UNSUPPORTED : LOOPQ_OK;
}

int32_t check_pages(int pages) {
  if (pages <= 0) return LOOPQ_ERR_INVALID_ARG;
  return pages > kKvMaxPages ? LOOPQ_ERR_UNSUPPORTED : LOOPQ_OK;
}

int32_t check_shape(int pages, int slabs, int heads, int page_size, int head_dim) {
  if (slabs <= 0 || heads <= 0 || head_dim <= 0) return LOOPQ_ERR_INVALID_ARG;
  int32_t st = check_pages(pages);
  if (st == LOOPQ_OK) st = check_page_size(page_size);
  if (st != LOOPQ_OK) return st;
  if (head_dim != 64 && head_dim != 96 && head_dim != 128) return LOOPQ_ERR_UNSUPPORTED;
  if ((int64_t)heads * head_dim > (1 << 20) || slabs > (1 << 16)) return LOOPQ_ERR_UNSUPPORTED;
  // a page's bytes are a 32-bit factor in the kernels' addresses
  if ((int64_t)slabs * 4 * heads * page_size * head_dim >= ((int64_t)1 << 31)) return LOOPQ_ERR_UNSUPPORTED;
  return LOOPQ_OK;
}

int64_t page_bytes(const loopq_kv_pool* p) {
  return (int64_t)p->slabs * 2 * p->heads * p->page_size * p->head_dim * 2;
}

}  // namespace

namespace loopq {

int32_t check_pool(const loopq_kv_pool* p) {
  if (!p) return LOOPQ_ERR_INVALID_ARG;
  int32_t st = check_shape(p->num_pages, p->slabs, p->heads, p->page_size, p->head_dim);
  if (st != LOOPQ_OK) return st;
  if (!p->data) return LOOPQ_ERR_INVALID_ARG;
  return aligned(p->data, 16) ? LOOPQ_OK : LOOPQ_ERR_ALIGNMENT;
}

int32_t check_table(const loopq_kv_table* t) {
  if (!t || t->rows < 0 || t->max_pages <= 0) return LOOPQ_ERR_INVALID_ARG;
  int32_t st = check_pages(t->num_pages);
  if (st != LOOPQ_OK) return st;
  if (t->rows > kKvMaxRows || (int64_t)t->rows * t->max_pages >= ((int64_t)1 << 31)) return LOOPQ_ERR_UNSUPPORTED;
  // positions are 32-bit: max_pages * page_size stays below 2^31 for every page size
  if (t->max_pages > (1 << 22)) return LOOPQ_ERR_UNSUPPORTED;
  if (t->rows > 0 && (!t->table || !t->lens)) return LOOPQ_ERR_INVALID_ARG;
  if (!t->refs) return LOOPQ_ERR_INVALID_ARG;
  if (!aligned(t->table, 4) || !aligned(t->lens, 4) || !aligned(t->refs, 4)) return LOOPQ_ERR_ALIGNMENT;
  return LOOPQ_OK;
}

KvTable table_of(const loopq_kv_table* t) {
  return KvTable{t->table, t->lens, t->refs, t->rows, t->max_pages, t->num_pages};
}

}  // namespace loopq

namespace {

// in and out of one call: the same three buffers, or nothing shared
int32_t check_pair(const loopq_kv_table* a, const loopq_kv_table* b, bool may_be_same) {
  int32_t st = check_table(a);
  if (st == LOOPQ_OK) st = check_table(b);
  if (st != LOOPQ_OK) return st;
  if (a->max_pages != b->max_pages || a->num_pages != b->num_pages) return LOOPQ_ERR_INVALID_ARG;
  if (may_be_same && a->rows != b->rows) return LOOPQ_ERR_INVALID_ARG;
  if (a->table == b->table && a->lens == b->lens && a->refs == b->refs && may_be_same) return LOOPQ_OK;
  const void* pa[3] = {a->table, a->lens, a->refs};
  const void* pb[3] = {b->table, b->lens, b->refs};
  const size_t na[3] = {(size_t)a->rows * a->max_pages * 4, (size_t)a->rows * 4, (size_t)a->num_pages * 4};
  const size_t nb[3] = {(size_t)b->rows * b->max_pages * 4, (size_t)b->rows * 4, (size_t)b->num_pages * 4};
  for (int i = 0; i < 3; ++i)
    for (int j = 0; j < 3; ++j)
      if (na[i] && nb[j] && overlap(pa[i], na[i], pb[j], nb[j])) return LOOPQ_ERR_INVALID_ARG;
  return LOOPQ_OK;
}

int32_t run_attn(const loopq_kv_pool* pool, int32_t slab, const loopq_kv_table* table, const int32_t* cu, const void* q,
                 int64_t ldq, int32_t dtype, int32_t queries, int32_t heads_q, float scale, int32_t window,
                 int32_t sinks, void* out, int64_t ldo, void* workspace, size_t workspace_bytes, void* stream) {
  int32_t st = check_pool(pool);
  if (st == LOOPQ_OK) st = check_table(table);
  if (st != LOOPQ_OK) return st;
  if (dtype != LOOPQ_F32 && dtype != LOOPQ_BF16) return LOOPQ_ERR_UNSUPPORTED;
  if (slab < 0 || slab >= pool->slabs || table->num_pages != pool->num_pages) return LOOPQ_ERR_INVALID_ARG;
  if (queries < 0 || heads_q <= 0 || window < 0 || sinks < 0 || !isfinite(scale)) return LOOPQ_ERR_INVALID_ARG;
  if (heads_q % pool->heads || (int64_t)heads_q * pool->head_dim > (1 << 20)) return LOOPQ_ERR_UNSUPPORTED;
  if (queries == 0 || table->rows == 0) return LOOPQ_OK;
  // query tiles of every head are counted in 32 bits
  if ((int64_t)queries * heads_q / 128 + (int64_t)table->rows * heads_q > (1 << 30)) return LOOPQ_ERR_UNSUPPORTED;
  const int64_t width = (int64_t)heads_q * pool->head_dim;
  st = check_rows(q, ldq, width, queries, dtype);
  if (st == LOOPQ_OK) st = check_rows(out, ldo, width, queries, dtype);
  if (st != LOOPQ_OK) return st;
  const int item = item_bytes(dtype);
  if (rows_overlap(q, ldq * item, width * item, out, ldo * item, width * item, queries)) return LOOPQ_ERR_INVALID_ARG;
  st = check_workspace(workspace, workspace_bytes, attn_workspace_bytes(queries, heads_q, table->rows, pool->head_dim));
  if (st != LOOPQ_OK) return st;
  AttnArgs a;
  a.plane = (int64_t)pool->heads * pool->page_size * pool->head_dim;
  a.page_stride = pool->slabs * 2 * a.plane;
  a.pool = reinterpret_cast<const uint16_t*>(pool->data) + slab * 2 * a.plane;
  a.num_pages = pool->num_pages;
  a.page_shift = 31 - __builtin_clz((unsigned)pool->page_size);
  a.table = table->table;
  a.lens = table->lens;
  a.rows = table->rows;
  a.width = table->max_pages;
  a.cu = cu;
  a.queries = queries;
  a.q = q;
  a.out = out;
  a.ldq = queries > 1 ? ldq : width;
  a.ldo = queries > 1 ? ldo : width;
  a.bf16 = dtype == LOOPQ_BF16;
  a.heads = pool->heads;
  a.group = heads_q / pool->heads;
  a.head_dim = pool->head_dim;
  a.scale = scale;
  a.window = window;
  a.sinks = sinks;
  a.ws = reinterpret_cast<float*>(workspace);
  hipStream_t s = as_stream(stream);
  TimingScope ts(LOOPQ_KERNEL_ATTN, s);
  return hip_status(launch_attn(a, s));
}

}  // namespace

extern "C" {

int32_t loopq_kv_pool_bytes(int32_t num_pages, int32_t slabs, int32_t heads, int32_t page_size, int32_t head_dim,
                            size_t* bytes) {
  if (!bytes) return LOOPQ_ERR_INVALID_ARG;
  const int32_t st = check_shape(num_pages, slabs, heads, page_size, head_dim);
  if (st != LOOPQ_OK) return st;
  *bytes = (size_t)num_pages * slabs * 2 * heads * page_size * head_dim * 2;
  return LOOPQ_OK;
}

int32_t loopq_kv_workspace_bytes(int32_t rows, int32_t num_pages, size_t* bytes) {
  if (!bytes || rows < 0) return LOOPQ_ERR_INVALID_ARG;
  const int32_t st = check_pages(num_pages);
  if (st != LOOPQ_OK) return st;
  if (rows > kKvMaxRows) return LOOPQ_ERR_UNSUPPORTED;
  *bytes = kv_scratch_bytes(rows, num_pages);
  return LOOPQ_OK;
}

int32_t loopq_kv_reserve(const loopq_kv_table* in, int32_t page_size, const int32_t* grow, const loopq_kv_table* out,
                         int32_t* info, void* workspace, size_t workspace_bytes, void* stream) {
  int32_t st = check_pair(in, out, true);
  if (st == LOOPQ_OK) st = check_page_size(page_size);
  if (st != LOOPQ_OK) return st;
  if (in->rows == 0) return LOOPQ_OK;
  if (!grow || !info) return LOOPQ_ERR_INVALID_ARG;
  if (!aligned(grow, 4) || !aligned(info, 4)) return LOOPQ_ERR_ALIGNMENT;
  st = check_workspace(workspace, workspace_bytes, kv_scratch_bytes(in->rows, in->num_pages));
  if (st != LOOPQ_OK) return st;
  hipStream_t s = as_stream(stream);
  TimingScope ts(LOOPQ_KERNEL_KV, s);
  return hip_status(launch_kv_reserve(table_of(in), table_of(out), page_size, grow, info,
                                      kv_carve(workspace, in->rows, in->num_pages), s));
}

int32_t loopq_kv_write(const loopq_kv_pool* pool, int32_t slab, const loopq_kv_table* table, const int32_t* cu,
                       const void* k, int64_t ldk, const void* v, int64_t ldv, int32_t dtype, int32_t tokens,
                       void* stream) {
  int32_t st = check_pool(pool);
  if (st == LOOPQ_OK) st = check_table(table);
  if (st != LOOPQ_OK) return st;
  if (dtype != LOOPQ_F32 && dtype != LOOPQ_BF16) return LOOPQ_ERR_UNSUPPORTED;
  if (slab < 0 || slab >= pool->slabs || tokens < 0 || table->num_pages != pool->num_pages)
    return LOOPQ_ERR_INVALID_ARG;
  if (tokens == 0 || table->rows == 0) return LOOPQ_OK;
  if (!cu) return LOOPQ_ERR_INVALID_ARG;
  if (!aligned(cu, 4)) return LOOPQ_ERR_ALIGNMENT;
  const int64_t width = (int64_t)pool->heads * pool->head_dim;
  st = check_rows(k, ldk, width, tokens, dtype);
  if (st == LOOPQ_OK) st = check_rows(v, ldv, width, tokens, dtype);
  if (st != LOOPQ_OK) return st;
  // a launch has fewer than 2^32 work-items: eight elements each, in work-groups of 256
  if (tokens * (width / 8) > ((int64_t)1 << 32) - 256) return LOOPQ_ERR_UNSUPPORTED;
  KvWriteArgs a;
  a.plane = (int64_t)pool->heads * pool->page_size * pool->head_dim;
  a.page_stride = pool->slabs * 2 * a.plane;
  a.pool = reinterpret_cast<uint16_t*>(pool->data) + slab * 2 * a.plane;
  a.t = table_of(table);
  a.cu = cu;
  a.k = k;
  a.v = v;
  a.ldk = tokens > 1 ? ldk : width;
  a.ldv = tokens > 1 ? ldv : width;
  a.bf16 = dtype == LOOPQ_BF16;
  a.tokens = tokens;
  a.heads = pool->heads;
  a.page_size = pool->page_size;
  a.head_dim = pool->head_dim;
  hipStream_t s = as_stream(stream);
  TimingScope ts(LOOPQ_KERNEL_KV, s);
  return hip_status(launch_kv_write(a, s));
}

int32_t loopq_kv_fork(const loopq_kv_pool* pool, const loopq_kv_table* in, const int32_t* parent,
                      const loopq_kv_table* out, int32_t* info, void* workspace, size_t workspace_bytes,
                      void* stream) {
  int32_t st = check_pool(pool);
  if (st == LOOPQ_OK) st = check_pair(in, out, false);
  if (st != LOOPQ_OK) return st;
  if (in->num_pages != pool->num_pages) return LOOPQ_ERR_INVALID_ARG;
  if (!info || (out->rows > 0 && !parent)) return LOOPQ_ERR_INVALID_ARG;
  if (!aligned(parent, 4) || !aligned(info, 4)) return LOOPQ_ERR_ALIGNMENT;
  const int rows = in->rows > out->rows ? in->rows : out->rows;
  st = check_workspace(workspace, workspace_bytes, kv_scratch_bytes(rows, in->num_pages));
  if (st != LOOPQ_OK) return st;
  hipStream_t s = as_stream(stream);
  TimingScope ts(LOOPQ_KERNEL_KV, s);
  return hip_status(launch_kv_fork(table_of(in), table_of(out), pool->page_size, pool->data, page_bytes(pool), parent,
                                   info, kv_carve(workspace, rows, in->num_pages), s));
}

int32_t loopq_kv_trim(const loopq_kv_table* in, int32_t page_size, int32_t window, int32_t sinks,
                      const loopq_kv_table* out, void* stream) {
  int32_t st = check_pair(in, out, true);
  if (st == LOOPQ_OK) st = check_page_size(page_size);
  if (st != LOOPQ_OK) return st;
  if (window < 1 || sinks < 0) return LOOPQ_ERR_INVALID_ARG;
  if (in->rows == 0) return LOOPQ_OK;
  hipStream_t s = as_stream(stream);
  TimingScope ts(LOOPQ_KERNEL_KV, s);
  return hip_status(launch_kv_trim(table_of(in), table_of(out), page_size, window, sinks, s));
}

int32_t loopq_kv_compact(const loopq_kv_pool* pool, const loopq_kv_table* in, const loopq_kv_table* out,
                         int32_t* page_map, int32_t* info, void* workspace, size_t workspace_bytes, void* stream) {
  int32_t st = check_pool(pool);
  if (st == LOOPQ_OK) st = check_pair(in, out, true);
  if (st != LOOPQ_OK) return st;
  if (in->num_pages != pool->num_pages || !page_map || !info) return LOOPQ_ERR_INVALID_ARG;
  if (!aligned(page_map, 4) || !aligned(info, 4)) return LOOPQ_ERR_ALIGNMENT;
  st = check_workspace(workspace, workspace_bytes, kv_scratch_bytes(in->rows, in->num_pages));
  if (st != LOOPQ_OK) return st;
  hipStream_t s = as_stream(stream);
  TimingScope ts(LOOPQ_KERNEL_KV, s);
  return hip_status(launch_kv_compact(table_of(in), table_of(out), pool->data, page_bytes(pool), page_map, info,
                                      kv_carve(workspace, in->rows, in->num_pages), s));
}

int32_t loopq_kv_copy_pages(const loopq_kv_pool* src_pool, const int32_t* src, const loopq_kv_pool* dst_pool,
                            const int32_t* dst, int32_t count, void* stream) {
  int32_t st = check_pool(src_pool);
  if (st == LOOPQ_OK) st = check_pool(dst_pool);
  if (st != LOOPQ_OK) return st;
  if (src_pool->slabs != dst_pool->slabs || src_pool->heads != dst_pool->heads ||
      src_pool->page_size != dst_pool->page_size || src_pool->head_dim != dst_pool->head_dim || count < 0)
    return LOOPQ_ERR_INVALID_ARG;
  if (count == 0) return LOOPQ_OK;
  if (!src || !dst) return LOOPQ_ERR_INVALID_ARG;
  if (!aligned(src, 4) || !aligned(dst, 4)) return LOOPQ_ERR_ALIGNMENT;
  hipStream_t s = as_stream(stream);
  TimingScope ts(LOOPQ_KERNEL_KV, s);
  return hip_status(launch_kv_copy(src_pool->data, src_pool->num_pages, src, dst_pool->data, dst_pool->num_pages, dst,
                                   count, page_bytes(src_pool), s));
}

int32_t loopq_attn_workspace_bytes(int32_t queries, int32_t heads_q, int32_t rows, int32_t head_dim, size_t* bytes) {
  if (!bytes || queries < 0 || heads_q <= 0 || rows < 0) return LOOPQ_ERR_INVALID_ARG;
  if ((head_dim != 64 && head_dim != 96 && head_dim != 128) || rows > kKvMaxRows) return LOOPQ_ERR_UNSUPPORTED;
  *bytes = attn_workspace_bytes(queries, heads_q, rows, head_dim);
  return LOOPQ_OK;
}

int32_t loopq_attn_decode(const loopq_kv_pool* pool, int32_t slab, const loopq_kv_table* table, const void* q,
                          int64_t ldq, int32_t dtype, int32_t heads_q, float scale, int32_t window, int32_t sinks,
                          void* out, int64_t ldo, void* workspace, size_t workspace_bytes, void* stream) {
  return run_attn(pool, slab, table, nullptr, q, ldq, dtype, table ? table->rows : 0, heads_q, scale, window, sinks, out,
                  ldo, workspace, workspace_bytes, stream);
}

int32_t loopq_attn_prefill(const loopq_kv_pool* pool, int32_t slab, const loopq_kv_table* table, const int32_t* cu,
                           const void* q, int64_t ldq, int32_t dtype, int32_t queries, int32_t heads_q, float scale,
                           int32_t window, int32_t sinks, void* out, int64_t ldo, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (!cu && queries > 0 && table && table->rows > 0) return LOOPQ_ERR_INVALID_ARG;
  if (!aligned(cu, 4)) return LOOPQ_ERR_ALIGNMENT;
  return run_attn(pool, slab, table, cu, q, ldq, dtype, queries, heads_q, scale, window, sinks, out, ldo, workspace,
                  workspace_bytes, stream);
}

}  // extern "C"
