// Host-side checks of arguments that the entry points of loopq_kv.h and
// loopq_block.h share.  Not part of the public C ABI.
#pragma once

#include "../../include/loopq_kv.h"
#include "kv_internal.h"

namespace loopq {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

inline int32_t hip_status(hipError_t e) { return e == hipSuccess ? LOOPQ_OK : LOOPQ_ERR_HIP; }

inline bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bn && y < x + an;
}

inline int32_t check_workspace(const void* ws, size_t have, size_t need) {
  if (!ws || have < need) return LOOPQ_ERR_WORKSPACE;
  return aligned(ws, 256) ? LOOPQ_OK : LOOPQ_ERR_ALIGNMENT;
}

inline int item_bytes(int dtype) { return dtype == LOOPQ_F32 ? 4 : 2; }

// rows of `width` elements `ld` apart, 16-byte aligned each
inline int32_t check_rows(const void* p, int64_t ld, int64_t width, int64_t rows, int dtype) {
  if (!p) return LOOPQ_ERR_INVALID_ARG;
  if (rows > 1 && ld < width) return LOOPQ_ERR_INVALID_ARG;
  if (!aligned(p, 16) || (rows > 1 && (ld * item_bytes(dtype)) % 16)) return LOOPQ_ERR_ALIGNMENT;
  return LOOPQ_OK;
}

// whether two matrices of `rows` rows (lda, ldb bytes apart, of wa and wb bytes)
// share a byte; columns of the same wider rows do not
inline bool rows_overlap(const void* a, int64_t lda, int64_t wa, const void* b, int64_t ldb, int64_t wb, int64_t rows) {
  if (!overlap(a, (rows - 1) * lda + wa, b, (rows - 1) * ldb + wb)) return false;
  if (rows == 1 || lda != ldb) return true;
  const int64_t far = (int64_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a)) % lda;
  const int64_t at = far < 0 ? far + lda : far;  // where a row of b starts, from that of a before it
  return at < wa || at > lda - wb;
}

// a pool's and a table's shapes, pointers and alignment (kv_api.hip)
int32_t check_pool(const loopq_kv_pool* p);
int32_t check_table(const loopq_kv_table* t);
KvTable table_of(const loopq_kv_table* t);

}  // namespace loopq
