// Attention over the paged key-value cache (include/loopq_kv.h): one new token
// a row (decode), or several (prefill), with a sliding window and sinks.
//
// For a query q with the visible keys J:  s_j = scale q . k_j,
// out = sum_J 2^(t_j - m) v_j / sum_J 2^(t_j - m),  t_j = s_j log2(e), m a running
// reference at or near the maximum, all sums in fp32 (one pass over the keys;
// m, l and the sums are rescaled when the reference grows).
//
// Both products run on the bf16 MFMA, transposed: S^T = K Q^T puts a query in a
// column, so its keys lie in the registers of two (four) lanes and the softmax
// needs one (two) lane exchanges; P^T then is the second product's B operand as
// it stands, O^T = V^T P^T, since the order of the summed keys is free as long
// as both operands keep the same: slot e of lane group h holds key
// 4h + e % 4 + 8 (e / 4) of its 16 (prefill), or 4h + e % 4 + 16 (e / 4) of its
// 32 (decode).  V^T comes from the row-major tile in LDS by transposing reads.
// fp32 queries and weights are split into three bf16 planes (24 bits), whose
// products with the bf16 keys and values are exact; bf16 queries are exact
// alone.
//
// fp32 queries and weights are cut, not rounded, into their planes, and no plane of
// a weight is 0 unless the weight is, so that an infinite key or value meets every
// plane as in the formula.  bf16 queries: weights go to the product as one bf16
// plane (rounded by up to 2^-8 of themselves, and l sums the rounded weights, so that
// what rounding does to all alike cancels), as two where few keys share the sum
// and in decode, where the product costs nothing beside the bytes.
//
// Work is cut by length, not by row: the visible key tiles of all (row, key
// head, query tile) items form one line, shared out evenly.  Decode cuts it into
// equal pieces, one per wave; prefill keeps items whole as tasks that work-groups
// take in turn, and splits those longer than a work-group's even share.  Lengths
// are read on the device, so ragged rows balance and the launch shape never
// depends on them.  An item that lies in one piece is finished there; the others
// leave (m, l, O) per piece, and a last launch joins them in the order of the keys:
// the result depends on the inputs alone.
#include "attn_core.h"

namespace loopq {

namespace {

struct AttnSizes {
  size_t part, ml, records, row, tasks;
  size_t all() const { return part + ml + records + row + tasks + 512; }
};
size_t up256(int64_t b) { return (size_t)((b + 255) / 256 * 256); }
AttnSizes attn_sizes(int64_t queries, int heads_q, int64_t rows, int D) {
  const int64_t n = max((int64_t)kDecodePieces * 2 * kDecodeRows, (int64_t)kPrefillSlots * kPrefillRows);
  AttnSizes s;
  s.part = up256(n * D * 4);
  s.ml = up256(n * 2 * 4);
  s.records = up256(max(kDecodePieces, kPrefillSlots) * sizeof(JoinRecord));
  s.row = up256((rows + 1) * 4);
  // query tiles have 128 rows at least, and are split into 256 parts more at most
  s.tasks = up256((queries * heads_q / 128 + rows + kPrefillGroups) * sizeof(PrefillTask));
  return s;
}

}  // namespace

size_t attn_workspace_bytes(int64_t queries, int heads_q, int64_t rows, int head_dim) {
  return attn_sizes(queries, heads_q, rows, head_dim).all();
}

hipError_t launch_attn(const AttnArgs& a, hipStream_t s) {
  const AttnSizes z = attn_sizes(a.queries, a.heads * a.group, a.rows, a.head_dim);
  char* p = reinterpret_cast<char*>(a.ws);
  AttnPlan pl;
  pl.part = reinterpret_cast<float*>(p);
  pl.ml = reinterpret_cast<float*>(p += z.part);
  pl.records = reinterpret_cast<JoinRecord*>(p += z.ml);
  pl.row_tiles = reinterpret_cast<int32_t*>(p += z.records);
  pl.tasks = reinterpret_cast<PrefillTask*>(p += z.row);
  pl.most_tiles = (int32_t)(z.tasks / sizeof(PrefillTask)) - kPrefillGroups;
  pl.zeros = reinterpret_cast<uint16_t*>(p += z.tasks);
  pl.head = reinterpret_cast<int32_t*>(p += 256);
  pl.next = reinterpret_cast<int32_t*>(p + 64);
  // t = s c with c > 0, so that the largest score has the largest t
  const float log2e = 1.4426950408889634f;
  pl.qmul = a.scale > 0.0f ? 1.0f : a.scale < 0.0f ? -1.0f : 0.0f;
  pl.c = a.scale != 0.0f ? fabsf(a.scale) * log2e : 1.0f;
  return a.cu ? launch_attn_prefill(a, pl, s) : launch_attn_decode(a, pl, s);
}

}  // namespace loopq
