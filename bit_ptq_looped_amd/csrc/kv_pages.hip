// Pages of the key-value cache: reserving, writing, forking, freeing,
// compacting and copying (include/loopq_kv.h has the definitions).
//
// The bookkeeping is whole-number work over the reference counts and the page
// table.  Free pages are found from the counts themselves (no free list to keep
// consistent): a bit per page, the words' prefix sums, and the k-th free page
// is a search in them, so "lowest index first" holds whatever the timing.
// Contents move page by page; a page is one contiguous run for all slabs, and
// sources and targets of one call are disjoint, so copies need no order.
#include "kv_internal.h"
#include "quant_core.h"

namespace loopq {

namespace {

constexpr int kScan = 1024;  // threads of the one-work-group kernels
// Tables and counts of up to this many entries are handled by one work-group,
// which saves a launch (about 3 us of host and 2 us of device time each).
constexpr int kOneGroup = 16384;
// Work-groups of a copy of pages, at most: 2048 leave the memory's queues short
// (evict of 0.8 GB 354 us, with 16384 331 us).
constexpr int kCopyGroups = 16384;

__device__ __forceinline__ int clamped_len(const KvTable& t, int row, int shift) {
  const int64_t cap = (int64_t)t.width << shift;
  const int64_t n = t.lens[row];
  return (int)(n < 0 ? 0 : n > cap ? cap : n);
}

// exclusive sum of v over the work-group's 1024 threads; total to every thread
__device__ __forceinline__ int block_exclusive(int v, int* total) {
  __shared__ int part[kScan / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int y = __shfl_up(x, off, 64);
    if (lane >= off) x += y;
  }
  __syncthreads();  // part is free again
  if (lane == 63) part[wave] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kScan / 64; ++w) {
    const int p = part[w];
    before += w < wave ? p : 0;
    all += p;
  }
  *total = all;
  return before + x - v;
}

// a bit per page that is free (or used), by all threads of a grid of `step`
__device__ __forceinline__ void page_bits(const int32_t* refs, int pages, uint64_t* bits, bool want_free, int64_t first,
                                          int64_t step) {
  const int64_t n = ((int64_t)pages + 63) / 64 * 64;
  for (int64_t p = first; p < n; p += step) {  // whole waves: first and step are the lane plus multiples of 64
    const bool in = p < pages;
    const bool is_free = in && refs[p] <= 0;
    const uint64_t w = __ballot(in && is_free == want_free);
    if ((p & 63) == 0) bits[p >> 6] = w;
  }
}

// the lowest `total` set bits as a list (the work-group's 1024 threads); returns how many bits are set
__device__ __forceinline__ int list_bits(const uint64_t* bits, int words, int32_t* list, int total) {
  int base = 0;
  for (int w0 = 0; w0 < words; w0 += kScan) {
    const int w = w0 + threadIdx.x;
    uint64_t x = w < words ? bits[w] : 0;
    int all;
    int at = base + block_exclusive(__popcll(x), &all);
    while (x != 0 && at < total) {
      list[at++] = (w << 6) + __ffsll((unsigned long long)x) - 1;
      x &= x - 1;
    }
    base += all;
  }
  return base;
}

// ------------------------------------------------------------------ reserve

__device__ __forceinline__ void reserve_copy(const KvTable& in, const KvTable& out, uint64_t* bits, int64_t first,
                                             int64_t step) {
  page_bits(in.refs, in.pages, bits, true, first, step);
  if (in.table == out.table) return;
  const int64_t n = (int64_t)in.rows * in.width;
  for (int64_t i = first; i < n; i += step) out.table[i] = in.table[i];
  for (int64_t i = first; i < in.pages; i += step) out.refs[i] = in.refs[i];
}

__global__ __launch_bounds__(256) void reserve_copy_kernel(KvTable in, KvTable out, uint64_t* bits) {
  reserve_copy(in, out, bits, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}

// One work-group: pages each row lacks, their prefix, the free pages by rank,
// and the new entries.  FUSED does the copy and the bits itself.
template <bool FUSED>
__global__ __launch_bounds__(kScan) void reserve_kernel(KvTable in, KvTable out, int shift, const int32_t* grow,
                                                        int32_t* info, KvScratch w) {
  __shared__ int s_full, s_before[kKvMaxRows + 1];
  const int tid = threadIdx.x, psz = 1 << shift;
  if (tid == 0) s_full = 0;
  if (FUSED) reserve_copy(in, out, w.bits, tid, kScan);
  __syncthreads();
  int total = 0;
  for (int r0 = 0; r0 < in.rows; r0 += kScan) {
    const int r = r0 + tid;
    int need = 0;
    if (r < in.rows) {
      const int len = clamped_len(in, r, shift);
      const int64_t more = max(grow[r], 0);
      const int64_t want = (len + more + psz - 1) >> shift;
      const int have = (len + psz - 1) >> shift;
      if (want > in.width) s_full = 1;
      else need = (int)want - have;
    }
    int all;
    const int before = block_exclusive(need, &all);
    if (r < in.rows) s_before[r] = total + before;
    total += all;
  }
  if (tid == 0) s_before[in.rows] = total;
  const int words = (in.pages + 63) >> 6;
  const int nfree = list_bits(w.bits, words, w.list, total);
  __syncthreads();
  const int what = s_full ? LOOPQ_KV_ROW_FULL : total > nfree ? LOOPQ_KV_NO_PAGES : LOOPQ_KV_DONE;
  if (tid == 0) {
    info[0] = what;
    info[1] = total;
  }
  for (int r = tid; r < in.rows; r += kScan) {
    const int old = in.lens[r];
    out.lens[r] = what == LOOPQ_KV_DONE ? clamped_len(in, r, shift) + max(grow[r], 0) : old;
  }
  if (what != LOOPQ_KV_DONE) return;
  __syncthreads();
  for (int k = tid; k < total; k += kScan) {
    int lo = 0, hi = in.rows;  // the row with s_before[row] <= k < s_before[row + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_before[mid] <= k) lo = mid;
      else hi = mid;
    }
    // its first missing entry: rows' lengths in `out` have grown by now
    const int want = (out.lens[lo] + psz - 1) >> shift;
    const int at = want - (s_before[lo + 1] - k);
    const int page = w.list[k];
    out.table[(int64_t)lo * out.width + at] = page;
    out.refs[page] = 1;
  }
}

// -------------------------------------------------------------------- write

// Eight elements (16 bytes of the pool) of a token per thread, keys and values;
// bound by the bytes of k, v and the pool: 14340 bf16 tokens of 20 heads of 128, 294 MB
// in 62 us, 4.7 TB/s.
__global__ __launch_bounds__(256) void write_kernel(KvWriteArgs a) {
  const int per_tok = a.heads * a.head_dim / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t t = i / per_tok;
  if (t >= a.tokens) return;
  const int e = (int)(i - t * per_tok) * 8;
  int lo = 0, hi = a.t.rows;
  if (a.cu[hi] <= t || a.cu[0] > t) return;
  while (hi - lo > 1) {  // cu[lo] <= t < cu[lo + 1]
    const int mid = (lo + hi) >> 1;
    if (a.cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int shift = 31 - __clz(a.page_size);
  const int64_t pos = (int64_t)clamped_len(a.t, lo, shift) - a.cu[lo + 1] + t;
  if (pos < 0 || pos >= (int64_t)a.t.width << shift) return;
  const int page = a.t.table[(int64_t)lo * a.t.width + (pos >> shift)];
  if (page < 0 || page >= a.t.pages) return;
  const int head = e / a.head_dim, d = e - head * a.head_dim;
  uint16_t* dst = a.pool + (int64_t)page * a.page_stride +
                  ((int64_t)head * a.page_size + (pos & (a.page_size - 1))) * a.head_dim + d;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const void* x = kv ? a.v : a.k;
    const int64_t at = t * (kv ? a.ldv : a.ldk) + e;
    uint4 o;
    if (a.bf16) {
      o = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(x) + at);
    } else {
      const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(x) + at);
      const float4 f0 = p[0], f1 = p[1];
      o = uint4{bf16x2_rne(f0.x, f0.y), bf16x2_rne(f0.z, f0.w), bf16x2_rne(f1.x, f1.y), bf16x2_rne(f1.z, f1.w)};
    }
    *reinterpret_cast<uint4*>(dst + kv * a.plane) = o;
  }
}

// ------------------------------------------------------------ page contents

constexpr int kChunk = 16384;  // bytes a work-group moves at a time

// 16 KiB (or the page's rest) from src to dst, both 16-byte aligned; every load
// is issued before the first store
__device__ __forceinline__ void copy_chunk(const char* src, char* dst, int64_t at, int64_t bytes) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const u32x4* s = reinterpret_cast<const u32x4*>(src + at);
  u32x4* d = reinterpret_cast<u32x4*>(dst + at);
  const int n = (int)(min((int64_t)kChunk, bytes - at) / 16);
  const int tid = threadIdx.x & 255;
  u32x4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (tid + 256 * i < n) v[i] = s[tid + 256 * i];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (tid + 256 * i < n) d[tid + 256 * i] = v[i];
}

// Bound by the bytes: 2000 pages of 1 MB 829 us, 5.1 TB/s read and written; 64 pages
// of 0.5 MB 12.7 us.
__global__ __launch_bounds__(256) void copy_pages_kernel(const char* src_pool, int src_pages, const int32_t* src,
                                                         char* dst_pool, int dst_pages, const int32_t* dst, int count,
                                                         int64_t page_bytes) {
  const int64_t chunks = (page_bytes + kChunk - 1) / kChunk;
  const int64_t n = chunks * count;
  for (int64_t i = blockIdx.x; i < n; i += gridDim.x) {
    const int m = (int)(i / chunks);
    const int s = src[m], d = dst[m];
    if (s < 0 || s >= src_pages || d < 0 || d >= dst_pages) continue;
    copy_chunk(src_pool + s * page_bytes, dst_pool + d * page_bytes, (i - m * chunks) * kChunk, page_bytes);
  }
}

// --------------------------------------------------------------------- fork

__device__ __forceinline__ int parent_of(const int32_t* parent, int i, int rows) {
  const int p = parent[i];
  return p >= 0 && p < rows ? p : -1;
}

__device__ __forceinline__ void fork_gather(const KvTable& in, const KvTable& out, const int32_t* parent, uint64_t* bits,
                                            int64_t first, int64_t step) {
  page_bits(in.refs, in.pages, bits, true, first, step);
  const int64_t n = (int64_t)out.rows * out.width;
  for (int64_t i = first; i < n; i += step) {
    const int row = (int)(i / out.width), k = (int)(i - (int64_t)row * out.width);
    const int p = parent_of(parent, row, in.rows);
    out.table[i] = p < 0 ? -1 : in.table[(int64_t)p * in.width + k];
  }
  for (int64_t i = first; i < out.rows; i += step) {
    const int p = parent_of(parent, (int)i, in.rows);
    out.lens[i] = p < 0 ? 0 : in.lens[p];
  }
  for (int64_t i = first; i < in.pages; i += step) out.refs[i] = in.refs[i];
}

__global__ __launch_bounds__(256) void fork_gather_kernel(KvTable in, KvTable out, const int32_t* parent, uint64_t* bits) {
  fork_gather(in, out, parent, bits, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}

// By one work-group of 1024: children of each row of in (and the first of them)
// into LDS, the pages that are copied into src and their places into dst, by
// rank; their number, or -1 if the free pages do not suffice (*need says how
// many it would take).  at_of(i, k, page) is told that row i's last page is copy
// k.
template <class F>
__device__ __forceinline__ int fork_plan(const KvTable& in, int out_rows, int shift, const int32_t* parent,
                                         const uint64_t* bits, int* first, int* children, int32_t* src, int32_t* dst,
                                         int* need, F at_of) {
  const int tid = threadIdx.x;
  for (int r = tid; r < in.rows; r += kScan) {
    first[r] = 0x7fffffff;
    children[r] = 0;
  }
  __syncthreads();
  for (int i = tid; i < out_rows; i += kScan) {
    const int p = parent_of(parent, i, in.rows);
    if (p >= 0) {
      atomicMin(&first[p], i);
      atomicAdd(&children[p], 1);
    }
  }
  __syncthreads();
  int total = 0;
  for (int i0 = 0; i0 < out_rows; i0 += kScan) {
    const int i = i0 + tid;
    int page = -1;
    if (i < out_rows) {
      const int p = parent_of(parent, i, in.rows);
      const int len = p < 0 ? 0 : clamped_len(in, p, shift);
      if (len & ((1 << shift) - 1)) {
        page = in.table[(int64_t)p * in.width + (len >> shift)];
        if (page < 0 || page >= in.pages || (first[p] == i && in.refs[page] == 1)) page = -1;
      }
    }
    int all;
    const int before = block_exclusive(page >= 0 ? 1 : 0, &all);
    if (i < out_rows) at_of(i, page >= 0 ? total + before : -1);
    if (page >= 0) src[total + before] = page;
    total += all;
  }
  *need = total;
  const int nfree = list_bits(bits, (in.pages + 63) >> 6, dst, total);
  __syncthreads();
  return total > nfree ? -1 : total;
}

__global__ __launch_bounds__(kScan) void fork_plan_kernel(KvTable in, KvTable out, int shift, const int32_t* parent,
                                                          int32_t* info, KvScratch w) {
  __shared__ int s_first[kKvMaxRows], s_children[kKvMaxRows];
  const int tid = threadIdx.x;
  int need;
  const int n = fork_plan(in, out.rows, shift, parent, w.bits, s_first, s_children, w.src, w.list, &need,
                          [&](int i, int k) { w.row_a[i] = k; });
  for (int r = tid; r < in.rows; r += kScan) w.row_b[r] = s_children[r];
  if (tid == 0) {
    info[0] = n < 0 ? LOOPQ_KV_NO_PAGES : LOOPQ_KV_DONE;
    info[1] = need;
    w.head[0] = max(n, 0);
    w.head[1] = n < 0;
  }
  if (n < 0) return;
  for (int i = tid; i < out.rows; i += kScan) {
    const int k = w.row_a[i];
    if (k < 0) continue;
    const int p = parent_of(parent, i, in.rows);
    w.dst[k] = w.list[k];
    out.table[(int64_t)i * out.width + (clamped_len(in, p, shift) >> shift)] = w.list[k];
  }
}

// The whole fork in one launch, for small tables and pools: every work-group
// plans it for itself (in LDS, from the same inputs), then takes its share of
// the rows and of the contents; the first one has the reference counts.
constexpr int kForkRows = 1024, kForkPages = 8192;
__global__ __launch_bounds__(kScan) void fork_one_kernel(KvTable in, KvTable out, int shift, const int32_t* parent,
                                                         int32_t* info, char* pool, int64_t page_bytes) {
  __shared__ uint64_t s_bits[kForkPages / 64];
  __shared__ int s_first[kForkRows], s_children[kForkRows], s_rank[kForkRows], s_src[kForkRows], s_dst[kForkRows];
  __shared__ int s_refs[kForkPages];
  const int tid = threadIdx.x;
  page_bits(in.refs, in.pages, s_bits, true, tid, kScan);
  int need;
  const int n = fork_plan(in, out.rows, shift, parent, s_bits, s_first, s_children, s_src, s_dst, &need,
                          [&](int i, int k) { s_rank[i] = k; });
  __syncthreads();
  for (int i = blockIdx.x; i < out.rows; i += gridDim.x) {
    const int p = parent_of(parent, i, in.rows), k = s_rank[i];
    const int copied = n >= 0 && k >= 0 ? clamped_len(in, p, shift) >> shift : -1;
    for (int c = tid; c < out.width; c += kScan)
      out.table[(int64_t)i * out.width + c] = p < 0 || n < 0 ? -1 : c == copied ? s_dst[k] : in.table[(int64_t)p * in.width + c];
    if (tid == 0) out.lens[i] = p < 0 || n < 0 ? 0 : in.lens[p];
  }
  if (blockIdx.x == gridDim.x - 1) {
    if (tid == 0) {
      info[0] = n < 0 ? LOOPQ_KV_NO_PAGES : LOOPQ_KV_DONE;
      info[1] = need;
    }
    for (int p = tid; p < in.pages; p += kScan) s_refs[p] = in.refs[p];
    __syncthreads();
    if (n >= 0) {
      for (int i = tid; i < in.rows * in.width; i += kScan) {
        const int more = s_children[i / in.width] - 1;
        const int page = in.table[i];
        if (more != 0 && page >= 0 && page < in.pages) atomicAdd(&s_refs[page], more);
      }
      for (int m = tid; m < n; m += kScan) {
        atomicAdd(&s_refs[s_src[m]], -1);
        atomicAdd(&s_refs[s_dst[m]], 1);
      }
    }
    __syncthreads();
    for (int p = tid; p < in.pages; p += kScan) out.refs[p] = s_refs[p];
  }
  // four chunks of 16 KiB at a time
  const int64_t chunks = (page_bytes + 4 * kChunk - 1) / (4 * kChunk), all = chunks * n;
  for (int64_t i = blockIdx.x; i < all; i += gridDim.x) {
    const int m = (int)(i / chunks);
    const int64_t at = (i - m * chunks) * 4 * kChunk + (tid >> 8) * kChunk;
    if (at < page_bytes) copy_chunk(pool + s_src[m] * page_bytes, pool + s_dst[m] * page_bytes, at, page_bytes);
  }
}

// Reference counts by their differences (whole numbers: the order of the
// additions does not matter), and the partial pages' contents.
__global__ __launch_bounds__(256) void fork_apply_kernel(KvTable in, KvTable out, char* pool, int64_t page_bytes,
                                                         KvScratch w) {
  const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
  if (w.head[1]) {  // not enough pages: empty rows, the old references
    for (int64_t i = first; i < (int64_t)out.rows * out.width; i += step) out.table[i] = -1;
    for (int64_t i = first; i < out.rows; i += step) out.lens[i] = 0;
    return;
  }
  for (int64_t i = first; i < (int64_t)in.rows * in.width; i += step) {
    const int more = w.row_b[i / in.width] - 1;
    const int page = in.table[i];
    if (more != 0 && page >= 0 && page < in.pages) atomicAdd(&out.refs[page], more);
  }
  const int moves = w.head[0];
  for (int64_t i = first; i < moves; i += step) {
    atomicAdd(&out.refs[w.src[i]], -1);
    atomicAdd(&out.refs[w.dst[i]], 1);
  }
  const int64_t chunks = (page_bytes + kChunk - 1) / kChunk, n = chunks * moves;
  for (int64_t i = blockIdx.x; i < n; i += gridDim.x) {
    const int m = (int)(i / chunks);
    copy_chunk(pool + w.src[m] * page_bytes, pool + w.dst[m] * page_bytes, (i - m * chunks) * kChunk, page_bytes);
  }
}

// --------------------------------------------------------------------- trim

__global__ __launch_bounds__(256) void copy_refs_kernel(const int32_t* in, int32_t* out, int n) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < n) out[i] = in[i];
}

__device__ __forceinline__ void trim_entries(const KvTable& in, const KvTable& out, int shift, int window, int sinks,
                                             int64_t first, int64_t step) {
  for (int64_t i = first; i < (int64_t)in.rows * in.width; i += step) {
    const int row = (int)(i / in.width);
    const int64_t k = i - (int64_t)row * in.width;
    int page = in.table[i];
    if (((k + 1) << shift) <= (int64_t)clamped_len(in, row, shift) - window + 1 && (k << shift) >= sinks) {
      if (page >= 0 && page < in.pages) atomicAdd(&out.refs[page], -1);
      page = -1;
    }
    out.table[i] = page;
    if (k == 0) out.lens[row] = in.lens[row];
  }
}

__global__ __launch_bounds__(256) void trim_kernel(KvTable in, KvTable out, int shift, int window, int sinks) {
  trim_entries(in, out, shift, window, sinks, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}

__global__ __launch_bounds__(kScan) void trim_one_kernel(KvTable in, KvTable out, int shift, int window, int sinks) {
  if (in.refs != out.refs)
    for (int p = threadIdx.x; p < in.pages; p += kScan) out.refs[p] = in.refs[p];
  __syncthreads();
  trim_entries(in, out, shift, window, sinks, threadIdx.x, kScan);
}

// ------------------------------------------------------------------ compact

__global__ __launch_bounds__(256) void used_bits_kernel(const int32_t* refs, int pages, uint64_t* bits) {
  page_bits(refs, pages, bits, false, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}

// used pages before each word; their number L and how many lie at L or above
__global__ __launch_bounds__(kScan) void compact_scan_kernel(KvScratch w, int words, int32_t* info, const int32_t* refs,
                                                             int pages) {
  if (refs) {  // the bits, too
    page_bits(refs, pages, w.bits, false, threadIdx.x, kScan);
    __syncthreads();
  }
  int base = 0;
  for (int w0 = 0; w0 < words; w0 += kScan) {
    const int i = w0 + threadIdx.x;
    int all;
    const int at = base + block_exclusive(i < words ? __popcll(w.bits[i]) : 0, &all);
    if (i < words) w.prefix[i] = at;
    base += all;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    const int L = base;
    const int below = L == 0 ? 0 : (L >> 6) < words ? (int)(w.prefix[L >> 6] + __popcll(w.bits[L >> 6] & ((1ull << (L & 63)) - 1))) : L;
    w.head[0] = L - below;
    w.head[1] = below;
    w.head[2] = L;
    info[0] = L;
    info[1] = L - below;
  }
}

__device__ __forceinline__ int nth_set(uint64_t x, int k) {
  for (; k > 0; --k) x &= x - 1;
  return __ffsll((unsigned long long)x) - 1;
}

struct Used {
  const uint64_t* bits;
  const uint32_t* prefix;
  int words, pages, L, below;  // below: used pages under index L
  __device__ bool used(int p) const { return (bits[p >> 6] >> (p & 63)) & 1; }
  __device__ int rank(int p) const { return (int)prefix[p >> 6] + __popcll(bits[p >> 6] & ((1ull << (p & 63)) - 1)); }
  __device__ int nth_used(int k) const {  // the k-th used page of all
    int lo = 0, hi = words;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((int)prefix[mid] <= k) lo = mid;
      else hi = mid;
    }
    return (lo << 6) + nth_set(bits[lo], k - (int)prefix[lo]);
  }
  __device__ int nth_free(int k) const {  // the k-th free page of all
    int lo = 0, hi = words;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((mid << 6) - (int)prefix[mid] <= k) lo = mid;
      else hi = mid;
    }
    return (lo << 6) + nth_set(~bits[lo], k - ((lo << 6) - (int)prefix[lo]));
  }
  __device__ int to(int p) const { return p < L ? p : nth_free(rank(p) - below); }  // a used page's new index
};

__global__ __launch_bounds__(256) void compact_apply_kernel(KvTable in, KvTable out, char* pool, int64_t page_bytes,
                                                            int32_t* page_map, KvScratch w) {
  const Used u{w.bits, w.prefix, (in.pages + 63) >> 6, in.pages, w.head[2], w.head[1]};
  const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
  for (int64_t p = first; p < in.pages; p += step) {
    // a free page below L is written by the page that moves there
    if (u.used((int)p)) {
      const int to = u.to((int)p), n = in.refs[p];
      page_map[p] = to;
      if (to != p) out.refs[p] = 0;
      out.refs[to] = n;
    } else {
      page_map[p] = -1;
      if (p >= u.L) out.refs[p] = 0;
    }
  }
  for (int64_t i = first; i < (int64_t)in.rows * in.width; i += step) {
    const int p = in.table[i];
    // an entry whose page nobody holds by the counts is no page any more
    out.table[i] = p >= 0 && p < in.pages && u.used(p) ? u.to(p) : -1;
  }
  if (in.lens != out.lens)
    for (int64_t i = first; i < in.rows; i += step) out.lens[i] = in.lens[i];
  // each work-group moves a run of chunks: the search for a page's places is paid once a page
  const int64_t chunks = (page_bytes + kChunk - 1) / kChunk, n = chunks * w.head[0];
  const int64_t per = (n + gridDim.x - 1) / gridDim.x, end = min((blockIdx.x + 1) * per, n);
  int last = -1;
  const char* from = nullptr;
  char* to = nullptr;
  for (int64_t i = blockIdx.x * per; i < end; ++i) {
    const int m = (int)(i / chunks);
    if (m != last) {
      const int p = u.nth_used(u.below + m);
      from = pool + p * page_bytes;
      to = pool + u.nth_free(m) * page_bytes;
      last = m;
    }
    copy_chunk(from, to, (i - m * chunks) * kChunk, page_bytes);
  }
}

int shift_of(int page_size) { return 31 - __builtin_clz((unsigned)page_size); }

// work-groups of 256 threads for n independent items, at most `most`
int blocks_for(int64_t n, int most) {
  const int64_t b = (n + 255) / 256;
  return (int)(b < 1 ? 1 : b > most ? most : b);
}

}  // namespace

size_t kv_scratch_bytes(int64_t rows, int64_t pages) {
  const auto up = [](int64_t b) { return (size_t)((b + 255) / 256 * 256); };
  const int64_t words = (pages + 63) / 64;
  return up(words * 8) + up(words * 4) + up(pages * 4) + 4 * up(rows * 4) + 256;
}

KvScratch kv_carve(void* ws, int64_t rows, int64_t pages) {
  char* p = reinterpret_cast<char*>(ws);
  const auto take = [&p](int64_t b) {
    char* at = p;
    p += (b + 255) / 256 * 256;
    return at;
  };
  const int64_t words = (pages + 63) / 64;
  KvScratch w;
  w.bits = reinterpret_cast<uint64_t*>(take(words * 8));
  w.prefix = reinterpret_cast<uint32_t*>(take(words * 4));
  w.list = reinterpret_cast<int32_t*>(take(pages * 4));
  w.row_a = reinterpret_cast<int32_t*>(take(rows * 4));
  w.row_b = reinterpret_cast<int32_t*>(take(rows * 4));
  w.src = reinterpret_cast<int32_t*>(take(rows * 4));
  w.dst = reinterpret_cast<int32_t*>(take(rows * 4));
  w.head = reinterpret_cast<int32_t*>(take(256));
  return w;
}

hipError_t launch_kv_reserve(KvTable in, KvTable out, int page_size, const int32_t* grow, int32_t* info, KvScratch w,
                             hipStream_t s) {
  const int shift = shift_of(page_size);
  const int64_t n = (int64_t)in.pages + (int64_t)in.rows * in.width;
  if (n <= kOneGroup) {
    reserve_kernel<true><<<1, kScan, 0, s>>>(in, out, shift, grow, info, w);
  } else {
    reserve_copy_kernel<<<blocks_for(n, 1024), 256, 0, s>>>(in, out, w.bits);
    reserve_kernel<false><<<1, kScan, 0, s>>>(in, out, shift, grow, info, w);
  }
  return hipGetLastError();
}

hipError_t launch_kv_write(const KvWriteArgs& a, hipStream_t s) {
  const int64_t n = (int64_t)a.tokens * (a.heads * a.head_dim / 8);
  write_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_kv_fork(KvTable in, KvTable out, int page_size, void* pool, int64_t page_bytes, const int32_t* parent,
                          int32_t* info, KvScratch w, hipStream_t s) {
  const int shift = shift_of(page_size);
  const int64_t n = (int64_t)in.pages + (int64_t)out.rows * out.width;
  if (in.pages <= kForkPages && max(in.rows, out.rows) <= kForkRows && (int64_t)in.rows * in.width <= kOneGroup) {
    const int64_t most = max((int64_t)out.rows * ((page_bytes + 4 * kChunk - 1) / (4 * kChunk)), (int64_t)1);
    fork_one_kernel<<<(int)min(most, (int64_t)256), kScan, 0, s>>>(in, out, shift, parent, info,
                                                                  reinterpret_cast<char*>(pool), page_bytes);
    return hipGetLastError();
  }
  fork_gather_kernel<<<blocks_for(n, 1024), 256, 0, s>>>(in, out, parent, w.bits);
  fork_plan_kernel<<<1, kScan, 0, s>>>(in, out, shift, parent, info, w);
  const int64_t items = max((int64_t)in.rows * in.width, (int64_t)out.rows * out.width);
  const int64_t chunks = out.rows * ((page_bytes + kChunk - 1) / kChunk);  // at most
  fork_apply_kernel<<<blocks_for(max(items, chunks * 256), kCopyGroups), 256, 0, s>>>(in, out, reinterpret_cast<char*>(pool),
                                                                             page_bytes, w);
  return hipGetLastError();
}

hipError_t launch_kv_trim(KvTable in, KvTable out, int page_size, int window, int sinks, hipStream_t s) {
  const int64_t n = (int64_t)in.rows * in.width;
  const int shift = shift_of(page_size);
  if (in.pages + n <= kOneGroup) {
    trim_one_kernel<<<1, kScan, 0, s>>>(in, out, shift, window, sinks);
  } else {
    if (in.refs != out.refs) copy_refs_kernel<<<(in.pages + 255) / 256, 256, 0, s>>>(in.refs, out.refs, in.pages);
    trim_kernel<<<blocks_for(n, 2048), 256, 0, s>>>(in, out, shift, window, sinks);
  }
  return hipGetLastError();
}

hipError_t launch_kv_compact(KvTable in, KvTable out, void* pool, int64_t page_bytes, int32_t* page_map, int32_t* info,
                             KvScratch w, hipStream_t s) {
  const bool one = in.pages <= kOneGroup;
  if (!one) used_bits_kernel<<<blocks_for(in.pages, 1024), 256, 0, s>>>(in.refs, in.pages, w.bits);
  compact_scan_kernel<<<1, kScan, 0, s>>>(w, (in.pages + 63) / 64, info, one ? in.refs : nullptr, in.pages);
  const int64_t chunks = in.pages * ((page_bytes + kChunk - 1) / kChunk);  // at most
  compact_apply_kernel<<<blocks_for(max((int64_t)in.rows * in.width, chunks * 256), kCopyGroups), 256, 0, s>>>(
      in, out, reinterpret_cast<char*>(pool), page_bytes, page_map, w);
  return hipGetLastError();
}

hipError_t launch_kv_copy(const void* src_pool, int src_pages, const int32_t* src, void* dst_pool, int dst_pages,
                          const int32_t* dst, int count, int64_t page_bytes, hipStream_t s) {
  const int64_t chunks = count * ((page_bytes + kChunk - 1) / kChunk);
  copy_pages_kernel<<<blocks_for(chunks * 256, kCopyGroups), 256, 0, s>>>(
      reinterpret_cast<const char*>(src_pool), src_pages, src, reinterpret_cast<char*>(dst_pool), dst_pages, dst, count,
      page_bytes);
  return hipGetLastError();
}

}  // namespace loopq
