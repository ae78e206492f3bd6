// Attention of several new tokens a row over the paged cache, causal, with a
// sliding window and sinks (attention.hip has the method).
//
// Bound by arithmetic where prompts are long: 2 prompts of 8192 tokens, 16 heads of
// 128, bf16: 0.55 TFLOP in 551 to 567 us, 970 to 998 TFLOP/s (a large bf16 matrix product
// reaches 1263 to 1302 here); the shader clock reads 1.7 GHz meanwhile, so that what counts is
// work per key tile, 2.1 us for 256 rows.  Steps on the way: products of 128 rows
// from K and V through registers 1438 us; copied to LDS without registers 887; the
// reference moved only when left behind, reads ahead of the products, tasks by XCD
// 655; 256 rows, a ring of buffers, heads in blocks 608; tiles without masks and
// checks as runs of numbers 563; one branch a tile for all that is rare, queries
// loaded after the first tiles, no spills 552.  Without effect: three buffers instead of four,
// barriers split in two, wave priorities, other mixes of products and vector work.
// fp32 queries, the same prompts: 1555 us, 354 TFLOP/s where three planes for one leave
// a third of 1300, since one wave a SIMD takes turns between products and vector work.
#include "attn_core.h"

namespace loopq {
namespace {

// Rows of a query tile are (query, head of the group) pairs, heads fastest.
template <int ROWS>
__device__ __forceinline__ int query_tiles(const AttnArgs& a, int n) {
  return (int)(((int64_t)n * a.group + ROWS - 1) / ROWS);
}
template <int ROWS>
__device__ __forceinline__ Tiles tile_keys(const AttnArgs& a, int t, int n, int len, int* lo, int* hi) {
  const int64_t r0 = (int64_t)t * ROWS, r1 = min(r0 + ROWS, (int64_t)n * a.group) - 1;
  *lo = len - n + (int)(r0 / a.group);
  *hi = len - n + (int)(r1 / a.group);
  return visible_tiles(a, *lo, *hi, 6);
}

// the larger of lanes x and x + 32, in both
__device__ __forceinline__ float max_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// exclusive sum over 1024 threads, and the sum of all; `part` is 16 values of scratch
__device__ __forceinline__ int64_t sum_before(int64_t v, int64_t* part, int64_t* all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t x = v;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t y = __shfl_up(x, off, 64);
    if (lane >= off) x += y;
  }
  __syncthreads();
  if (lane == 63) part[wave] = x;
  __syncthreads();
  int64_t before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) {
    before += w < wave ? part[w] : 0;
    sum += part[w];
  }
  *all = sum;
  return before + x - v;
}

// One work-group.  A task is an item or, where an item has more than L key
// tiles, a part of it of at most L; L is a work-group's even share of all key
// tiles, so that few long items are split over the whole chip and many stay
// whole.  Slots take the results of split items' tasks: at most 2 tiles / L.  All
// key heads have the same tasks; they are written down once.
template <int ROWS>
__global__ __launch_bounds__(1024) void prefill_plan_kernel(AttnArgs a, AttnPlan pl) {
  __shared__ int64_t part[16];
  __shared__ int32_t s_rows[1025];
  const int tid = threadIdx.x;
  if (tid < 64) reinterpret_cast<uint32_t*>(const_cast<uint16_t*>(pl.zeros))[tid] = 0;
  if (tid < 8) pl.next[tid] = 0;
  int64_t T = 0, all;  // query tiles; only an order of cu that is not ascending gives more than there is room for
  for (int r0 = 0; r0 < a.rows; r0 += 1024) {
    const int r = r0 + tid;
    int first;
    const int n = r < a.rows ? query_tiles<ROWS>(a, row_queries(a, r, &first)) : 0;
    const int64_t at = min(T + sum_before(n, part, &all), (int64_t)pl.most_tiles);
    if (r < a.rows) {
      pl.row_tiles[r] = (int32_t)at;
      if (r < 1024) s_rows[r] = (int32_t)at;
    }
    T = min(T + all, (int64_t)pl.most_tiles);
  }
  __syncthreads();
  const int32_t* row_tiles = a.rows <= 1024 ? s_rows : pl.row_tiles;
  const auto item_of = [&](int t, Tiles* tl) {
    PrefillTask x;
    x.row = find(row_tiles, a.rows, t);
    x.n = row_queries(a, x.row, &x.first);
    x.len = row_len(a, x.row);
    x.tile = t - row_tiles[x.row];
    *tl = tile_keys<ROWS>(a, x.tile, x.n, x.len, &x.lo, &x.hi);
    x.head = tl->head;
    x.from = tl->from;
    return x;
  };
  int64_t keys = 0;
  PrefillTask mine;  // query tile tid: most calls have no more than 1024
  Tiles mine_tl{0, 0, 0};
  for (int64_t t = tid; t < T; t += 1024) {
    Tiles tl;
    const PrefillTask x = item_of((int)t, &tl);
    if (t < 1024) {
      mine = x;
      mine_tl = tl;
    }
    keys += tl.n;
  }
  sum_before(keys, part, &all);
  const int64_t L = max((int64_t)4, (all * a.heads + kPrefillGroups - 1) / kPrefillGroups);
  int64_t base = 0;  // tasks in the low half, slots in the high one
  for (int64_t t0 = 0; t0 < T; t0 += 1024) {
    const int64_t t = t0 + tid;
    Tiles tl{0, 0, 0};
    PrefillTask x;
    if (t < 1024) {
      x = mine;
      tl = mine_tl;
    } else if (t < T) {
      x = item_of((int)t, &tl);
    }
    const int64_t parts = (tl.n + L - 1) / L;
    const int64_t at = base + sum_before(parts + (parts > 1 ? parts << 32 : 0), part, &all);
    x.parts = (int32_t)parts;
    x.slot = (int32_t)(at >> 32);
    for (int i = 0; i < (int)parts; ++i) {
      x.part = i;
      x.k0 = (int32_t)(i * L);
      x.k1 = (int32_t)min((i + 1) * L, (int64_t)tl.n);
      x.pad[0] = x.pad[1] = 0;
      pl.tasks[(int32_t)at + i] = x;
    }
    base += all;
  }
  if (tid == 0) {
    pl.head[0] = (int32_t)base;
    pl.head[1] = (int32_t)(base >> 32);
    pl.head[2] = min(max(a.heads * a.rows / 8, 1), a.heads);
  }
}

// Task x of Z for each of the key heads.  Heads come in blocks, as many as share
// an XCD; in a block the tasks of a head go from the last, since a row's last
// query tile has the most keys, to the first, each for every head: work-groups
// that run together read the same keys, and what is handed out at the end is
// short.
__device__ __forceinline__ int which_task(const AttnArgs& a, int Z, int block, int x, int* kvh) {
  const int b = x / (block * Z), heads = min(block, a.heads - b * block);
  x -= b * block * Z;
  const int y = x / heads;
  *kvh = b * block + x - y * heads;
  return Z - 1 - y;
}

// a task that lies in LDS, for the whole wave
__device__ __forceinline__ PrefillTask read_task(const PrefillTask& t) {
  PrefillTask r;
  const int32_t* from = reinterpret_cast<const int32_t*>(&t);
  int32_t* to = reinterpret_cast<int32_t*>(&r);
#pragma unroll
  for (int i = 0; i < 16; ++i) to[i] = __builtin_amdgcn_readfirstlane(from[i]);
  return r;
}

// 16 bytes per lane from src + OFF (bytes, per lane) to LDS at byte dst + DST +
// 16 lane (dst a scalar), without passing the registers.  The compiler does not see
// the write: a reader waits for loads_done() and the barrier after it.  The
// offset counts for the target, too; one wait state lies between the write of
// m0 and its use.
template <int OFF, int DST>
__device__ __forceinline__ void load_lds16(const void* src, uint32_t dst) {
  asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off offset:%2" ::"s"(dst), "v"(src), "n"(OFF),
               "n"(DST - OFF)
               : "memory", "m0", "scc");
}
// 4 bytes per lane to LDS at byte dst + 4 lane, in the same manner
__device__ __forceinline__ void load_lds4(const void* src, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(dst), "v"(src) : "memory", "m0");
}
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}
// all but the wave's last N vector memory operations are done
template <int N>
__device__ __forceinline__ void loads_done() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ bool finite_bf16x2(uint32_t w) {
  return (w & 0x7f80u) != 0x7f80u && (w & 0x7f800000u) != 0x7f800000u;
}

// a barrier that waits for LDS operations, but not for copies to LDS under way
__device__ __forceinline__ void sync_lds() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// A work-group takes a task after another: W waves of 32 rows each over tiles of
// 64 keys, K and V of the next three tiles on their way to a ring of four
// buffers in LDS while one is multiplied.  The next task is asked for late, so
// that no work-group keeps one waiting while another is idle, its description and
// page entries are fetched during the last three tiles, and its first tiles are on
// their way while results are stored (12 rows with 1500 new tokens, 32 query heads of
// 96, window 1000: asked for at the start 209 us, late 190, fetched ahead 180; 171
// with the steps above).  Keys that no query of the item
// sees are read from a line of zeros.  fp32 queries hold three planes in registers
// and take half the rows.
template <int D, bool F32, int W>
__global__ __launch_bounds__(64 * W, W / 4) void prefill_attn_kernel(AttnArgs a, AttnPlan pl) {
  constexpr int NQ = F32 ? 3 : 1;
  constexpr int ROWS = 32 * W, THREADS = 64 * W;
  constexpr int C = D / 8, S = D / 32;  // chunks and blocks of a row
  constexpr int kTile = kPrefillKeys * C;
  constexpr int kCopies = 8 * S / W;  // of a wave for one tile
  constexpr int R = 4;  // buffers of the ring: copies run three tiles ahead
  __shared__ u32x4 s_k[R * kTile], s_v[R * kTile];
  __shared__ __attribute__((aligned(8))) uint16_t s_valid[R][4];  // keys of a tile that some query sees, 16 a wave
  __shared__ int64_t s_pages[512];  // 64 tiles' groups of eight keys: their place in the pool in bytes, -1 for no page
  __shared__ int s_entry[512];      // the next task's page entries
  __shared__ PrefillTask s_tasks[2];  // the task at work and the next one, in turn
  __shared__ int s_task, s_head;    // its number, or -1; its key head
  __shared__ int s_odd;     // some result is not finite
  __shared__ int s_paged;   // every group of those 64 tiles that some query sees has a page
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n32 = lane & 31, h = lane >> 5;
  const int in_page = (1 << a.page_shift) - 1;
  const int Z = pl.head[0], block = pl.head[2];
  const int64_t tasks = (int64_t)Z * a.heads;
  // Work-groups go round the eight XCDs; each XCD has an eighth of the tasks
  // (neighbours share keys, and with them an L2), a first one per work-group and
  // the rest in turn, then helps out in the other eighths.  Which work-group
  // takes a task does not change its result.
  constexpr int kPer = kPrefillGroups / 8;
  const int eighth = blockIdx.x & 7;
  const auto start_of = [&](int e) { return (int)(tasks * e / 8); };
  const int own = start_of(eighth) + kPer, own_left = start_of(eighth + 1) - own;
  int task = own - kPer + (int)(blockIdx.x >> 3);
  if (task >= start_of(eighth + 1)) task = -1;

  // this lane's share of a tile's copy: its key, and a chunk of each block
  const int wave0 = __builtin_amdgcn_readfirstlane(wave);
  const int my_key = (wave0 & 3) * 16 + (lane >> 2);
  const int my_off = (my_key & 7) * (2 * D) + 16 * ((lane & 3) ^ (lane >> 4));  // bytes from its group of eight keys
  const uint32_t to_k = lds_offset(s_k) + (wave0 & 3) * 1024, to_v = lds_offset(s_v) + (wave0 & 3) * 1024;
  const int64_t* my_pages = s_pages + (my_key >> 3);
  // chunks this lane multiplies
  int k_at[2], v_at[2];  // in the first block; the others follow every 256 chunks
#pragma unroll
  for (int c = 0; c < 2; ++c) k_at[c] = chunk_at<6, false>(n32, 2 * c + h);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int x = lane & 15, g = lane >> 4;
    v_at[e] = chunk_at<6, false>(4 * h + 8 * e + (x >> 2), 2 * (g & 1) + ((x & 3) >> 1));
  }

  int turn = 0, kvh = 0;  // the task at work is s_tasks[turn]: scalar registers are short
  // What follows down to q0 is set by start(), and is the next task's from there on:
  // results are stored by the finished task's own description.
  // Its tiles by number n.  A tile is copied plainly if every key of it is seen by
  // some query, and taken whole if every key is seen by every query; both are
  // runs of numbers (tiles of sinks count as neither), as long as the pages are
  // there.
  int tiles, k0, head, from, hi, low;  // low: the first key in some query's window
  int plain0, plain1, whole0, whole1;
  const char* base;  // this lane's first byte of its key head's keys or values in page 0
  bool paged;        // of the tiles that are copied
  bool few, busy;    // few keys a query; the wave has rows
  int pos;           // of this lane's query
  int64_t q0;        // where this lane's part of its query starts

  const auto key_in = [&](int k0, int head, int from, int n) {  // first key of tile n of a task
    const int i = k0 + n;
    return (i < head ? i : from + i - head) << 6;
  };
  const auto key_of = [&](int n) { return key_in(k0, head, from, n); };
  const auto in_window = [&](int p) { return a.window > 0 ? (int)max((int64_t)p - a.window + 1, (int64_t)0) : 0; };  // first key
  // some query sees a key of group j .. j + 7 (of those up to hi)
  const auto any_sees = [&](int j, int hi, int low) { return j <= hi && (j + 7 >= low || j < a.sinks); };
  // places of tiles n .. n + 63, from the table or from the entries fetched; barriers on both sides
  const auto read_pages = [&](int n, bool fetched) {
    sync_lds();
    if (tid == 0) s_paged = 1;
    sync_lds();
    const int32_t* table = a.table + (int64_t)__builtin_amdgcn_readfirstlane(s_tasks[turn].row) * a.width;
    for (int e = tid; e < 512; e += THREADS) {
      const int i = n + (e >> 3), j = key_of(i) + 8 * (e & 7);
      int64_t at = -1;
      if (i < tiles && any_sees(j, hi, low)) {
        const int page = fetched ? s_entry[e] : table[j >> a.page_shift];
        if ((uint32_t)page < (uint32_t)a.num_pages) at = 2 * (page * a.page_stride + (j & in_page) * D);
        else s_paged = 0;
      }
      s_pages[e] = at;
    }
    sync_lds();
    return __builtin_amdgcn_readfirstlane(s_paged) != 0;
  };
  // where this wave's copies of tile i come from: K and V with four waves, one of
  // them with eight; past the last tile, zeros (so that the loop needs no branch)
  struct Source {
    const char *k, *v;
  };
  const auto plain_source = [&](int64_t at) { return Source{base + at, base + at + (W == 4 ? 2 * a.plane : 0)}; };
  const auto masked_source = [&](int n, int64_t at, int buf) {
    bool in = n < tiles && at >= 0;
    if (in) {
      const int j = key_of(n) + my_key;
      in = j <= hi && (j >= low || j < a.sinks);
    }
    const unsigned long long there = __ballot(in);
    if (lane == 0 && wave0 < 4) s_valid[buf][wave0] = every_fourth(there);
    const char* zero = reinterpret_cast<const char*>(pl.zeros);
    return Source{in ? base + at : zero, W == 4 && in ? base + at + 2 * a.plane : zero};
  };
  const auto copy_block = [&](const Source& x, int buf, int b) {  // b a constant once unrolled
    const auto go = [&](const char* p, uint32_t dst) {
      if (b == 0) load_lds16<0, 0>(p, dst);
      else if (b == 1) load_lds16<64, 4096>(p, dst);
      else if (b == 2) load_lds16<128, 8192>(p, dst);
      else load_lds16<192, 12288>(p, dst);
    };
    go(x.k, (W == 8 && wave0 >= 4 ? to_v : to_k) + buf * (kTile * 16));
    if (W == 4) go(x.v, to_v + buf * (kTile * 16));
  };
  // this lane's row of a task: its query, head and position
  struct Row {
    bool has;
    int qi, hq, pos;
  };
  const auto row_of = [&](const PrefillTask& t, int kvh) {
    const int q = t.lo - (t.len - t.n);  // the tile's first query
    const int64_t before = (int64_t)t.tile * ROWS;
    const int g0 = (int)(before - (int64_t)q * a.group);  // and the head of its first row
    const int left = (int)min((int64_t)t.n * a.group - before, (int64_t)ROWS), x = wave0 * 32 + n32;
    const uint32_t u = g0 + min(x, left - 1), dq = u / (uint32_t)a.group;
    Row r;
    r.has = x < left;
    r.qi = q + (int)dq;
    r.hq = kvh * a.group + (int)(u - dq * a.group);
    r.pos = t.len - t.n + r.qi;
    return r;
  };
  const auto has_rows = [&](const PrefillTask& t) { return (int64_t)t.tile * ROWS + wave0 * 32 < (int64_t)t.n * a.group; };  // this wave
  // the task's first tiles on their way; no copy may be under way
  const auto start = [&](bool fetched) {
    const PrefillTask t = read_task(s_tasks[turn]);
    tiles = t.k1 - t.k0;
    k0 = t.k0;
    head = t.head;
    from = t.from;
    hi = t.hi;
    low = in_window(t.lo);
    const int low_all = in_window(t.hi), shift0 = t.head - t.from - t.k0;  // window tile w is number w + shift0
    plain0 = max(((low + 63) >> 6) + shift0, max(head - k0, 0));
    plain1 = min(((hi + 1) >> 6) + shift0, tiles);
    whole0 = max(((low_all + 63) >> 6) + shift0, plain0);
    whole1 = min(((t.lo + 1) >> 6) + shift0, tiles);
    // bf16 weights are rounded by up to 2^-8 of themselves; over many keys that
    // averages out, with few the weights take a second plane
    few = !F32 && (t.lo < 255 || (a.window > 0 && a.window < 256));
    base = reinterpret_cast<const char*>(a.pool + (((int64_t)kvh << a.page_shift) * D) + (W == 8 && wave0 >= 4 ? a.plane : 0)) + my_off;
    const Row r = row_of(t, kvh);
    pos = r.pos;
    busy = has_rows(t);
    q0 = (int64_t)(t.first + r.qi) * a.ldq + (int64_t)r.hq * D + 8 * h;
    paged = read_pages(0, fetched);
#pragma unroll
    for (int t = 0; t < R - 1; ++t) {
      const Source x = masked_source(t, my_pages[t * 8], t);
#pragma unroll
      for (int b = 0; b < S; ++b) copy_block(x, t, b);
    }
  };

  f32x16 o[S];
  float m, l;
  bool started = false;
  for (;;) {
    if (!started) {
      if (task < 0) {  // what the other eighths have left
        __syncthreads();  // every wave has read s_task
        if (wave0 == 0) {
          int found = -1;
          uint64_t open = 0xff;  // a try that fails closes an eighth for good: nine rounds at most
          for (;;) {
            const int e = (eighth + lane) & 7;
            const int left = max(start_of(e + 1) - start_of(e) - kPer, 0);
            const int taken = __hip_atomic_load(pl.next + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            open &= __ballot(lane < 8 && taken < left);
            if (open == 0) break;
            const int at = __ffsll((unsigned long long)open) - 1, f = (eighth + at) & 7;
            int x = lane == 0 ? atomicAdd(pl.next + f, 1) : 0;
            x = __builtin_amdgcn_readfirstlane(x);
            if (x < start_of(f + 1) - start_of(f) - kPer) {
              found = start_of(f) + kPer + x;
              break;
            }
            open &= ~(1ull << at);
          }
          if (lane == 0) s_task = found;
        }
        __syncthreads();
        task = __builtin_amdgcn_readfirstlane(s_task);
        if (task < 0) return;
      }
      const PrefillTask* p = pl.tasks + which_task(a, Z, block, task, &kvh);
      int i = tid;
      asm("" : "+v"(i));  // formed here: addresses kept for it through the loop would spill
      if (i < 16) reinterpret_cast<int32_t*>(s_tasks + turn)[i] = reinterpret_cast<const int32_t*>(p)[i];
      __syncthreads();
      start(false);
    }
    const int ask = own_left > 0 && tiles >= 3 ? tiles - 3 : 0x3fffffff;

    const auto run_tiles = [&](auto planes, bool careful) {
      constexpr int NP = decltype(planes)::n;
      bf16x8 q[D / 16][NQ];
#pragma unroll
      for (int c = 0; c < D / 16; ++c) load_query(a, pl.qmul, q0 + 16 * c, true, q[c]);
#pragma unroll
      for (int d = 0; d < S; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[d][r] = 0.0f;
      m = -INFINITY;
      l = 0.0f;
      if (tid == 0) s_odd = 0;
      bool paged_now = paged;  // of the tiles that are multiplied
      const int asking = careful ? 0x3fffffff : ask;
      int event = 0, buf = 0;
      for (int n = 0; n < tiles; ++n, buf = (buf + 1) & (R - 1)) {
        const int ahead = n + R - 1, after = (buf + R - 1) & (R - 1);  // the tile to copy, where tile n - 1 was
        // this wave's copies of tile n have landed (those of the next two may be under way), then everybody's
        loads_done<(R - 2) * kCopies>();
        sync_lds();
        if (n == event) {  // one branch for all that most tiles have not
          if ((ahead & 63) == 0) paged = read_pages(ahead, false);
          if ((n & 63) == 0) paged_now = paged;
          if (n >= asking) {
            // the next task: its number, two tiles later its description, at the
            // end of the last tile its page entries
            if (n == ask) {
              if (wave0 == 0) {
                const int x = __builtin_amdgcn_readfirstlane(lane == 0 ? atomicAdd(pl.next + eighth, 1) : 0);
                if (lane == 0) s_task = x < own_left ? own + x : -1;
                if (x < own_left) {
                  int head;
                  const PrefillTask* p = pl.tasks + which_task(a, Z, block, own + x, &head);
                  if (lane == 0) s_head = head;
                  if (lane < 16) load_lds4(reinterpret_cast<const int32_t*>(p) + lane, lds_offset(s_tasks + (turn ^ 1)));
                }
              }
            } else if (n == ask + 2 && __builtin_amdgcn_readfirstlane(s_task) >= 0) {
              const PrefillTask t = read_task(s_tasks[turn ^ 1]);
              const int t_low = in_window(t.lo);
              for (int e = wave0 * 64; e < 512; e += THREADS) {
                const int i = (e + lane) >> 3, j = key_in(t.k0, t.head, t.from, i) + 8 * (lane & 7);
                const bool any = i < t.k1 - t.k0 && any_sees(j, t.hi, t_low);
                load_lds4(a.table + (int64_t)t.row * a.width + (any ? j >> a.page_shift : 0), lds_offset(s_entry) + e * 4);
              }
            }
          }
          // the next of: ahead and n at multiples of 64, the last three tiles
          event = min(min(((ahead + 64) & ~63) - (R - 1), (n + 64) & ~63), max(asking, n + 1));
        }
        const int64_t at = my_pages[(ahead & 63) * 8];
        __builtin_amdgcn_sched_barrier(0);
        const u32x4 *kt = s_k + buf * kTile, *vt = s_v + buf * kTile;
        f32x16 s[2];
        if (busy) {
          // all reads of K ahead of its products
          u32x4 kf[D / 16][2];
#pragma unroll
          for (int c = 0; c < D / 16; ++c)
#pragma unroll
            for (int t = 0; t < 2; ++t) kf[c][t] = kt[k_at[c & 1] + (c >> 1) * 256 + t * 128];
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[t][r] = 0.0f;
#pragma unroll
          for (int c = 0; c < D / 16; ++c)
#pragma unroll
            for (int n = NQ - 1; n >= 0; --n)
#pragma unroll
              for (int t = 0; t < 2; ++t)
                s[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, kf[c][t]), q[c][n], s[t], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
        mfma_settle_before_join();
        const bool whole = paged_now && n >= whole0 && n < whole1;
        if (careful) {
          for (int at = tid; at < kTile; at += THREADS) {
            u32x4 v = s_v[buf * kTile + at];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if ((v[e] & 0x7f80u) == 0x7f80u) v[e] &= 0xffff0000u;
              if ((v[e] & 0x7f800000u) == 0x7f800000u) v[e] &= 0xffffu;
            }
            s_v[buf * kTile + at] = v;
          }
          __syncthreads();
        }
        Source src;
        if (paged && ahead >= plain0 && ahead < plain1) src = plain_source(at);
        else src = masked_source(ahead, at, after);
        if (!busy) {
#pragma unroll
          for (int b = 0; b < S; ++b) copy_block(src, after, b);
          continue;
        }
        // V of the first two key quarters while the products finish
        bf16x8 vf[2][S];
        const auto read_v = [&](int kc) {
#pragma unroll
          for (int d = 0; d < S; ++d)
            vf[kc & 1][d] = join_halves(read_tr(vt, v_at[0] + d * 256 + kc * 64, lane & 1), read_tr(vt, v_at[1] + d * 256 + kc * 64, lane & 1));
        };
        read_v(0);
        read_v(1);
        __builtin_amdgcn_sched_barrier(0);
        if (!whole) {
          const int j0 = key_of(n);
          uint64_t seen = below(pos - j0 + 1);
          if (a.window > 0) seen &= ~below((int64_t)pos - a.window + 1 - j0) | below((int64_t)a.sinks - j0);
          // the first tiles of a task are copied by masks, too
          if (n < R - 1 || !(paged_now && n >= plain0 && n < plain1)) seen &= *reinterpret_cast<const uint64_t*>(s_valid[buf]);
          seen >>= 4 * h;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const uint32_t w = (uint32_t)(seen >> (32 * t));
#pragma unroll
            for (int r = 0; r < 16; ++r)
              if (!(w & (1u << (8 * (r >> 2) + (r & 3))))) s[t][r] = -INFINITY;
          }
        }
        float tops[2] = {s[0][0], s[1][0]};
#pragma unroll
        for (int r = 1; r < 16; ++r)
#pragma unroll
          for (int t = 0; t < 2; ++t) tops[t] = fmaxf(tops[t], s[t][r]);
        const float top = max_halves(fmaxf(tops[0], tops[1])) * pl.c;
        // the reference follows only when it is left far behind: weights up to 2^8
        // are as exact, and rescaling costs a pass over o; each query's by its own
        // scores, so that keys which only its neighbours see leave no trace
        if (__any(top > m + 8.0f)) {
          const float mn = top > m + 8.0f ? top : m;
          const float f = __builtin_amdgcn_exp2f(m - (mn == -INFINITY ? 0.0f : mn));
          m = mn;
          l *= f;
#pragma unroll
          for (int d = 0; d < S; ++d) o[d] *= f;
        }
        const float ref = m == -INFINITY ? 0.0f : m;
        bf16x8 w[2][NP];
        const auto weights = [&](int kc) {
          float p[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            p[e] = __builtin_amdgcn_exp2f(fmaf(s[kc >> 1][8 * (kc & 1) + e], pl.c, -ref));
            if (NP > 1) l += p[e];
          }
          split_weights<NP>(p, w[kc & 1]);
          if (NP == 1) {  // the sum of the rounded weights: what rounding does to all of them alike cancels
            typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
            const bf16x2 one = {(__bf16)1.0f, (__bf16)1.0f};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              l = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{w[kc & 1][0][2 * e], w[kc & 1][0][2 * e + 1]}, one, l, false);
          }
        };
        weights(0);
        __builtin_amdgcn_sched_barrier(0);
        // the next quarter's weights are formed beside this one's products, and
        // the copies of the tile ahead spread between them
#pragma unroll
        for (int kc = 0; kc < 4; ++kc) {
          if (kc < S) copy_block(src, after, kc);
          if (kc < 3) weights(kc + 1);
#pragma unroll
          for (int d = 0; d < S; ++d)
#pragma unroll
            for (int n = NP - 1; n >= 0; --n) o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[kc & 1][d], w[kc & 1][n], o[d], 0, 0, 0);
          if (kc < 2) read_v(kc + 2);
          if (NP == 1 && kc < 3) {
#pragma unroll
            for (int d = 0; d < S; ++d) {
              __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);    // a product,
              __builtin_amdgcn_sched_group_barrier(0x402, 7, 0);  // its share of the vector work
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      mfma_settle_before_join();
      loads_done<0>();
    };
    // A weight of 0 does not keep out a value that is infinite or NaN.  Where a
    // result is not finite, the task is run once more with such values taken out
    // of the tiles; then they are added for the queries that see them.
    bool careful = false;
    for (;;) {
      if constexpr (F32) run_tiles(Planes<3>(), careful);
      else if (few) run_tiles(Planes<2>(), careful);
      else run_tiles(Planes<1>(), careful);
      bool odd = false;
#pragma unroll
      for (int d = 0; d < S; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) odd |= !(fabsf(o[d][r]) < INFINITY);
      if (!careful && odd) s_odd = 1;
      if (!careful && tiles < 3 && tid == 0) {  // too short to ask ahead
        const int x = own_left > 0 ? atomicAdd(pl.next + eighth, 1) : 0;
        s_task = x < own_left ? own + x : -1;
      }
      __syncthreads();  // also: the next tiles go over buffers that may still be read
      if (careful || s_odd == 0) break;
      careful = true;
      start(false);
    }
    const PrefillTask done = read_task(s_tasks[turn]);
    const int done_head = kvh;
    task = own_left > 0 ? __builtin_amdgcn_readfirstlane(s_task) : -1;
    started = task >= 0 && ask < 0x3fffffff;
    turn ^= 1;
    if (started) {
      kvh = __builtin_amdgcn_readfirstlane(s_head);
      start(true);
    }
    const Row mine = row_of(done, done_head);  // `pos` is the next task's by now
    if (careful) {
      for (int j = key_in(done.k0, done.head, done.from, 0); j <= done.hi; ++j) {
        const int tile = j >> 6, i = tile < done.head ? tile : tile - done.from + done.head;
        if ((tile >= done.head && tile < done.from) || i < done.k0 || i >= done.k1) continue;
        const int page = a.table[(int64_t)done.row * a.width + (j >> a.page_shift)];
        if ((uint32_t)page >= (uint32_t)a.num_pages || !sees(a, mine.pos, j)) continue;
        const uint16_t* v = a.pool + a.plane + page * a.page_stride + (((int64_t)done_head << a.page_shift) + (j & in_page)) * D + 4 * h;
#pragma unroll
        for (int d = 0; d < S; ++d)
#pragma unroll
          for (int r = 0; r < 16; r += 4) {
            const u32x2 y = *reinterpret_cast<const u32x2*>(v + 32 * d + 2 * r);
            if (finite_bf16x2(y[0]) && finite_bf16x2(y[1])) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float z = bf16_bits_to_float(e & 1 ? y[e >> 1] >> 16 : y[e >> 1] & 0xffffu);
              if (!(fabsf(z) < INFINITY)) o[d][r + e] += z;
            }
          }
      }
    }
    l += __shfl_xor(l, 32, 64);
    if (done.parts == 1) {
      const float f = l > 0.0f || l != l ? 1.0f / l : 0.0f;
      if (mine.has) {
        const int64_t at = (int64_t)(done.first + mine.qi) * a.ldo + (int64_t)mine.hq * D + 4 * h;
#pragma unroll
        for (int d = 0; d < S; ++d)
#pragma unroll
          for (int r = 0; r < 16; r += 4) {
            const f32x4 v = f32x4{o[d][r], o[d][r + 1], o[d][r + 2], o[d][r + 3]} * f;
            if (a.bf16)
              *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(a.out) + at + 32 * d + 2 * r) = u32x2{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3])};
            else
              *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.out) + at + 32 * d + 2 * r) = v;
          }
      }
    } else if (has_rows(done)) {  // `busy` is the next task's by now
      const int slot = done_head * pl.head[1] + done.slot + done.part;
      if (tid == 0) pl.records[slot] = JoinRecord{done.part == 0 ? done.parts : 0, done.row, done_head, done.tile};
      int r0 = wave0 * 32 + n32;
      asm("" : "+v"(r0));  // formed here: addresses kept for it through the loop would spill
      float* dst = pl.part + ((int64_t)slot * ROWS + r0) * D + 4 * h;
#pragma unroll
      for (int d = 0; d < S; ++d)
#pragma unroll
        for (int r = 0; r < 16; r += 4)
          *reinterpret_cast<f32x4*>(dst + 32 * d + 2 * r) = f32x4{o[d][r], o[d][r + 1], o[d][r + 2], o[d][r + 3]};
      if (h == 0) {
        pl.ml[slot * 2 * ROWS + r0] = m;
        pl.ml[(slot * 2 + 1) * ROWS + r0] = l;
      }
    }
  }
}

// Joins split items, a wave per row, and clears rows whose query tile no key
// tile belongs to.  16 parts of 16 x 256 rows (33 MB): 10.5 us.
template <int D, int ROWS>
__global__ __launch_bounds__(256) void prefill_join_kernel(AttnArgs a, AttnPlan pl) {
  __shared__ SplitItem s_list[kPrefillSlots];
  const int wave = threadIdx.x >> 6, waves = gridDim.x * 4, me = blockIdx.x * 4 + wave;
  const int n = split_items(pl.records, pl.head[1] * a.heads, s_list);
  for (int x = me; x < n * ROWS; x += waves) {
    const SplitItem rec = s_list[x / ROWS];
    const int slot = rec.at, r = x % ROWS;
    int first;
    const int64_t rows = (int64_t)row_queries(a, rec.row, &first) * a.group, rr = (int64_t)rec.tile * ROWS + r;
    if (rr >= rows) continue;
    float o[2];
    const float l = join_parts<D, ROWS>(pl, rec.parts, 0, 1, r, [&](int i) { return (int64_t)slot + i; }, o);
    const int qi = (int)(rr / a.group), hq = rec.item * a.group + (int)(rr - (int64_t)qi * a.group);
    store_row<D>(a, (int64_t)(first + qi) * a.ldo + (int64_t)hq * D, o, l);
  }
  // queries at negative positions whose whole tile sees nothing
  for (int row = blockIdx.x; row < a.rows; row += gridDim.x) {
    int first;
    const int n = row_queries(a, row, &first), len = row_len(a, row);
    if (n <= len) continue;
    for (int t = 0; t < query_tiles<ROWS>(a, n); ++t) {
      int lo, hi;
      if (tile_keys<ROWS>(a, t, n, len, &lo, &hi).n > 0) break;
      const int64_t r1 = min(((int64_t)t + 1) * ROWS, (int64_t)n * a.group);
      for (int64_t r = (int64_t)t * ROWS + wave; r < r1; r += 4) {
        const int qi = (int)(r / a.group), g = (int)(r - (int64_t)qi * a.group);
        const float z[2] = {0.0f, 0.0f};
        for (int kvh = 0; kvh < a.heads; ++kvh)
          store_row<D>(a, (int64_t)(first + qi) * a.ldo + (int64_t)(kvh * a.group + g) * D, z, 0.0f);
      }
    }
  }
}

template <int D, bool F32>
hipError_t launch(const AttnArgs& a, const AttnPlan& pl, hipStream_t s) {
  constexpr int W = F32 ? 4 : 8;
  prefill_plan_kernel<32 * W><<<1, 1024, 0, s>>>(a, pl);
  prefill_attn_kernel<D, F32, W><<<kPrefillGroups, 64 * W, 0, s>>>(a, pl);
  prefill_join_kernel<D, 32 * W><<<512, 256, 0, s>>>(a, pl);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_prefill(const AttnArgs& a, const AttnPlan& pl, hipStream_t s) {
  switch (a.head_dim) {
    case 64: return a.bf16 ? launch<64, false>(a, pl, s) : launch<64, true>(a, pl, s);
    case 96: return a.bf16 ? launch<96, false>(a, pl, s) : launch<96, true>(a, pl, s);
    default: return a.bf16 ? launch<128, false>(a, pl, s) : launch<128, true>(a, pl, s);
  }
}

}  // namespace loopq
