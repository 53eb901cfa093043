// Book-keeping of the paged key / value cache: growing, writing, forking,
// freeing, compacting and copying pages.
//
// None of it computes: each call moves 4-byte table cells and whole K / V rows,
// and what bounds it is the latency of a few dependent loads for the
// book-keeping (a table cell names a page, the page's count says whether it is
// shared) and memory bandwidth for the rows.  The number of pages that a call
// takes or moves is known on the device only, so a call is a plan kernel, which
// writes the list of moves, and a move kernel whose warps walk that list; the
// host never waits and the calls can be captured.
#include <cuda_bf16.h>

#include <algorithm>
#include <climits>
#include <initializer_list>
#include <numeric>

#include "cache.h"
#include "kernels.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kPlanThreads = 1024;  // one block: its scans order entries and pages
constexpr int kSms = 148;
// Entries of a fork or a page copy: each looks at all others for its destination,
// 0.4 s (fork) and 1 s (copy) at this many, and four times that at twice.
constexpr int kMaxPairs = 1 << 20;

// Moves of a call, in the workspace: page src[i] -> dst[i], its first rows[i]
// rows of every head and layer (0: nothing), i < *count.
struct Moves {
  int32_t* count;
  int32_t* src;
  int32_t* dst;
  int32_t* rows;
  int cap;  // entries the lists can hold
};

// Inclusive prefix sum over the block's threads; *total gets the sum of all.
// Every thread of the block takes part.  smem: 33 ints.
__device__ __forceinline__ int block_scan(int x, int* smem, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) smem[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int t = lane < static_cast<int>(blockDim.x >> 5) ? smem[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += y;
    }
    smem[lane] = t;
  }
  __syncthreads();
  const int before = warp > 0 ? smem[warp - 1] : 0;
  *total = smem[31];
  __syncthreads();  // smem may be reused by the next scan
  return x + before;
}

__device__ __forceinline__ int slot_length(const Cache& c, int s) {
  return min(max(get(c, c.lengths, s, c.slots), 0), c.max_pages * c.page_size);
}

// ---------------------------------------------------------------------------
// extend
// ---------------------------------------------------------------------------

struct ExtendWork {
  Moves moves;    // copies of shared last pages: entry i's at index i
  int32_t* mark;  // [slots]: first entry that names the slot
  int32_t* upto;  // [n]: pages needed by the entries up to and including i
  int32_t* info;  // [n]: bit 0 its last page is shared, bit 1 it may be granted
  int32_t* free;  // [pages]: free pages, lowest first, as many as are needed
};

__global__ void __launch_bounds__(kPlanThreads) extend_kernel(const Cache c, const int32_t* slots,
                                                             const int32_t* tokens, int n,
                                                             int32_t* start, const ExtendWork w) {
  __shared__ int scan[33];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  const int P = c.page_size;
  // the first entry of each slot
  for (int i = tid; i < n; i += kPlanThreads) {
    const int s = slots[i];
    if (s >= 0 && s < c.slots) put(c, w.mark, s, c.slots, INT_MAX);
  }
  __syncthreads();
  for (int i = tid; i < n; i += kPlanThreads) {
    const int s = slots[i];
    if (s >= 0 && s < c.slots && FA_IN_BOUNDS(c.status, s, 1, c.slots)) atomicMin(&w.mark[s], i);
  }
  __syncthreads();
  // pages each entry needs, and their running sum
  long long need_all = 0;
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int i = i0 + tid;
    int need = 0, info = 0;
    if (i < n) {
      const int s = slots[i];
      const int more = tokens[i];
      if (s >= 0 && s < c.slots && get(c, w.mark, s, c.slots) == i && more >= 0) {
        const int len = slot_length(c, s);
        const long long want = (static_cast<long long>(len) + more + P - 1) / P;
        if (want <= c.max_pages) {
          info = 2;
          const int have = (len + P - 1) / P;
          if (more > 0 && len % P != 0) {
            const int page =
                get(c, c.table, static_cast<long long>(s) * c.max_pages + have - 1, table_cells(c));
            if (page >= 0 && page < c.pages && get(c, c.refs, page, c.pages) > 1) info = 3;
          }
          need = static_cast<int>(want) - have + (info & 1);
        }
      }
    }
    int total = 0;
    const int upto = block_scan(need, scan, &total);  // at most 1024 * 2^20 + 1024
    if (i < n) {
      const long long u = need_all + upto;
      put(c, w.upto, i, w.moves.cap, static_cast<int>(u < INT_MAX ? u : INT_MAX));
      put(c, w.info, i, w.moves.cap, info | (need > 0 ? 4 : 0));
    }
    need_all += total;
  }
  // that many free pages, or all there are
  const int limit = static_cast<int>(need_all < c.pages ? need_all : c.pages);
  int found = 0;
  for (int p0 = 0; p0 < c.pages && found < limit; p0 += 4 * kPlanThreads) {
    const int p = p0 + 4 * tid;
    bool is_free[4];
    int mine = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      is_free[u] = p + u < c.pages && get(c, c.refs, p + u, c.pages) <= 0;
      mine += is_free[u];
    }
    int total = 0;
    int at = found + block_scan(mine, scan, &total) - mine;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (is_free[u]) {
        if (at < limit) put(c, w.free, at, c.pages, p + u);
        ++at;
      }
    found += total;
  }
  __syncthreads();
  // grant: a warp per entry, its lanes over the entry's new table cells
  const int lane = tid & 31;
  for (int i = tid >> 5; i < n; i += kPlanThreads / 32) {
    const int info = get(c, w.info, i, w.moves.cap), upto = get(c, w.upto, i, w.moves.cap);
    const bool granted = (info & 2) && (!(info & 4) || upto <= found);
    int copy_src = 0, copy_dst = 0, copy_rows = 0, first = -1;
    if (granted) {
      const int s = slots[i];
      const int len = slot_length(c, s);
      const int have = (len + P - 1) / P, shared = info & 1;
      const int want = (len + tokens[i] + P - 1) / P;
      const int need = want - have + shared;
      const long long row = static_cast<long long>(s) * c.max_pages;  // of the table
      if (shared) {
        copy_src = get(c, c.table, row + have - 1, table_cells(c));
        copy_dst = get(c, w.free, upto - need, c.pages);
        copy_rows = len % P;
      }
      __syncwarp();
      for (int j = lane; j < need; j += 32) {
        const int page = get(c, w.free, upto - need + j, c.pages);
        put(c, c.table, row + have - shared + j, table_cells(c), page);
        put(c, c.refs, page, c.pages, 1);
      }
      if (lane == 0) {
        if (shared && FA_IN_BOUNDS(c.status, copy_src, 1, c.pages)) atomicSub(&c.refs[copy_src], 1);
        put(c, c.lengths, s, c.slots, len + tokens[i]);
      }
      first = len;
    }
    if (lane == 0) {
      start[i] = first;
      put(c, w.moves.src, i, w.moves.cap, copy_src);
      put(c, w.moves.dst, i, w.moves.cap, copy_dst);
      put(c, w.moves.rows, i, w.moves.cap, copy_rows);
    }
  }
  if (tid == 0) *w.moves.count = n;
}

// ---------------------------------------------------------------------------
// moves: a warp per (move, layer, K or V, head)
// ---------------------------------------------------------------------------

constexpr int kAhead = 8;

__global__ void __launch_bounds__(256) move_kernel(const Cache from, const Cache to, const Moves m) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int chunks = from.d / 8;  // 16-byte pieces of a row
  const long long per_move = 2ll * from.layers * from.heads_kv;
  const long long items = *m.count * per_move;
  const long long warps = static_cast<long long>(gridDim.x) * (blockDim.x / 32);
  for (long long it = static_cast<long long>(blockIdx.x) * (blockDim.x / 32) + (threadIdx.x >> 5);
       it < items; it += warps) {
    const int i = static_cast<int>(it / per_move);
    const int rows = get(from, m.rows, i, m.cap);
    if (rows == 0) continue;
    const int page = get(from, m.src, i, m.cap), page_to = get(from, m.dst, i, m.cap);
    int r = static_cast<int>(it - i * per_move);
    const int h = r % from.heads_kv;
    r /= from.heads_kv;
    const int layer = r >> 1;
    const bool is_v = (r & 1) != 0;
    const long long src_at = is_v ? layer * from.v_layer + page * from.v_page + h * from.v_head
                                  : layer * from.k_layer + page * from.k_page + h * from.k_head;
    const long long dst_at = is_v ? layer * to.v_layer + page_to * to.v_page + h * to.v_head
                                  : layer * to.k_layer + page_to * to.k_page + h * to.k_head;
    const long long src_row = is_v ? from.v_row : from.k_row, dst_row = is_v ? to.v_row : to.k_row;
    // (a run of whole rows: its ends are the farthest elements)
    if (!FA_IN_BOUNDS(from.status, src_at, (rows - 1) * src_row + from.d, is_v ? from.ext_v : from.ext_k) ||
        !FA_IN_BOUNDS(to.status, dst_at, (rows - 1) * dst_row + to.d, is_v ? to.ext_v : to.ext_k))
      continue;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(is_v ? from.v : from.k) + src_at;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_v ? to.v : to.k) + dst_at;
    // eight loads in flight a lane, then their stores (697 MB read and written:
    // 116 us, 6.0 TB/s; with each load followed by its store 124)
    const int total = rows * chunks;
    for (int x0 = lane; x0 < total; x0 += 32 * kAhead) {
      uint4 v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int x = x0 + 32 * u, row = x / chunks, col = 8 * (x - row * chunks);
        if (x < total) v[u] = *reinterpret_cast<const uint4*>(src + row * src_row + col);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int x = x0 + 32 * u, row = x / chunks, col = 8 * (x - row * chunks);
        if (x < total) *reinterpret_cast<uint4*>(dst + row * dst_row + col) = v[u];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// write: a warp per token
// ---------------------------------------------------------------------------

struct WriteParams {
  Cache c;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  long long k_row, k_head, v_row, v_head;
  const int32_t* slots;
  const int32_t* start;
  const int32_t* cu;
  int layer, n, total;
#ifdef FA_DEBUG_BOUNDS
  long long ext_k, ext_v;  // elements of the new rows
#endif
};

__global__ void __launch_bounds__(256) write_kernel(const WriteParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (t >= p.total) return;
  int i = t, within = 0;
  if (p.cu != nullptr) {
    // last entry that begins at or before token t (entries may be empty)
    int lo = 0, hi = p.n;  // cu[lo] <= t < cu[hi] where t belongs to an entry
    if (p.cu[0] > t || p.cu[p.n] <= t) return;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (get(p.c, p.cu, mid, p.n + 1) <= t) lo = mid;
      else hi = mid;
    }
    i = lo;
    within = t - get(p.c, p.cu, lo, p.n + 1);
  }
  const int first = get(p.c, p.start, i, p.n), s = get(p.c, p.slots, i, p.n);
  if (first < 0 || s < 0 || s >= p.c.slots) return;
  const long long pos = static_cast<long long>(first) + within;
  const long long cell = pos / p.c.page_size;
  if (cell >= p.c.max_pages) return;
  const int page = get(p.c, p.c.table, static_cast<long long>(s) * p.c.max_pages + cell, table_cells(p.c));
  if (page < 0 || page >= p.c.pages) return;
  const int row = static_cast<int>(pos - cell * p.c.page_size);
  const int chunks = p.c.d / 8, half = p.c.heads_kv * chunks;
  const __nv_bfloat16 *ks = p.k + t * p.k_row, *vs = p.v + t * p.v_row;
  const long long k_at = p.layer * p.c.k_layer + page * p.c.k_page + row * p.c.k_row;
  const long long v_at = p.layer * p.c.v_layer + page * p.c.v_page + row * p.c.v_row;
  const int more = p.c.heads_kv - 1;  // (the last head's row is the farthest)
  if (!FA_IN_BOUNDS(p.c.status, k_at, more * p.c.k_head + p.c.d, p.c.ext_k) ||
      !FA_IN_BOUNDS(p.c.status, v_at, more * p.c.v_head + p.c.d, p.c.ext_v) ||
      !FA_IN_BOUNDS(p.c.status, t * p.k_row, more * p.k_head + p.c.d, p.ext_k) ||
      !FA_IN_BOUNDS(p.c.status, t * p.v_row, more * p.v_head + p.c.d, p.ext_v))
    return;
  __nv_bfloat16* kd = static_cast<__nv_bfloat16*>(p.c.k) + k_at;
  __nv_bfloat16* vd = static_cast<__nv_bfloat16*>(p.c.v) + v_at;
  constexpr int kPieces = 4;  // loads in flight a lane, as in move_kernel
  for (int x0 = lane; x0 < 2 * half; x0 += 32 * kPieces) {
    uint4 v[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int x = x0 + 32 * u, y = x >= half ? x - half : x;
      const int h = y / chunks, col = 8 * (y - h * chunks);
      if (x < 2 * half)
        v[u] = *reinterpret_cast<const uint4*>(x >= half ? vs + h * p.v_head + col
                                                         : ks + h * p.k_head + col);
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int x = x0 + 32 * u, y = x >= half ? x - half : x;
      const int h = y / chunks, col = 8 * (y - h * chunks);
      if (x < 2 * half)
        *reinterpret_cast<uint4*>(x >= half ? vd + h * p.c.v_head + col : kd + h * p.c.k_head + col) = v[u];
    }
  }
}

// ---------------------------------------------------------------------------
// fork and free: a block per entry
// ---------------------------------------------------------------------------

struct ForkWork {
  int32_t* rows;    // [n][max_pages]: the sources' table rows
  int32_t* lens;    // [n]: their lengths, -1 for entries that are skipped
  int n;
};

__global__ void __launch_bounds__(256) fork_take_kernel(const Cache c, const int32_t* src,
                                                        const int32_t* dst, const ForkWork w) {
  griddep_wait();
  griddep_launch_dependents();
  const int i = blockIdx.x;
  const int s = src[i], d = dst[i];
  bool skip = s == d || s < 0 || s >= c.slots || d < 0 || d >= c.slots;
  for (int j = threadIdx.x; j < i; j += blockDim.x) skip = skip || dst[j] == d;
  if (__syncthreads_or(skip)) {
    if (threadIdx.x == 0) put(c, w.lens, i, w.n, -1);
    return;
  }
  const long long row = static_cast<long long>(s) * c.max_pages;  // of the table
  const long long out = static_cast<long long>(i) * c.max_pages;  // of the saved rows
  for (int j = threadIdx.x; j < c.max_pages; j += blockDim.x) {
    const int page = get(c, c.table, row + j, table_cells(c));
    put(c, w.rows, out + j, static_cast<long long>(w.n) * c.max_pages, page);
    if (page >= 0 && page < c.pages && FA_IN_BOUNDS(c.status, page, 1, c.pages)) atomicAdd(&c.refs[page], 1);
  }
  if (threadIdx.x == 0) put(c, w.lens, i, w.n, slot_length(c, s));
}

__global__ void __launch_bounds__(256) fork_put_kernel(const Cache c, const int32_t* dst,
                                                       const ForkWork w) {
  griddep_wait();
  griddep_launch_dependents();
  const int i = blockIdx.x;
  const int len = get(c, w.lens, i, w.n);
  if (len < 0) return;
  const int d = dst[i];
  const long long row = static_cast<long long>(d) * c.max_pages;  // of the table
  const long long in = static_cast<long long>(i) * c.max_pages;   // of the saved rows
  for (int j = threadIdx.x; j < c.max_pages; j += blockDim.x) {
    const int page = get(c, c.table, row + j, table_cells(c));
    if (page >= 0 && page < c.pages && FA_IN_BOUNDS(c.status, page, 1, c.pages)) atomicSub(&c.refs[page], 1);
    put(c, c.table, row + j, table_cells(c), get(c, w.rows, in + j, static_cast<long long>(w.n) * c.max_pages));
  }
  if (threadIdx.x == 0) put(c, c.lengths, d, c.slots, len);
}

// The exchange lets a slot that is named twice go once.
__global__ void __launch_bounds__(256) free_kernel(const Cache c, const int32_t* slots) {
  griddep_wait();
  griddep_launch_dependents();
  const int s = slots[blockIdx.x];
  if (s < 0 || s >= c.slots) return;
  const long long row = static_cast<long long>(s) * c.max_pages;  // of the table
  for (int j = threadIdx.x; j < c.max_pages; j += blockDim.x) {
    if (!FA_IN_BOUNDS(c.status, row + j, 1, table_cells(c))) continue;
    const int page = atomicExch(&c.table[row + j], -1);
    if (page >= 0 && page < c.pages && FA_IN_BOUNDS(c.status, page, 1, c.pages)) atomicSub(&c.refs[page], 1);
  }
  if (threadIdx.x == 0) put(c, c.lengths, s, c.slots, 0);
}

// ---------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------

struct CompactWork {
  Moves moves;
  int32_t* now;  // [pages]: new number of a page that is numbered U or more
};

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const Cache c, int32_t* used,
                                                                   const CompactWork w) {
  __shared__ int scan[33];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  int mine = 0;
#pragma unroll 8
  for (int p = tid; p < c.pages; p += kPlanThreads) mine += get(c, c.refs, p, c.pages) > 0;
  int count = 0;
  block_scan(mine, scan, &count);
  // the k-th free page below `count` receives the k-th used one from it on;
  // eight consecutive pages a thread and scan
  constexpr int kPer = 8;
  int holes = 0, movers = 0;
  for (int p0 = 0; p0 < c.pages; p0 += kPer * kPlanThreads) {
    const int p = p0 + kPer * tid;
    uint32_t used_bits = 0;
#pragma unroll
    for (int u = 0; u < kPer; ++u)
      if (p + u < c.pages && get(c, c.refs, p + u, c.pages) > 0) used_bits |= 1u << u;
    const uint32_t below = low_bits(min(kPer, count - p)), inside = low_bits(min(kPer, c.pages - p));
    const uint32_t hole_bits = below & inside & ~used_bits, mover_bits = ~below & used_bits;
    int total = 0;
    const int own = __popc(hole_bits) | __popc(mover_bits) << 16;
    const int at = block_scan(own, scan, &total) - own;
    int hole = holes + (at & 0xFFFF), mover = movers + (at >> 16);
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      if ((hole_bits >> u) & 1u) put(c, w.moves.dst, hole++, w.moves.cap, p + u);
      if ((mover_bits >> u) & 1u) put(c, w.moves.src, mover++, w.moves.cap, p + u);
      else if (p + u >= count && p + u < c.pages) put(c, w.now, p + u, c.pages, p + u);
    }
    holes += total & 0xFFFF;
    movers += total >> 16;
  }
  __syncthreads();
  for (int k = tid; k < movers; k += kPlanThreads) {
    const int s = get(c, w.moves.src, k, w.moves.cap), d = get(c, w.moves.dst, k, w.moves.cap);
    put(c, w.moves.rows, k, w.moves.cap, c.page_size);
    put(c, w.now, s, c.pages, d);
    put(c, c.refs, d, c.pages, get(c, c.refs, s, c.pages));
    put(c, c.refs, s, c.pages, 0);
  }
  if (tid == 0) {
    *w.moves.count = movers;
    *used = count;
  }
}

__global__ void __launch_bounds__(256) renumber_kernel(const Cache c, const int32_t* used,
                                                       const int32_t* now) {
  griddep_wait();
  griddep_launch_dependents();
  const int count = *used;
  const long long cells = table_cells(c);
  for (long long x = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; x < cells;
       x += static_cast<long long>(gridDim.x) * blockDim.x) {
    const int page = get(c, c.table, x, table_cells(c));
    if (page >= count && page < c.pages) put(c, c.table, x, table_cells(c), get(c, now, page, c.pages));
  }
}

// ---------------------------------------------------------------------------
// copy: which pairs are made
// ---------------------------------------------------------------------------

// Where the two caches of a copy share memory, page for page: page s of the
// source lies (in some layer) where page d of the destination does iff
// by + s * from == d * to.
struct Shared {
  static constexpr int kMost = 16;
  int n;
  long long by[kMost], from[kMost], to[kMost];
};

__global__ void __launch_bounds__(256) copy_plan_kernel(const Cache from, const Cache to, const Shared sh,
                                                        const int32_t* src, const int32_t* dst,
                                                        int n, const Moves m) {
  griddep_wait();
  griddep_launch_dependents();
  const int i = blockIdx.x;
  const int s = src[i], d = dst[i];
  bool skip = s < 0 || s >= from.pages || d < 0 || d >= to.pages;
  for (int j = threadIdx.x; j < i; j += blockDim.x) skip = skip || dst[j] == d;
  for (int k = 0; k < sh.n; ++k) {
    // the source's page that lies where page d does (each = 0: it has one page)
    const long long at = d * sh.to[k] - sh.by[k], each = sh.from[k];
    const long long o = each > 0 ? at / each : 0;
    if (o * each != at || o < 0 || o >= from.pages) continue;
    const int page = static_cast<int>(o);
    for (int j = threadIdx.x; j < n; j += blockDim.x) skip = skip || src[j] == page;
  }
  skip = __syncthreads_or(skip);
  if (threadIdx.x == 0) {
    put(to, m.src, i, m.cap, s);
    put(to, m.dst, i, m.cap, d);
    put(to, m.rows, i, m.cap, skip ? 0 : to.page_size);
    if (i == 0) *m.count = n;
  }
}

// ---------------------------------------------------------------------------
// workspaces and launches
// ---------------------------------------------------------------------------

// ints, each array rounded up to 64 of them
int64_t round64(int64_t x) { return (x + 63) / 64 * 64; }

struct Carve {
  int32_t* at;
  int32_t* take(int64_t ints) {
    int32_t* p = at;
    at += round64(ints);
    return p;
  }
};

Moves carve_moves(Carve* w, int64_t n) {
  Moves m;
  m.count = w->take(1);
  m.src = w->take(n);
  m.dst = w->take(n);
  m.rows = w->take(n);
  m.cap = static_cast<int>(n);
  return m;
}

// Each call's workspace.  Only a fork saves table rows: n * max_pages cells,
// which the others' lists have no use for (65536 entries of 8192 pages: 2 GiB).
int64_t moves_ints(int64_t n) { return 64 + 3 * round64(n); }
int64_t extend_ints(const Cache& c, int n) {
  return moves_ints(n) + 2 * round64(n) + round64(c.slots) + round64(c.pages);
}
int64_t fork_ints(const Cache& c, int n) {
  return round64(n) + round64(static_cast<int64_t>(n) * c.max_pages);
}
int64_t compact_ints(const Cache& c) { return moves_ints(c.pages) + round64(c.pages); }

bool workspace_ok(int64_t ints, const void* ws, size_t bytes) {
  return cache_aligned(ws, 256) && bytes >= static_cast<size_t>(ints) * 4;
}

// The places at which K or V of `of` shares memory with K or V of `to`: views of
// one pool, their pages or layers apart.  False if there are more of them than
// fit (no such views of one pool are known).
bool shared_of(const Cache& of, const Cache& to, Shared* sh) {
  struct Part {
    const void* base;
    long long layer, page, head, row;
  };
  const Part f[2] = {{of.k, of.k_layer, of.k_page, of.k_head, of.k_row},
                     {of.v, of.v_layer, of.v_page, of.v_head, of.v_row}};
  const Part t[2] = {{to.k, to.k_layer, to.k_page, to.k_head, to.k_row},
                     {to.v, to.v_layer, to.v_page, to.v_head, to.v_row}};
  sh->n = 0;
  for (const Part& a : f)
    for (const Part& b : t) {
      // other strides: not the same pages
      if ((of.layers > 1 && a.layer != b.layer) || (of.heads_kv > 1 && a.head != b.head) ||
          (of.page_size > 1 && a.row != b.row))
        continue;
      const long long pf = of.pages > 1 ? a.page : 0, pt = to.pages > 1 ? b.page : 0;
      const long long apart = static_cast<long long>(reinterpret_cast<intptr_t>(a.base) -
                                                     reinterpret_cast<intptr_t>(b.base)) / 2;
      const long long low = -(of.pages - 1) * pf, high = (to.pages - 1) * pt;  // of `by`, below
      const long long step = std::gcd(pf, pt);
      long long l0 = 0, l1 = 0;  // layers of the source ahead of the destination's
      if (of.layers > 1) {
        l0 = std::max<long long>(-(of.layers - 1), (low - apart) / a.layer - 1);
        l1 = std::min<long long>(of.layers - 1, (high - apart) / a.layer + 1);
      }
      for (long long l = l0; l <= l1; ++l) {
        const long long by = apart + l * a.layer;
        if (by < low || by > high || (step > 0 ? by % step : by) != 0) continue;
        // in steps (pages, where both have the same): K's and V's are mostly one
        const long long unit = step > 0 ? step : 1;
        bool known = false;
        for (int i = 0; i < sh->n; ++i)
          known = known || (sh->by[i] == by / unit && sh->from[i] == pf / unit && sh->to[i] == pt / unit);
        if (known) continue;
        if (sh->n == Shared::kMost) return false;
        sh->by[sh->n] = by / unit;
        sh->from[sh->n] = pf / unit;
        sh->to[sh->n++] = pt / unit;
      }
    }
  return true;
}

bool ints_ok(const void* p) { return cache_aligned(p, 4); }

// Warps for every (move, layer, tensor, head) of up to `moves` moves, within
// two waves of 8-warp blocks: the move kernel's warps walk the rest.
unsigned move_blocks(const Cache& c, int64_t moves) {
  const int64_t warps = moves * 2 * c.layers * c.heads_kv;
  const int64_t blocks = (warps + 7) / 8;
  return static_cast<unsigned>(blocks < kSms * 16 ? (blocks < 1 ? 1 : blocks) : kSms * 16);
}

fa_status_t done(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

}  // namespace
}  // namespace fa

extern "C" {

size_t fa_cache_extend_workspace_size(const fa_cache_t* cache, int n) {
  fa::Cache c;
  if (fa::cache_resolve(cache, false, &c) != FA_OK || n < 0) return 0;
  return static_cast<size_t>(fa::extend_ints(c, n)) * 4;
}

size_t fa_cache_fork_workspace_size(const fa_cache_t* cache, int n) {
  fa::Cache c;
  if (fa::cache_resolve(cache, false, &c) != FA_OK || n < 0) return 0;
  return static_cast<size_t>(fa::fork_ints(c, n)) * 4;
}

size_t fa_cache_compact_workspace_size(const fa_cache_t* cache) {
  fa::Cache c;
  if (fa::cache_resolve(cache, false, &c) != FA_OK) return 0;
  return static_cast<size_t>(fa::compact_ints(c)) * 4;
}

size_t fa_cache_copy_pages_workspace_size(const fa_cache_t* cache, int n) {
  fa::Cache c;
  if (fa::cache_resolve(cache, false, &c) != FA_OK || n < 0) return 0;
  return static_cast<size_t>(fa::moves_ints(n)) * 4;
}

size_t fa_cache_workspace_size(const fa_cache_t* cache, int n) {
  size_t most = 0;
  for (const size_t x : {fa_cache_extend_workspace_size(cache, n), fa_cache_fork_workspace_size(cache, n),
                         n < 0 ? size_t{0} : fa_cache_compact_workspace_size(cache),
                         fa_cache_copy_pages_workspace_size(cache, n)})
    most = x > most ? x : most;
  return most;
}

fa_status_t fa_cache_extend(const fa_cache_t* cache, const int32_t* slots, const int32_t* tokens,
                            int n, int32_t* start, void* workspace, size_t workspace_bytes,
                            void* stream) {
  fa::Cache c;
  const fa_status_t st = fa::cache_resolve(cache, true, &c);
  if (st != FA_OK) return st;
  if (n < 0) return FA_ERR_INVALID_ARG;
  if (n == 0) return FA_OK;
  if (!fa::ints_ok(slots) || !fa::ints_ok(tokens) || !fa::ints_ok(start)) return FA_ERR_INVALID_ARG;
  if (!fa::workspace_ok(fa::extend_ints(c, n), workspace, workspace_bytes)) return FA_ERR_WORKSPACE;
  fa::Carve carve{static_cast<int32_t*>(workspace)};
  fa::ExtendWork w;
  w.moves = fa::carve_moves(&carve, n);
  w.upto = carve.take(n);
  w.info = carve.take(n);
  w.mark = carve.take(c.slots);
  w.free = carve.take(c.pages);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = fa::launch_overlapped(fa::extend_kernel, dim3(1), dim3(fa::kPlanThreads), 0, s, c,
                                        slots, tokens, n, start, w);
  if (e == cudaSuccess)
    e = fa::launch_overlapped(fa::move_kernel, dim3(fa::move_blocks(c, n)), dim3(256), 0, s, c, c,
                              w.moves);
  return fa::done(e);
}

fa_status_t fa_cache_write(const fa_cache_t* cache, int layer, const void* k, const void* v,
                           int64_t k_row, int64_t k_head, int64_t v_row, int64_t v_head,
                           const int32_t* slots, const int32_t* start, const int32_t* cu, int n,
                           int total, void* stream) {
  fa::WriteParams p;
  const fa_status_t st = fa::cache_resolve(cache, false, &p.c);
  if (st != FA_OK) return st;
  if (layer < 0 || layer >= p.c.layers || n < 0 || total < 0 || (cu == nullptr && total != n))
    return FA_ERR_INVALID_ARG;
  if (n == 0 || total == 0) return FA_OK;
  if (!fa::cache_aligned(k, 16) || !fa::cache_aligned(v, 16) || !fa::ints_ok(slots) ||
      !fa::ints_ok(start) || (reinterpret_cast<uintptr_t>(cu) & 3u) != 0)
    return FA_ERR_INVALID_ARG;
  if (!fa::cache_stride_ok(k_row, 1) || !fa::cache_stride_ok(v_row, 1) ||
      !fa::cache_stride_ok(k_head, 1) || !fa::cache_stride_ok(v_head, 1))
    return FA_ERR_INVALID_ARG;
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.k_row = k_row;
  p.k_head = k_head;
  p.v_row = v_row;
  p.v_head = v_head;
  p.slots = slots;
  p.start = start;
  p.cu = cu;
  p.layer = layer;
  p.n = n;
  p.total = total;
#ifdef FA_DEBUG_BOUNDS
  p.ext_k = (total - 1) * k_row + (p.c.heads_kv - 1) * k_head + p.c.d;
  p.ext_v = (total - 1) * v_row + (p.c.heads_kv - 1) * v_head + p.c.d;
#endif
  return fa::done(fa::launch_overlapped(fa::write_kernel, dim3((static_cast<unsigned>(total) + 7) / 8),
                                        dim3(256), 0, static_cast<cudaStream_t>(stream), p));
}

fa_status_t fa_cache_fork(const fa_cache_t* cache, const int32_t* src, const int32_t* dst, int n,
                          void* workspace, size_t workspace_bytes, void* stream) {
  fa::Cache c;
  const fa_status_t st = fa::cache_resolve(cache, true, &c);
  if (st != FA_OK) return st;
  if (n < 0) return FA_ERR_INVALID_ARG;
  if (n == 0) return FA_OK;
  if (n > fa::kMaxPairs) return FA_ERR_UNSUPPORTED;
  if (!fa::ints_ok(src) || !fa::ints_ok(dst)) return FA_ERR_INVALID_ARG;
  if (!fa::workspace_ok(fa::fork_ints(c, n), workspace, workspace_bytes)) return FA_ERR_WORKSPACE;
  fa::Carve carve{static_cast<int32_t*>(workspace)};
  fa::ForkWork w;
  w.lens = carve.take(n);
  w.rows = carve.take(static_cast<int64_t>(n) * c.max_pages);
  w.n = n;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = fa::launch_overlapped(fa::fork_take_kernel, dim3(static_cast<unsigned>(n)),
                                        dim3(256), 0, s, c, src, dst, w);
  if (e == cudaSuccess)
    e = fa::launch_overlapped(fa::fork_put_kernel, dim3(static_cast<unsigned>(n)), dim3(256), 0, s,
                              c, dst, w);
  return fa::done(e);
}

fa_status_t fa_cache_free(const fa_cache_t* cache, const int32_t* slots, int n, void* stream) {
  fa::Cache c;
  const fa_status_t st = fa::cache_resolve(cache, true, &c);
  if (st != FA_OK) return st;
  if (n < 0) return FA_ERR_INVALID_ARG;
  if (n == 0) return FA_OK;
  if (!fa::ints_ok(slots)) return FA_ERR_INVALID_ARG;
  return fa::done(fa::launch_overlapped(fa::free_kernel, dim3(static_cast<unsigned>(n)), dim3(256), 0,
                                        static_cast<cudaStream_t>(stream), c, slots));
}

fa_status_t fa_cache_compact(const fa_cache_t* cache, int32_t* used, void* workspace,
                             size_t workspace_bytes, void* stream) {
  fa::Cache c;
  const fa_status_t st = fa::cache_resolve(cache, true, &c);
  if (st != FA_OK) return st;
  if (!fa::ints_ok(used)) return FA_ERR_INVALID_ARG;
  if (!fa::workspace_ok(fa::compact_ints(c), workspace, workspace_bytes)) return FA_ERR_WORKSPACE;
  fa::Carve carve{static_cast<int32_t*>(workspace)};
  fa::CompactWork w;
  w.moves = fa::carve_moves(&carve, c.pages);
  w.now = carve.take(c.pages);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = fa::launch_overlapped(fa::compact_plan_kernel, dim3(1), dim3(fa::kPlanThreads), 0, s,
                                        c, used, w);
  if (e == cudaSuccess)
    e = fa::launch_overlapped(fa::move_kernel, dim3(fa::move_blocks(c, c.pages)), dim3(256), 0, s, c, c,
                              w.moves);
  if (e == cudaSuccess) {
    const int64_t blocks = (static_cast<int64_t>(c.slots) * c.max_pages + 255) / 256;
    e = fa::launch_overlapped(fa::renumber_kernel,
                              dim3(static_cast<unsigned>(blocks < fa::kSms * 8 ? blocks : fa::kSms * 8)),
                              dim3(256), 0, s, c, static_cast<const int32_t*>(used),
                              static_cast<const int32_t*>(w.now));
  }
  return fa::done(e);
}

fa_status_t fa_cache_copy_pages(const fa_cache_t* cache, const fa_cache_t* from, const int32_t* src,
                                const int32_t* dst, int n, void* workspace,
                                size_t workspace_bytes, void* stream) {
  fa::Cache to, of;
  fa_status_t st = fa::cache_resolve(cache, false, &to);
  if (st == FA_OK) st = fa::cache_resolve(from != nullptr ? from : cache, false, &of);
  if (st != FA_OK) return st;
  if (n < 0) return FA_ERR_INVALID_ARG;
  if (of.layers != to.layers || of.page_size != to.page_size || of.heads_kv != to.heads_kv ||
      of.d != to.d)
    return FA_ERR_INVALID_ARG;
  if (n == 0) return FA_OK;
  if (n > fa::kMaxPairs) return FA_ERR_UNSUPPORTED;
  if (!fa::ints_ok(src) || !fa::ints_ok(dst)) return FA_ERR_INVALID_ARG;
  if (!fa::workspace_ok(fa::moves_ints(n), workspace, workspace_bytes)) return FA_ERR_WORKSPACE;
  fa::Carve carve{static_cast<int32_t*>(workspace)};
  const fa::Moves m = fa::carve_moves(&carve, n);
  fa::Shared shared;
  if (!fa::shared_of(of, to, &shared)) return FA_ERR_UNSUPPORTED;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = fa::launch_overlapped(fa::copy_plan_kernel, dim3(static_cast<unsigned>(n)), dim3(256),
                                        0, s, of, to, shared, src, dst, n, m);
  if (e == cudaSuccess)
    e = fa::launch_overlapped(fa::move_kernel, dim3(fa::move_blocks(to, n)), dim3(256), 0, s, of, to, m);
  return fa::done(e);
}

}  // extern "C"
