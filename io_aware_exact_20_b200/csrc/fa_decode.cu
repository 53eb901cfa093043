// Attention of one new token per sequence over the paged key / value cache.
//
// Per (sequence, K / V head) the group's query heads (up to 16 at a time)
// attend the visible keys in one pass: S = Q K^T, the running row maximum and
// sum of the online softmax, O += P V.  Every K / V row is read once from
// memory and serves the whole group, 2 G operations per byte, so the kernel is
// bound by memory bandwidth as long as the arithmetic keeps out of the way.
// The products are transposed, S^T = K Q^T and O^T = V^T P^T, on warp-level bf16
// matrix instructions (m16n8k16): the 16 rows are keys, or columns of V, and the
// 8 columns the group's heads (twice 8 for groups of 9 and more), so a group
// of up to 8 heads wastes at most its padding to 8.  (With the heads as the 16
// rows, half the instructions of a group of 4 worked on padding and the
// accumulators left registers for two warps per scheduler, which then waited
// for their own instructions more than for memory; a 128-row tcgen05 tile would
// be nearly all padding.)  Every warp works on its own tiles of KT keys with
// its own ring of asynchronous copies, so that no warp waits for another before
// the end.
//
// The work is cut evenly whatever the lengths are: each (sequence, K / V head,
// block of heads) is a row of tiles, the rows of the batch lie end to end, and
// every warp of the grid takes an equal share of them, found from the lengths
// on the device.  Its copies run ahead across the ends of rows.  A row that ends
// in another share than it begins is written as one partial result per share
// (fp32 sums with their maximum and row sum) and joined, in the order of the
// shares, by a second kernel; other rows are written at once.
//
// Few rows of few tiles, where latency counts, take another way to the same sums:
// a cluster of up to 8 blocks per row, whose warps take turns, and whose parts
// meet through the cluster's shared memory: one launch, no shares to work out
// and nothing to join (one sequence of 500 keys 6.6 us instead of 7.8, 32 of 64 keys
// over 8 K / V heads 5.2 instead of 9.4).
//
// Visible keys are counted u = 0 .. n_vis - 1: the first `sinks` that the window
// does not reach, then the window.  A tile is KT consecutive u, each with its
// own table lookup, so pages may be of any size, tiles may straddle pages, and
// the window and first tokens cost no partly used tiles.  Keys past the end
// and keys of a missing page are filled with zeros and masked: what stands in
// a page behind a sequence's end (infinities, NaN) never enters a product.
#include <cuda_bf16.h>

#include "cache.h"
#include "devctx.h"
#include "kernels.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr float kLn2 = 0.693147180559945309f;
constexpr double kLog2e = 1.4426950408889634074;

struct AttendParams {
  Cache c;
  const __nv_bfloat16* k;  // of the layer
  const __nv_bfloat16* v;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  long long q_batch, q_head, o_batch, o_head;
  const int32_t* slots;
  int batch, heads, group;
  int block_heads;   // query heads of a row: 8, or 16 where a K / V head has more than 8
  int head_blocks;   // rows per K / V head
  float scale_log2;  // softmax_scale * log2(e)
  int window, sinks;
  // partial results of the shares, null where no row can be cut
  int cluster;            // blocks per row (CL)
  uint32_t grid;          // blocks, and the shares they can have at most
  int shares;
  float2* part_stat;      // [2 * shares][16]: maximum (log2 units), row sum
  float* part_acc;        // [2 * shares][16][D]
  // [batch + 1]: spans of the sequences before each, and of all, for batches that
  // are longer than a joining block should add up by itself; else null
  uint32_t* spans;
#ifdef FA_DEBUG_BOUNDS
  long long ext_k, ext_v;  // elements from the layer's k, v to the pool's end
  long long ext_q, ext_o;
#endif
};

// Rows of partial results and LSE entries of a call.
__device__ __forceinline__ long long part_rows(const AttendParams& p) {
  return p.part_stat != nullptr ? 32ll * p.shares : 0;
}
__device__ __forceinline__ long long lse_count(const AttendParams& p) {
  return static_cast<long long>(p.batch) * p.heads;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  const int bytes = live ? 16 : 0;  // 0: sixteen zero bytes, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Sixteen bytes of the pool, base its layer's first element.
__device__ __forceinline__ void copy16(const AttendParams& p, uint32_t dst, const __nv_bfloat16* src,
                                       const __nv_bfloat16* base, long long extent) {
  if (FA_IN_BOUNDS(p.c.status, src - base, 8, extent)) cp_async16(dst, src, true);
  else cp_async16(dst, base, false);
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// C (16 x 8, fp32) += A (16 x 16, bf16) B (16 x 8, bf16)
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of bf16 held as pairs: (row g, columns 2 q4,
// 2 q4 + 1) in, (column g, rows 2 q4, 2 q4 + 1) out.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Sum over the eight rows of a column: the lanes with the same q4.
__device__ __forceinline__ float sum_rows(float x) {
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}
// Asks for a line that will be read soon.
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// All threads of the cluster's blocks meet; what they wrote to shared memory
// before is seen by all of them after.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// Two floats from the same place in the shared memory of the cluster's block c.
__device__ __forceinline__ float2 cluster_load2(const void* p, uint32_t c) {
  uint32_t at;
  float2 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(c));
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
  return v;
}

constexpr int kWarps = 4;

// D: head dim in the kernel, NB: blocks of 8 query heads of a row.
template <int D, int NB>
struct DecodeCfg {
  static constexpr int KT = D == 64 ? 32 : 16;   // keys of a warp's tile
  static constexpr int STAGES = 3;               // tiles in a warp's ring
  static constexpr uint32_t ROW = D * 2;         // bytes of a row in shared memory
  static constexpr uint32_t STAGE = 2 * KT * ROW;  // K then V
  static constexpr uint32_t WARP = STAGES * STAGE;
  static constexpr uint32_t OFF_VALID = kWarps * WARP;  // [warp][stage] key bits
  static constexpr uint32_t SMEM = OFF_VALID + kWarps * STAGES * 4;
  static constexpr int MIN_BLOCKS = D == 256 ? 1 : 2;
};

constexpr int kThreads = kWarps * 32;
// W tiles in n shares: the first W % n hold one tile more.  All tile counts
// fit 32 bits (checked on the host: 64-bit divisions took 1 us of every call).
struct Shares {
  uint32_t n, each, more;
  __device__ __forceinline__ Shares(uint32_t W, uint32_t count) : n(count), each(W / count), more(W % count) {}
  __device__ __forceinline__ uint32_t begin(uint32_t c) const { return c * each + min(c, more); }
  __device__ __forceinline__ uint32_t holding(uint32_t f) const {
    const uint32_t big = more * (each + 1);
    return f < big ? f / (each + 1) : more + (f - big) / each;
  }
};

// Keys a query sees: u -> key position (see the head of the file).
struct Visible {
  int count, first, from;  // u < first: key u; else key u - first + from
  __device__ __forceinline__ int key(int u) const { return u < first ? u : u - first + from; }
};

__device__ __forceinline__ Visible visible_of(int n, int window, int sinks) {
  Visible s;
  s.from = window > 0 && window < n ? n - window : 0;
  s.first = min(sinks, s.from);
  s.count = s.first + n - s.from;
  return s;
}

// Eight columns of query head h of sequence b: O = out / sum, LSE = ln2 (m + log2 sum).
// A sum of zero is a row that sees nothing (0, -inf); one that is not a number stays so in both.
__device__ __forceinline__ void write_row(const AttendParams& p, int b, int h, int col, float m, float sum,
                                          const float (&out)[8]) {
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const long long at = b * p.o_batch + h * p.o_head + col;
  if (FA_IN_BOUNDS(p.c.status, at, 8, p.ext_o))
    *reinterpret_cast<uint4*>(p.o + at) =
        make_uint4(pack_bf16(out[0] * inv, out[1] * inv), pack_bf16(out[2] * inv, out[3] * inv),
                   pack_bf16(out[4] * inv, out[5] * inv), pack_bf16(out[6] * inv, out[7] * inv));
  if (col == 0)
    put(p.c, p.lse, static_cast<long long>(b) * p.heads + h, lse_count(p),
        sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2);
}

// out += f * eight consecutive sums
__device__ __forceinline__ void add_row8(float (&out)[8], float f, const float* a) {
  const float4 a0 = reinterpret_cast<const float4*>(a)[0], a1 = reinterpret_cast<const float4*>(a)[1];
  const float v[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
  for (int e = 0; e < 8; ++e) out[e] = fmaf(f, v[e], out[e]);
}

// Beginning, ending and switching a row costs a warp about as much as a tile:
// rows count as that much longer in the shares (64 ragged sequences of up to
// 8192 keys 39 -> 30 us, the longest share no longer 13 us behind the median).
constexpr int kRowCost = 2;

// Tiles of sequence b's rows, 0 for a slot out of range or without keys, and
// its slot and length.
template <int KT>
__device__ __forceinline__ int tiles_of(const AttendParams& p, int b, int* slot, int* len) {
  *slot = p.slots != nullptr ? get(p.c, p.slots, b, p.batch) : b;
  *len = 0;
  if (*slot >= 0 && *slot < p.c.slots)
    *len = min(max(get(p.c, p.c.lengths, *slot, p.c.slots), 0), p.c.max_pages * p.c.page_size);
  return (visible_of(*len, p.window, p.sinks).count + KT - 1) / KT;
}
// What a row of that many tiles takes up in the shares.
__device__ __forceinline__ uint32_t span_of(int tiles) { return tiles > 0 ? tiles + kRowCost : 0; }

// The sequences that a block looks at together, in shared memory: four a thread
// (with one a thread, 256 ragged sequences took 71 us where these take 59).
constexpr int kSeqsPerThread = 4, kSeqs = kThreads * kSeqsPerThread;

struct Seqs {
  int len[kSeqs], tiles[kSeqs], slot[kSeqs];
  uint32_t upto[kSeqs];  // running sum of spans
  uint32_t scan[kWarps];
};

// A place in the walk: tile f of the row that has tiles [lo, hi) of the batch's,
// row rs (K / V head hk, block of heads) of sequence j of the chunk.
struct Cursor {
  uint32_t f, lo, hi;
  int j, rs, hk;
};

// CL: a cluster per row (see the head of the file).
template <int D, int NB, bool CL>
__global__ void __launch_bounds__(kThreads, DecodeCfg<D, NB>::MIN_BLOCKS)
    attend_kernel(const AttendParams p) {
  using C = DecodeCfg<D, NB>;
  constexpr int KT = C::KT, STAGES = C::STAGES;
  // in this order: join_kernel, released below, reads lengths and slots before its
  // own wait, so all that wrote them has to be done by then
  griddep_wait();
  griddep_launch_dependents();
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Seqs sq;
  const uint32_t warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2, q4 = lane & 3;  // row, and pair of columns, of the matrix fragments
  constexpr int HB = 8 * NB;               // query heads of a row
  const int rows_per_seq = p.c.heads_kv * p.head_blocks;

  // ---- the shares: tiles of every sequence, their sum and this warp's part
  // Loads the sequences from b0 on and the running sums of their spans; returns
  // the sum of all.
  auto load_seqs = [&](int b0) -> uint32_t {
    uint32_t upto[kSeqsPerThread], x = 0;
    const int j0 = threadIdx.x * kSeqsPerThread;
#pragma unroll
    for (int i = 0; i < kSeqsPerThread; ++i) {
      int n = 0, slot = -1, tiles = 0;
      if (b0 + j0 + i < p.batch) tiles = tiles_of<KT>(p, b0 + j0 + i, &slot, &n);
      sq.len[j0 + i] = n;
      sq.slot[j0 + i] = slot;
      sq.tiles[j0 + i] = tiles;
      x += span_of(tiles);
      upto[i] = x;
    }
    const uint32_t own = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    if (lane == 31) sq.scan[warp] = x;
    __syncthreads();
    uint32_t before = x - own, all = 0;
#pragma unroll
    for (uint32_t w = 0; w < kWarps; ++w) {
      if (w < warp) before += sq.scan[w];
      all += sq.scan[w];
    }
#pragma unroll
    for (int i = 0; i < kSeqsPerThread; ++i) sq.upto[j0 + i] = before + upto[i];
    __syncthreads();
    return all;
  };
  const uint32_t ring = smem_u32(smem) + warp * C::WARP;
  uint32_t* valid = reinterpret_cast<uint32_t*>(smem + C::OFF_VALID) + warp * STAGES;

  if (p.c.d < D)
    for (uint32_t x = lane; x < C::WARP / 16; x += 32) st_shared_v4(ring + 16 * x, 0u, 0u, 0u, 0u);
  __syncwarp();

  uint32_t lo = 0, blk_lo = 0, blk_hi = 0, blk0 = 0, share = 0;  // of the shares, below
  // The tiles of one warp: from `at` to `end` in steps of `step`, through the rows
  // of the sequences that begin at b0.  block_row: all of the block's warps work
  // on this one row, and their parts meet at the end.
  auto walk = [&](int b0, Cursor at, uint32_t end, uint32_t step, bool block_row) {
    auto advance = [&](Cursor& c) {  // a tile on; c.f < end afterwards or the cursor is not used
      c.f += step;
      if (c.f < c.hi || c.f >= end) return;
      c.lo = c.f = c.hi + kRowCost;
      if (c.f >= end) return;
      if (++c.rs == rows_per_seq) {
        c.rs = 0;
        do ++c.j;
        while (sq.tiles[c.j] == 0);
      }
      c.hk = p.head_blocks == 1 ? c.rs : c.rs / p.head_blocks;
      c.hi = c.lo + sq.tiles[c.j];
    };
    if (!CL && at.f >= at.hi) {  // the share begins behind a row's last tile
      at.f = at.hi - 1;
      advance(at);
    }

    // Page and row of this lane's key (lane & (KT - 1)) of the cursor's tile,
    // and the tile's K / V head.  The table cell is asked for a round before
    // copies need it, and nothing is computed from it until then.
    struct Key {
      int page, row, hk;
    };
    auto locate = [&](const Cursor& c) -> Key {
      Key r{-1, 0, c.hk};
      if (c.f >= end) return r;
      if (c.f == c.lo || c.f == at.f) {
        // a row begins: its Q into L2, a 128-byte line a lane
        const int hb = c.rs - c.hk * p.head_blocks, lines = (2 * p.c.d + 127) / 128;
        const int h = lane / lines;
        if (h < min(HB, p.group - hb * HB))
          prefetch_l2(p.q + (b0 + c.j) * p.q_batch + (c.hk * p.group + hb * HB + h) * p.q_head +
                      (lane - h * lines) * 64);
      }
      const Visible vis = visible_of(sq.len[c.j], p.window, p.sinks);
      const int u = static_cast<int>(c.f - c.lo) * KT + (lane & (KT - 1));
      if (u < vis.count) {
        const int j = vis.key(u);
        const int cell = j / p.c.page_size;
        r.row = j - cell * p.c.page_size;
        r.page = get(p.c, p.c.table, static_cast<long long>(sq.slot[c.j]) * p.c.max_pages + cell,
                     table_cells(p.c));
      }
      return r;
    };
    // copies of one tile into a stage: whole rows, 16 bytes a lane
    auto load = [&](int stage, const Key& r) {
      constexpr int CH = D / 8, RPI = 32 / CH;  // pieces of a row, rows per step
      const int c = lane % CH;
      const uint32_t kdst = ring + stage * C::STAGE, vdst = kdst + KT * C::ROW;
      const uint32_t live = __ballot_sync(0xffffffffu, r.page >= 0 && r.page < p.c.pages);
      if (lane == 0) valid[stage] = live;
      const bool col_ok = 8 * c < p.c.d;  // past d the ring holds zeros
      const __nv_bfloat16* kh = p.k + r.hk * p.c.k_head + 8 * c;
      const __nv_bfloat16* vh = p.v + r.hk * p.c.v_head + 8 * c;
      // Most tiles are one run of consecutive rows, or two (where the tile crosses
      // a page, or from the first tokens into the window): one or two places to
      // start from instead of one per row.  (With two places for every tile, d =
      // 256 took 119 us where it takes 93.)
      const int x = lane & (KT - 1);
      const int page0 = __shfl_sync(0xffffffffu, r.page, 0), row0 = __shfl_sync(0xffffffffu, r.row, 0);
      const uint32_t other = __ballot_sync(0xffffffffu, r.page != page0 || r.row != row0 + x);
      const bool all_live = live == 0xffffffffu;
      const int row_l = lane / CH;
      const __nv_bfloat16* k0 = kh + page0 * p.c.k_page + (row0 + row_l) * p.c.k_row;
      const __nv_bfloat16* v0 = vh + page0 * p.c.v_page + (row0 + row_l) * p.c.v_row;
      if (all_live && other == 0u) {
#pragma unroll
        for (int s = 0; s < KT / RPI; ++s) {
          const int row = s * RPI + row_l;
          const uint32_t dst = row * C::ROW + ((c ^ (row & 7)) << 4);
          if (!col_ok) break;
          copy16(p, kdst + dst, k0 + s * RPI * p.c.k_row, p.k, FA_EXTENT(p.ext_k));
          copy16(p, vdst + dst, v0 + s * RPI * p.c.v_row, p.v, FA_EXTENT(p.ext_v));
        }
        return;
      }
      const int cut = other ? __ffs(other) - 1 : 0;  // first row of the second run
      const int page1 = __shfl_sync(0xffffffffu, r.page, cut);
      const int row1 = __shfl_sync(0xffffffffu, r.row, cut) - cut;
      if (__all_sync(0xffffffffu, all_live && (x < cut || (r.page == page1 && r.row == row1 + x)))) {
        const __nv_bfloat16* k1 = kh + page1 * p.c.k_page + (row1 + row_l) * p.c.k_row;
        const __nv_bfloat16* v1 = vh + page1 * p.c.v_page + (row1 + row_l) * p.c.v_row;
#pragma unroll
        for (int s = 0; s < KT / RPI; ++s) {
          const int row = s * RPI + row_l;
          const uint32_t dst = row * C::ROW + ((c ^ (row & 7)) << 4);
          if (!col_ok) break;
          copy16(p, kdst + dst, (row < cut ? k0 : k1) + s * RPI * p.c.k_row, p.k, FA_EXTENT(p.ext_k));
          copy16(p, vdst + dst, (row < cut ? v0 : v1) + s * RPI * p.c.v_row, p.v, FA_EXTENT(p.ext_v));
        }
      } else {
#pragma unroll
        for (int s = 0; s < KT / RPI; ++s) {
          const int row = s * RPI + lane / CH;
          const int page = __shfl_sync(0xffffffffu, r.page, row), at_row = __shfl_sync(0xffffffffu, r.row, row);
          const bool ok = (live >> row) & 1u;
          const uint32_t dst = row * C::ROW + ((c ^ (row & 7)) << 4);
          if (!col_ok) continue;
          const __nv_bfloat16* ks = ok ? kh + page * p.c.k_page + at_row * p.c.k_row : p.k;
          const __nv_bfloat16* vs = ok ? vh + page * p.c.v_page + at_row * p.c.v_row : p.v;
          cp_async16(kdst + dst, ks, ok && FA_IN_BOUNDS(p.c.status, ks - p.k, 8, p.ext_k));
          cp_async16(vdst + dst, vs, ok && FA_IN_BOUNDS(p.c.status, vs - p.v, 8, p.ext_v));
        }
      }
    };

    Cursor fill = at;
    {
      Key ahead[STAGES - 1];
      bool ahead_live[STAGES - 1];
#pragma unroll
      for (int s = 0; s < STAGES - 1; ++s) {
        ahead_live[s] = fill.f < end;
        ahead[s] = locate(fill);
        advance(fill);
      }
#pragma unroll
      for (int s = 0; s < STAGES - 1; ++s) {
        if (ahead_live[s]) load(s, ahead[s]);
        cp_async_commit();
      }
    }
    Key next = locate(fill);

    uint32_t qb[NB][D / 16][2];  // Q as the B operand: column g is a head
    float o[NB][D / 16][4];      // O^T: rows g, g + 8 of 16 columns of V; heads 2 q4, 2 q4 + 1
    float m[NB][2], l[NB][2];    // of those heads; l: this lane's keys alone
    bool begin = true;
    int stage = 0;
    if constexpr (CL) {  // a warp without tiles takes part in the meeting all the same
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int u = 0; u < 4; ++u) o[nb][i][u] = 0.f;
        m[nb][0] = m[nb][1] = -INFINITY;
        l[nb][0] = l[nb][1] = 0.f;
      }
    }
    while (at.f < end) {
      // the next free stage was read in the previous round
      __syncwarp();
      if (fill.f < end) load(stage == 0 ? STAGES - 1 : stage - 1, next);
      cp_async_commit();
      advance(fill);
      next = locate(fill);
      const int hk = at.hk, hb = at.rs - hk * p.head_blocks;
      const int h0 = hk * p.group + hb * HB;      // first query head of the row
      const int hn = min(HB, p.group - hb * HB);  // its query heads
      const int b = b0 + at.j;
      if (begin) {
        // Q: zero past the row's heads and past d
        const __nv_bfloat16* q0 = p.q + b * p.q_batch + h0 * p.q_head;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const int h = 8 * nb + g;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int col = 16 * kk + 8 * u + 2 * q4;
              qb[nb][kk][u] = h < hn && col < p.c.d &&
                                      FA_IN_BOUNDS(p.c.status, q0 + h * p.q_head + col - p.q, 2, p.ext_q)
                                  ? *reinterpret_cast<const uint32_t*>(q0 + h * p.q_head + col)
                                  : 0u;
            }
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int u = 0; u < 4; ++u) o[nb][i][u] = 0.f;
          m[nb][0] = m[nb][1] = -INFINITY;
          l[nb][0] = l[nb][1] = 0.f;
        }
        begin = false;
      }
      cp_async_wait<STAGES - 1>();
      __syncwarp();
      const uint32_t kbase = ring + stage * C::STAGE, vbase = kbase + KT * C::ROW;
      const uint32_t live = valid[stage];
      constexpr int MT = KT / 16;  // 16-key rows of S^T
      // two sums per score, over the even and the odd steps: half the chain
      float s[MT][NB][4], s1[MT][NB][4];
#pragma unroll
      for (int kt = 0; kt < MT; ++kt)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int u = 0; u < 4; ++u) s[kt][nb][u] = s1[kt][nb][u] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int kt = 0; kt < MT; ++kt) {
          uint32_t ka[4];
          const int row = kt * 16 + (lane & 15), ch = 2 * kk + (lane >> 4);
          ldsm_x4(kbase + row * C::ROW + ((ch ^ (row & 7)) << 4), ka);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            mma16816(kk & 1 ? s1[kt][nb] : s[kt][nb], ka, qb[nb][kk][0], qb[nb][kk][1]);
        }
#pragma unroll
      for (int kt = 0; kt < MT; ++kt)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int u = 0; u < 4; ++u) s[kt][nb][u] += s1[kt][nb][u];
      constexpr uint32_t kAll = KT == 32 ? 0xffffffffu : (1u << (KT & 31)) - 1u;
      if ((live & kAll) != kAll) {
#pragma unroll
        for (int kt = 0; kt < MT; ++kt)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int u = 0; u < 4; ++u)
              s[kt][nb][u] = (live >> (16 * kt + g + 8 * (u >> 1))) & 1u ? s[kt][nb][u] : -INFINITY;
      }
      // Online softmax over the tile's keys, per head of this lane's pair; P is
      // rounded to bf16 for the second product, as in the other attention
      // kernels (V is bf16, and both operands have one type: at most 2^-8 of each weight,
      // less than the rounding of O itself once a row has a few keys), and turned
      // from rows of keys to columns (the B operand); the row sum keeps the
      // unrounded values
      uint32_t pb[NB][MT][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float alpha[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float mx = -INFINITY;
#pragma unroll
          for (int kt = 0; kt < MT; ++kt) mx = fmax3(mx, s[kt][nb][u], s[kt][nb][u + 2]);
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
          const float m_new = fmaxf(m[nb][u], mx * p.scale_log2);
          const float ref = m_new == -INFINITY ? 0.f : m_new;
          alpha[u] = fast_exp2(m[nb][u] - ref);
          m[nb][u] = m_new;
          float sum = 0.f;
#pragma unroll
          for (int kt = 0; kt < MT; ++kt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float e = fast_exp2(fmaf(s[kt][nb][u + 2 * r], p.scale_log2, -ref));
              s[kt][nb][u + 2 * r] = e;
              sum += e;
            }
          l[nb][u] = l[nb][u] * alpha[u] + sum;
        }
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int u = 0; u < 4; ++u) o[nb][i][u] *= alpha[u & 1];
        }
#pragma unroll
        for (int kt = 0; kt < MT; ++kt)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            pb[nb][kt][r] = transpose8x8(pack_bf16(s[kt][nb][2 * r], s[kt][nb][2 * r + 1]));
      }
#pragma unroll
      for (int kt = 0; kt < MT; ++kt)
#pragma unroll
        for (int dd = 0; dd < D / 16; ++dd) {
          uint32_t va[4];
          const int row = kt * 16 + (lane & 7) + (lane >> 4) * 8, ch = 2 * dd + ((lane >> 3) & 1);
          ldsm_x4_trans(vbase + row * C::ROW + ((ch ^ (row & 7)) << 4), va);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mma16816(o[nb][dd], va, pb[nb][kt][0], pb[nb][kt][1]);
        }
      stage = stage + 1 == STAGES ? 0 : stage + 1;

      const uint32_t f1 = at.f + 1;
      if (block_row) {
        if (at.f + step < end) {
          advance(at);
          continue;
        }
        break;  // the warps' parts of this row meet below
      } else if (f1 == at.hi || f1 == end) {
        // the row ends, or the share: the whole row goes to O and LSE, a part of
        // it to the share's partial results, index 1 where the row begins in
        // this share, 0 where it goes on
        const bool begins = at.lo >= lo, whole = begins && f1 == at.hi;
        const long long pr = (2ll * share + (begins ? 1 : 0)) * 16;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float inv[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            l[nb][u] = sum_rows(l[nb][u]);
            inv[u] = l[nb][u] == 0.f ? 0.f : 1.f / l[nb][u];
            const int h = 8 * nb + 2 * q4 + u;
            if (g == 0 && h < hn) {
              if (whole)
                put(p.c, p.lse, static_cast<long long>(b) * p.heads + h0 + h, lse_count(p),
                    l[nb][u] == 0.f ? -INFINITY : (m[nb][u] + log2f(l[nb][u])) * kLn2);
              else
                put(p.c, p.part_stat, pr + h, part_rows(p), make_float2(m[nb][u], l[nb][u]));
            }
          }
          if (whole) {
            // pairs of columns of V for head g, out of pairs of heads
            __nv_bfloat16* dst = p.o + b * p.o_batch + (h0 + 8 * nb + g) * p.o_head + 2 * q4;
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const uint32_t x =
                    transpose8x8(pack_bf16(o[nb][i][2 * r] * inv[0], o[nb][i][2 * r + 1] * inv[1]));
                const int col = 16 * i + 8 * r;
                if (8 * nb + g < hn && col < p.c.d && FA_IN_BOUNDS(p.c.status, dst + col - p.o, 2, p.ext_o))
                  *reinterpret_cast<uint32_t*>(dst + col) = x;
              }
          } else {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int h = 8 * nb + 2 * q4 + u;
              float* dst = p.part_acc + (pr + h) * D + g;
              if (h < hn && FA_IN_BOUNDS(p.c.status, pr + h, 1, part_rows(p)))
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                  dst[16 * i] = o[nb][i][u];
                  dst[16 * i + 8] = o[nb][i][2 + u];
                }
            }
          }
        }
        begin = true;
      }
      advance(at);
    }
    cp_async_wait<0>();
    if (block_row) {
      // one partial result for the block, in its first share's place: a quarter
      // of what the joining kernel would read
      const int hk = at.hk, hb = at.rs - hk * p.head_blocks;
      const int hn = min(HB, p.group - hb * HB);
      constexpr int LD = D + 4;  // (a warp's eight heads in different banks)
      __syncthreads();
      float2* stat = reinterpret_cast<float2*>(smem);  // [warp][HB], then [warp][HB][LD] sums
      float* acc = reinterpret_cast<float*>(smem + kWarps * HB * sizeof(float2));
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int h = warp * HB + 8 * nb + 2 * q4 + u;
          const float sum = sum_rows(l[nb][u]);
          if (g == 0) stat[h] = make_float2(m[nb][u], sum);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            acc[h * LD + 16 * i + g] = o[nb][i][u];
            acc[h * LD + 16 * i + 8 + g] = o[nb][i][2 + u];
          }
        }
      float2* stat2 = reinterpret_cast<float2*>(acc + kWarps * HB * LD);  // CL: [HB], then [HB][D]
      float* acc2 = reinterpret_cast<float*>(stat2 + HB);
      __syncthreads();
      const bool begins = at.lo >= blk_lo, whole = begins && at.hi == blk_hi;
      for (int x = threadIdx.x; x < hn * (D / 8); x += kThreads) {
        const int r = x / (D / 8), col = 8 * (x % (D / 8));
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, stat[w * HB + r].x);
        const float ref = mm == -INFINITY ? 0.f : mm;
        float rs = 0.f, out[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) out[e] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float2 st = stat[w * HB + r];
          const float f = fast_exp2(st.x - ref);
          rs += f * st.y;
          add_row8(out, f, acc + (w * HB + r) * LD + col);
        }
        if constexpr (CL) {  // to the cluster: sums and statistics of this block
          float4* a = reinterpret_cast<float4*>(acc2 + r * D + col);
          a[0] = make_float4(out[0], out[1], out[2], out[3]);
          a[1] = make_float4(out[4], out[5], out[6], out[7]);
          if (col == 0) stat2[r] = make_float2(mm, rs);
          continue;
        }
        if (whole) {
          if (col < p.c.d) write_row(p, b0 + at.j, hk * p.group + hb * HB + r, col, mm, rs, out);
          continue;
        }
        const long long row = (2ll * blk0 + (begins ? 1 : 0)) * 16 + r;
        if (!FA_IN_BOUNDS(p.c.status, row, 1, part_rows(p))) continue;
        float4* a = reinterpret_cast<float4*>(p.part_acc + row * D + col);
        a[0] = make_float4(out[0], out[1], out[2], out[3]);
        a[1] = make_float4(out[4], out[5], out[6], out[7]);
        if (col == 0) {
          p.part_stat[row] = make_float2(mm, rs);
        }
      }
      if constexpr (CL) {
        cluster_sync();
        const uint32_t cs = p.cluster, rank = blockIdx.x % cs;
        for (uint32_t x = rank * kThreads + threadIdx.x; x < hn * (D / 8); x += cs * kThreads) {
          const int r = x / (D / 8), col = 8 * (x % (D / 8));
          if (col >= p.c.d) continue;
          float2 st[8];
          float mm = -INFINITY, rs = 0.f, out[8];
#pragma unroll
          for (uint32_t c = 0; c < 8; ++c) {
            st[c] = c < cs ? cluster_load2(stat2 + r, c) : make_float2(-INFINITY, 0.f);
            mm = fmaxf(mm, st[c].x);
          }
          const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll
          for (int e = 0; e < 8; ++e) out[e] = 0.f;
#pragma unroll
          for (uint32_t c = 0; c < 8; ++c) {
            if (c >= cs) break;
            const float f = fast_exp2(st[c].x - ref);
            rs += f * st[c].y;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 v = cluster_load2(acc2 + r * D + col + 2 * e, c);
              out[2 * e] = fmaf(f, v.x, out[2 * e]);
              out[2 * e + 1] = fmaf(f, v.y, out[2 * e + 1]);
            }
          }
          write_row(p, b0, hk * p.group + hb * HB + r, col, mm, rs, out);
        }
        cluster_sync();  // nobody leaves while the others still read
      }
      if (p.batch > kSeqs) {
        __syncthreads();
        if (p.c.d < D)  // the ring held fp32 sums
          for (uint32_t x = lane; x < C::WARP / 16; x += 32) st_shared_v4(ring + 16 * x, 0u, 0u, 0u, 0u);
        __syncwarp();
      }
    }
  };

  if constexpr (CL) {
    const int cs = p.cluster, rank = blockIdx.x % cs, row = blockIdx.x / cs;
    const int b = row / rows_per_seq, rs = row - b * rows_per_seq;
    int slot, len;
    const int tiles = tiles_of<KT>(p, b, &slot, &len);
    if (threadIdx.x == 0) {
      sq.len[0] = len;
      sq.slot[0] = slot;
      sq.tiles[0] = tiles;
    }
    __syncthreads();
    const uint32_t n = tiles;
    walk(b, Cursor{rank * kWarps + warp, 0, n, 0, rs, rs / p.head_blocks}, n, cs * kWarps, true);
    return;
  }

  uint32_t sum = 0, part = 0;  // spans of one row per sequence
  for (int b0 = 0; b0 < p.batch; b0 += kSeqs) {
    part = load_seqs(b0);
    sum += part;
  }
  const uint32_t W = sum * rows_per_seq;
  // (down to one tile each: shares of at least four took 10.8 us for one
  // sequence of 500 keys where these take 8.7, joining included)
  const uint32_t grid = gridDim.x;
  const Shares sh(W, min(max(W, 1u), static_cast<uint32_t>(p.shares)));
  // few shares: one or two warps of a block, so that they spread over the SMs
  const uint32_t active = sh.n <= grid ? 1 : sh.n <= 2 * grid ? 2 : kWarps;
  blk0 = blockIdx.x * active;
  share = warp < active ? blk0 + warp : sh.n;
  lo = share < sh.n ? sh.begin(share) : W;
  const uint32_t hi = share < sh.n ? sh.begin(share + 1) : W;
  // the block's own range, where all its warps have a share
  const bool full = active == kWarps && blk0 + kWarps <= sh.n;
  blk_lo = full ? sh.begin(blk0) : 0;
  blk_hi = full ? sh.begin(blk0 + kWarps) : 0;

  // the sequence of tile f of the chunk that begins at tile lo with sequence b0:
  // the first whose running sum passes it
  auto seq_at = [&](uint32_t f, uint32_t chunk, int b0) -> int {
    const uint32_t fs = (f - chunk) / rows_per_seq;
    int a = 0, z = min(kSeqs, p.batch - b0) - 1;
    while (a < z) {
      const int mid = (a + z) / 2;
      if (sq.upto[mid] > fs) z = mid;
      else a = mid + 1;
    }
    return a;
  };
  // rows without keys belong to no share: the last block's warps write theirs
  auto write_empty = [&](int b0) {
    if (blockIdx.x != grid - 1) return;
    for (int i = 0; i < kSeqsPerThread; ++i) {
      const int j = threadIdx.x * kSeqsPerThread + i;
      uint32_t none = __ballot_sync(0xffffffffu, b0 + j < p.batch && sq.tiles[j] == 0);
      for (; none != 0u; none &= none - 1u) {
        const int b = b0 + static_cast<int>(32 * warp + __ffs(none) - 1) * kSeqsPerThread + i;
        for (int x = lane; x < p.heads * (p.c.d / 8); x += 32) {
          const int h = x / (p.c.d / 8), col = 8 * (x % (p.c.d / 8));
          const long long at = b * p.o_batch + h * p.o_head + col;
          if (FA_IN_BOUNDS(p.c.status, at, 8, p.ext_o))
            *reinterpret_cast<uint4*>(p.o + at) = make_uint4(0u, 0u, 0u, 0u);
          if (col == 0)
            put(p.c, p.lse, static_cast<long long>(b) * p.heads + h, lse_count(p), -INFINITY);
        }
      }
    }
  };

  // The sequences that the block looks at begin with the one of its first share
  // (begun at a multiple of kSeqs instead, the warps of one block that lay on both
  // sides of such a place waited for one another and ended last, twice as late)
  const uint32_t blk_from = blk0 < sh.n ? sh.begin(blk0) : W;
  const uint32_t blk_end = blk0 < sh.n ? sh.begin(min(blk0 + active, sh.n)) : W;
  uint32_t chunk_lo = 0;  // tile at which the chunk of sequences begins
  int b_from = 0;
  if (p.batch > kSeqs) {
    uint32_t from_lo = W, before = 0;  // spans before the chunk
    const bool tells = p.spans != nullptr && blockIdx.x == 0;
    if (tells && threadIdx.x == 0) put(p.c, p.spans, p.batch, p.batch + 1ll, sum);
    for (int b0 = 0; b0 < p.batch; b0 += kSeqs) {
      part = load_seqs(b0);
      write_empty(b0);
      if (tells)
        for (int j = threadIdx.x; j < kSeqs && b0 + j < p.batch; j += kThreads)
          put(p.c, p.spans, b0 + j, p.batch + 1ll, before + sq.upto[j] - span_of(sq.tiles[j]));
      before += part;
      const uint32_t next_lo = chunk_lo + part * rows_per_seq;
      if (blk_from >= chunk_lo && blk_from < next_lo) {
        const int j = seq_at(blk_from, chunk_lo, b0);
        b_from = b0 + j;
        from_lo = chunk_lo + (sq.upto[j] - span_of(sq.tiles[j])) * rows_per_seq;
      }
      chunk_lo = next_lo;
      __syncthreads();  // the next chunk overwrites the sequences
    }
    chunk_lo = from_lo;
  } else {
    write_empty(0);
  }
  for (int b0 = b_from; b0 < p.batch && chunk_lo < blk_end; b0 += kSeqs) {
    if (p.batch > kSeqs) part = load_seqs(b0);  // else they are still there
    const uint32_t chunk_hi = chunk_lo + part * rows_per_seq;
    const uint32_t from = max(lo, chunk_lo);
    uint32_t end = min(hi, chunk_hi), step = 1;
    if (from < end) {
      // the row of tile `from`
      Cursor at;
      {
        const int a = seq_at(from, chunk_lo, b0);
        at.j = a;
        const uint32_t span = span_of(sq.tiles[a]);
        const uint32_t seq_lo = chunk_lo + (sq.upto[a] - span) * rows_per_seq;
        at.rs = (from - seq_lo) / span;
        at.hk = at.rs / p.head_blocks;
        at.lo = seq_lo + at.rs * span;
        at.hi = at.lo + sq.tiles[a];
        at.f = from;
      }
      // Where the block's four shares lie in one row its warps take turns, so that
      // they read neighbouring rows at a time, and their parts meet at the end.
      const bool block_row = full && at.lo <= blk_lo && at.hi >= blk_hi;
      if (block_row) {
        at.f = blk_lo + warp;
        end = blk_hi;
        step = kWarps;
      }
      walk(b0, at, end, step, block_row);
    }
    chunk_lo = chunk_hi;
    if (p.batch > kSeqs) __syncthreads();  // the next chunk overwrites the sequences
  }
}

// Joins the parts of rows that were cut: a block per (row, kJoinHeads of its query
// heads), one head where there are few rows, which then have many parts (one row
// of 100000 keys, 8 heads: 43 us with four heads a block, 26 with one).  First
// the maximum and row sum of all parts' statistics at once, then the weighted
// sums: D / 8 threads over a head's columns, the others over the parts, whose
// loads wait for nothing (with the maximum carried from part to part, 16 rows of
// 37 parts at d = 256 took 13 us).  Which rows were cut, and where, follows from
// the lengths alone, so all of that happens before the wait for the attention
// kernel (which starts its dependents only once the kernels before it are done):
// small enough to be resident beside it, a block goes on at once when it ends.
// Above kSeqs sequences the attention kernel's first block has written their
// running sums instead: a block that adds up the whole batch, once per row, is
// quadratic (8 K / V heads of 64: 1000 sequences of 100 keys 82 us, 77 with the
// sums; 16000 of 60 keys 2515 and 762; 60000 of 40 keys 28700 and 2720).
constexpr int kJoinThreads = 256;

template <int D, int KT, int kJoinHeads>
__global__ void __launch_bounds__(kJoinThreads, 5) join_kernel(const AttendParams p) {
  constexpr int TPR = D / 8, GROUPS = kJoinThreads / (TPR * kJoinHeads), kJoinWarps = kJoinThreads / 32;
  __shared__ uint2 seqs[kJoinWarps];
  __shared__ float2 red[kJoinWarps][kJoinHeads];
  __shared__ __align__(16) float acc[GROUPS][kJoinHeads][D];
  const int rows_per_seq = p.c.heads_kv * p.head_blocks;
  const int b = blockIdx.x / rows_per_seq, rs = blockIdx.x - b * rows_per_seq;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint2 sum = make_uint2(0u, 0u);  // spans of all sequences, and of those before b
  int slot, len;
  const int tiles = tiles_of<KT>(p, b, &slot, &len);
  if (p.spans == nullptr) {
#pragma unroll 4
    for (int i = threadIdx.x; i < p.batch; i += kJoinThreads) {
      int s, n;
      const uint32_t span = span_of(tiles_of<KT>(p, i, &s, &n));
      sum.x += span;
      sum.y += i < b ? span : 0u;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      sum.x += __shfl_xor_sync(0xffffffffu, sum.x, o);
      sum.y += __shfl_xor_sync(0xffffffffu, sum.y, o);
    }
    if (lane == 0) seqs[warp] = sum;
    __syncthreads();
    sum = make_uint2(0u, 0u);
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      sum.x += seqs[w].x;
      sum.y += seqs[w].y;
    }
  }
  griddep_launch_dependents();
  // one block waits whatever its row: this grid must not be done before the
  // attention kernel is, or a kernel behind it could start beside that one
  if (p.spans != nullptr || (blockIdx.x == 0 && blockIdx.y == 0)) griddep_wait();
  if (tiles == 0) return;
  if (p.spans != nullptr)
    sum = make_uint2(get(p.c, p.spans, p.batch, p.batch + 1ll), get(p.c, p.spans, b, p.batch + 1ll));
  const uint32_t W = sum.x * rows_per_seq;
  const Shares sh(W, min(max(W, 1u), static_cast<uint32_t>(p.shares)));
  const uint32_t lo = sum.y * rows_per_seq + rs * span_of(tiles), hi = lo + tiles;
  const uint32_t c0 = sh.holding(lo), c1 = sh.holding(hi - 1);
  if (c0 == c1) return;  // written by the attention kernel
  // The row's parts in order: shares c0 .. first - 1 one by one, from there to
  // `last` the first share of every block that lies in the row, then one by one
  // again to c1.
  const uint32_t active = sh.n <= p.grid ? 1 : sh.n <= 2 * p.grid ? 2 : kWarps;
  uint32_t first = (c0 + kWarps - 1) / kWarps * kWarps, last = c1 / kWarps * kWarps;
  if (c0 % kWarps == 0 && lo != sh.begin(c0)) first += kWarps;
  if ((c1 + 1) % kWarps == 0 && hi == sh.begin(c1 + 1)) last += kWarps;
  if (active != kWarps || first >= last) first = last = c1 + 1;
  const uint32_t n1 = first - c0, n2 = n1 + (last - first) / kWarps;
  const uint32_t parts = n2 + c1 + 1 - last;
  if (parts == 1) return;  // one block's shares were the whole row: written already
  auto share_at = [&](uint32_t i) {
    return i < n1 ? c0 + i : i < n2 ? first + (i - n1) * kWarps : last + (i - n2);
  };
  const int hk = rs / p.head_blocks, hb = rs - hk * p.head_blocks;
  const int HB = p.block_heads;
  const int hn = min(HB, p.group - hb * HB) - blockIdx.y * kJoinHeads;  // this block's heads, and more
  // partial result of share c for head r of this block (see attend_kernel)
  auto row_of = [&](uint32_t c, int r) {
    return (2ll * c + (c == c0 ? 1 : 0)) * 16 + blockIdx.y * kJoinHeads + r;
  };
  griddep_wait();

  // statistics: thread = (head threadIdx.x % kJoinHeads, every (kJoinThreads /
  // kJoinHeads)-th part from threadIdx.x / kJoinHeads on)
  const int hr = threadIdx.x % kJoinHeads;
  float m = -INFINITY, l = 0.f;
  if (hr < hn)
    for (uint32_t i = threadIdx.x / kJoinHeads; i < parts; i += kJoinThreads / kJoinHeads) {
      const float2 st = get(p.c, p.part_stat, row_of(share_at(i), hr), part_rows(p));
      const float mm = fmaxf(m, st.x), ref = mm == -INFINITY ? 0.f : mm;
      l = l * fast_exp2(m - ref) + st.y * fast_exp2(st.x - ref);
      m = mm;
    }
#pragma unroll
  for (int o = kJoinHeads; o < 32; o <<= 1) {  // in a fixed order
    const float m1 = __shfl_xor_sync(0xffffffffu, m, o), l1 = __shfl_xor_sync(0xffffffffu, l, o);
    const float mm = fmaxf(m, m1), ref = mm == -INFINITY ? 0.f : mm;
    l = l * fast_exp2(m - ref) + l1 * fast_exp2(m1 - ref);
    m = mm;
  }
  if (lane < kJoinHeads) red[warp][lane] = make_float2(m, l);
  __syncthreads();
  const int col = 8 * (threadIdx.x % TPR), x = threadIdx.x / TPR;
  const int r = x % kJoinHeads, group = x / kJoinHeads;
  m = -INFINITY;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, red[w][r].x);
  const float ref = m == -INFINITY ? 0.f : m;
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) l += red[w][r].y * fast_exp2(red[w][r].x - ref);
  float out[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) out[e] = 0.f;
  if (r < hn) {
#pragma unroll 4
    for (uint32_t i = group; i < parts; i += GROUPS) {
      const long long row = row_of(share_at(i), r);
      if (!FA_IN_BOUNDS(p.c.status, row, 1, part_rows(p))) continue;
      add_row8(out, fast_exp2(p.part_stat[row].x - ref), p.part_acc + row * D + col);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[group][r][col + e] = out[e];
  __syncthreads();
  if (group != 0 || col >= p.c.d || r >= hn) return;
#pragma unroll
  for (int w = 1; w < GROUPS; ++w) add_row8(out, 1.f, &acc[w][r][col]);
  write_row(p, b, hk * p.group + hb * HB + blockIdx.y * kJoinHeads + r, col, m, l, out);
}

// Grid and workspace of a call, from what the host knows: the longest that a
// sequence may see.  One block per resident slot of the GPU, fewer where the
// batch cannot have as many tiles; no row can be cut, and none has to be
// joined, where none can have more than one tile.
struct Plan {
  long long tiles;  // at most, of the whole batch
  int cluster;      // > 0: a cluster of that many blocks per row
  long long grid;
  bool cut;
  int join_heads;   // of a joining block: one where few rows are joined, from many parts each
  size_t off_acc, off_spans, bytes;
};

template <int NB>
void sizes_of(int D, int* KT, int* per_sm) {
  *KT = D == 64 ? DecodeCfg<64, NB>::KT : D == 128 ? DecodeCfg<128, NB>::KT : DecodeCfg<256, NB>::KT;
  *per_sm = D == 64    ? DecodeCfg<64, NB>::MIN_BLOCKS
            : D == 128 ? DecodeCfg<128, NB>::MIN_BLOCKS
                       : DecodeCfg<256, NB>::MIN_BLOCKS;
}

// Query heads of a row for a group of G per K / V head.
int block_heads_of(int G) { return G <= 8 ? 8 : 16; }

Plan plan_of(const Cache& c, int batch, int heads, int window, int sinks) {
  const int D = c.d <= 64 ? 64 : c.d <= 128 ? 128 : 256;
  const int G = heads / c.heads_kv, HB = block_heads_of(G);
  int KT = 0, per_sm = 0;
  if (HB == 8) sizes_of<1>(D, &KT, &per_sm);
  else sizes_of<2>(D, &KT, &per_sm);
  long long most = static_cast<long long>(c.max_pages) * c.page_size;
  if (window > 0 && static_cast<long long>(window) + sinks < most) most = static_cast<long long>(window) + sinks;
  const long long tiles = (most + KT - 1) / KT;
  const long long rows = static_cast<long long>(batch) * c.heads_kv * ((G + HB - 1) / HB);
  Plan p;
  p.tiles = rows * (tiles + kRowCost);
  // A cluster per row where all rows' clusters are resident at once (of clusters
  // of 8 at one block per SM, 12 are and 16 are not: 7.8 and 14.1 us at d = 256, 512
  // keys) and the longest row that the table has room for gives a warp at most
  // four tiles.  A cluster's time is that of its longest row, equal shares' that
  // of the mean one and 3 us more.  Clusters and shares, d = 128, groups of 4, at 1, 4,
  // 8 and 32 tiles a warp: 32 sequences over 4 K / V heads, all as long as the
  // table, 5.7 / 8.9, 9.5 / 11.9, 14.5 / 16.2 and 49 / 51 us; lengths spread over
  // their logarithm 5.8 / 8.8, 8.8 / 9.9, 13.9 / 10.9 and 41 / 15; one sequence, as
  // long as the table, 6.6 / 7.4, 9.5 / 9.9, 14.0 / 8.7 and 41 / 13, a quarter of it
  // 6.3 / 6.9, 6.4 / 7.6, 7.4 / 8.4 and 14 / 8.7.
  auto resident = [&](int blocks) { return blocks == 8 && per_sm == 1 ? 96ll : 128ll * per_sm; };
  int cs = 8;
  while (cs > 1 && rows * cs > resident(cs)) cs /= 2;
  while (cs > 1 && tiles <= cs / 2 * kWarps) cs /= 2;  // no warps without tiles
  p.cluster = rows * cs <= resident(cs) && tiles <= 4ll * cs * kWarps ? cs : 0;
  p.grid = p.cluster > 0                  ? rows * p.cluster
           : p.tiles < 148ll * per_sm ? p.tiles
                                      : 148ll * per_sm;
  p.cut = p.cluster == 0 && tiles > 1;
  p.join_heads = rows * HB <= 4 * 148 ? 1 : 4;
  const size_t parts = static_cast<size_t>(p.grid) * kWarps * 2 * 16;
  p.off_acc = parts * sizeof(float2);
  p.off_spans = p.off_acc + parts * D * sizeof(float);
  p.bytes = !p.cut          ? 0
            : batch > kSeqs ? p.off_spans + (static_cast<size_t>(batch) + 1) * sizeof(uint32_t)
                            : p.off_spans;
  return p;
}

template <int D, int KT, int JH>
cudaError_t launch_join(const AttendParams& p, cudaStream_t stream) {
  const int heads = p.group < p.block_heads ? p.group : p.block_heads;  // of a row
  return launch_overlapped(join_kernel<D, KT, JH>,
                           dim3(static_cast<unsigned>(p.batch * p.c.heads_kv * p.head_blocks),
                                static_cast<unsigned>((heads + JH - 1) / JH)),
                           dim3(kJoinThreads), 0, stream, p);
}

template <int D, int NB>
cudaError_t launch_attend(const AttendParams& p, void* workspace, cudaStream_t stream) {
  using C = DecodeCfg<D, NB>;
  static_assert(kWarps * 8 * NB * (8 + (D + 4) * 4) <= C::OFF_VALID, "a block's parts fit the ring");
  auto kern = attend_kernel<D, NB, false>;
  auto kern_cl = attend_kernel<D, NB, true>;
  static_assert(kWarps * 8 * NB * (8 + (D + 4) * 4) + 8 * NB * (8 + D * 4) <= C::OFF_VALID,
                "and the cluster's");
  static OncePerContext prepared;
  const cudaError_t e = prepared.run([&]() -> cudaError_t {
    const cudaError_t first = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(C::SMEM));
    if (first != cudaSuccess) return first;
    return cudaFuncSetAttribute(kern_cl, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(C::SMEM));
  });
  if (e != cudaSuccess) return e;
  const Plan plan = plan_of(p.c, p.batch, p.heads, p.window, p.sinks);
  AttendParams a = p;
  a.grid = static_cast<uint32_t>(plan.grid);
  a.shares = static_cast<int>(plan.grid) * kWarps;
  a.cluster = plan.cluster;
  if (plan.cluster > 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(plan.grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {static_cast<unsigned>(plan.cluster), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern_cl, a);
  }
  if (plan.cut) {
    char* ws = static_cast<char*>(workspace);
    a.part_stat = reinterpret_cast<float2*>(ws);
    a.part_acc = reinterpret_cast<float*>(ws + plan.off_acc);
    if (p.batch > kSeqs) a.spans = reinterpret_cast<uint32_t*>(ws + plan.off_spans);
  }
  cudaError_t r = launch_overlapped(kern, dim3(static_cast<unsigned>(plan.grid)), dim3(kThreads), C::SMEM,
                                    stream, a);
  if (r == cudaSuccess && plan.cut)
    r = plan.join_heads == 1 ? launch_join<D, C::KT, 1>(a, stream) : launch_join<D, C::KT, 4>(a, stream);
  return r;
}

}  // namespace
}  // namespace fa

extern "C" {

size_t fa_cache_attend_workspace_size(const fa_cache_t* cache, int batch, int heads, int window,
                                      int sinks) {
  fa::Cache c;
  if (fa::cache_resolve(cache, false, &c) != FA_OK || batch < 1 || heads < 1 || heads % c.heads_kv ||
      window < 0 || sinks < 0)
    return 0;
  return fa::plan_of(c, batch, heads, window, sinks).bytes;
}

fa_status_t fa_cache_attend(const fa_cache_t* cache, int layer, const void* q, void* o, float* lse,
                            int64_t q_batch, int64_t q_head, int64_t o_batch, int64_t o_head,
                            const int32_t* slots, int batch, int heads, float softmax_scale,
                            int window, int sinks, void* workspace, size_t workspace_bytes,
                            void* stream) {
  fa::AttendParams p;
  const fa_status_t st = fa::cache_resolve(cache, false, &p.c);
  if (st != FA_OK) return st;
  if (layer < 0 || layer >= p.c.layers || batch < 0 || heads < 1 || heads % p.c.heads_kv != 0 ||
      window < 0 || sinks < 0)
    return FA_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f) || !(softmax_scale < INFINITY)) return FA_ERR_INVALID_ARG;
  if (!fa::cache_stride_ok(q_batch, 1) || !fa::cache_stride_ok(q_head, 1) ||
      !fa::cache_stride_ok(o_batch, batch) || !fa::cache_stride_ok(o_head, heads))
    return FA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(slots) & 3u) != 0) return FA_ERR_INVALID_ARG;
  if (batch == 0) return FA_OK;
  if (!fa::cache_aligned(q, 16) || !fa::cache_aligned(o, 16) || !fa::cache_aligned(lse, 4))
    return FA_ERR_INVALID_ARG;
  if (heads > 65535 || static_cast<int64_t>(batch) * heads > 0x7FFFFFFF) return FA_ERR_UNSUPPORTED;
  const fa::Plan plan = fa::plan_of(p.c, batch, heads, window, sinks);
  if (plan.tiles > 0xFFFFFFFFll - 65536) return FA_ERR_UNSUPPORTED;  // 32-bit counts in the kernels
  const size_t need = plan.bytes;
  if (need > 0 && (!fa::cache_aligned(workspace, 256) || workspace_bytes < need)) return FA_ERR_WORKSPACE;
  p.k = static_cast<const __nv_bfloat16*>(p.c.k) + layer * p.c.k_layer;
  p.v = static_cast<const __nv_bfloat16*>(p.c.v) + layer * p.c.v_layer;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.q_batch = q_batch;
  p.q_head = q_head;
  p.o_batch = o_batch;
  p.o_head = o_head;
  p.slots = slots;
  p.batch = batch;
  p.heads = heads;
  p.group = heads / p.c.heads_kv;
  p.block_heads = fa::block_heads_of(p.group);
  p.head_blocks = (p.group + p.block_heads - 1) / p.block_heads;
  p.scale_log2 = static_cast<float>(static_cast<double>(softmax_scale) * fa::kLog2e);
  p.window = window;
  p.sinks = sinks;
  p.part_stat = nullptr;
  p.part_acc = nullptr;
  p.spans = nullptr;
#ifdef FA_DEBUG_BOUNDS
  p.ext_k = p.c.ext_k - layer * p.c.k_layer;
  p.ext_v = p.c.ext_v - layer * p.c.v_layer;
  p.ext_q = (batch - 1) * q_batch + (heads - 1) * q_head + p.c.d;
  p.ext_o = (batch - 1) * o_batch + (heads - 1) * o_head + p.c.d;
#endif
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto launch = p.block_heads == 8 ? (p.c.d <= 64    ? fa::launch_attend<64, 1>
                                      : p.c.d <= 128 ? fa::launch_attend<128, 1>
                                                     : fa::launch_attend<256, 1>)
                                   : (p.c.d <= 64    ? fa::launch_attend<64, 2>
                                      : p.c.d <= 128 ? fa::launch_attend<128, 2>
                                                     : fa::launch_attend<256, 2>);
  const cudaError_t e = launch(p, workspace, s);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
