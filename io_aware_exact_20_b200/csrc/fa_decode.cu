// Attention of one new token per sequence over the paged key / value cache.
//
// Per (sequence, K / V head) the group's query heads (up to 16 at a time)
// attend the visible keys in one pass: S = Q K^T, the running row maximum and
// sum of the online softmax, O += P V.  Every K / V row is read once from
// memory and serves the whole group, 2 G operations per byte, so the kernel is
// bound by memory bandwidth as long as the arithmetic keeps out of the way:
// the products run on warp-level bf16 matrix instructions (m16n8k16; the 16
// rows are the group's heads, so a 128-row tcgen05 tile would be 7/8 or more
// padding and would need the scores to leave TMEM for one row in eight), and
// every warp works on its own tiles of KT keys with its own ring of
// asynchronous copies, so that no warp waits for another before the end.
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
  int head_blocks;   // blocks of up to 16 query heads per K / V head
  float scale_log2;  // softmax_scale * log2(e)
  int window, sinks;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  const int bytes = live ? 16 : 0;  // 0: sixteen zero bytes, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
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

constexpr int kWarps = 4;

template <int D>
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

template <int D>
__global__ void __launch_bounds__(kWarps * 32, DecodeCfg<D>::MIN_BLOCKS)
    attend_kernel(const AttendParams p) {
  using C = DecodeCfg<D>;
  constexpr int KT = C::KT, STAGES = C::STAGES;
  griddep_wait();
  griddep_launch_dependents();
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q4 = lane & 3;  // row and column group of the matrix fragments

  // this block's sequence, K / V head and block of query heads
  int unit = blockIdx.x;
  const int hb = unit % p.head_blocks;
  unit /= p.head_blocks;
  const int hk = unit % p.c.heads_kv;
  const int b = unit / p.c.heads_kv;
  const int h0 = hk * p.group + hb * 16;               // first query head
  const int hn = min(16, p.group - hb * 16);           // query heads
  const int slot = p.slots != nullptr ? p.slots[b] : b;
  int n = 0;
  if (slot >= 0 && slot < p.c.slots)
    n = min(max(p.c.lengths[slot], 0), p.c.max_pages * p.c.page_size);
  const Visible vis = visible_of(n, p.window, p.sinks);
  const int tiles = (vis.count + KT - 1) / KT;
  const int32_t* pages = p.c.table + static_cast<long long>(slot) * p.c.max_pages;

  // Q as the A operand: rows g and g + 8, zero past the block's heads and past d
  uint32_t qa[D / 16][4];
  {
    const __nv_bfloat16* q0 = p.q + b * p.q_batch + h0 * p.q_head;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int r = g + 8 * (u & 1), col = 16 * kk + 8 * (u >> 1) + 2 * q4;
        qa[kk][u] = r < hn && col < p.c.d
                        ? *reinterpret_cast<const uint32_t*>(q0 + r * p.q_head + col)
                        : 0u;
      }
  }

  const uint32_t ring = smem_u32(smem) + warp * C::WARP;
  uint32_t* valid = reinterpret_cast<uint32_t*>(smem + C::OFF_VALID) + warp * STAGES;

  // K and V element offsets of this lane's key of a tile (lane & (KT - 1)), -1: none
  struct Row {
    long long k, v;
    bool live;
  };
  auto locate = [&](int tile) -> Row {
    Row r{0, 0, false};
    const int u = tile * KT + (lane & (KT - 1));
    if (u < vis.count) {
      const int j = vis.key(u);
      const int cell = j / p.c.page_size;
      const int page = pages[cell];
      if (page >= 0 && page < p.c.pages) {
        const int row = j - cell * p.c.page_size;
        r.k = page * p.c.k_page + hk * p.c.k_head + row * p.c.k_row;
        r.v = page * p.c.v_page + hk * p.c.v_head + row * p.c.v_row;
        r.live = true;
      }
    }
    return r;
  };
  // copies of one tile into a stage: whole rows, 16 bytes a lane
  auto load = [&](int stage, const Row& r) {
    constexpr int CH = D / 8, RPI = 32 / CH > 0 ? 32 / CH : 1;  // pieces of a row, rows per step
    const int c = lane % CH;
    const uint32_t kdst = ring + stage * C::STAGE, vdst = kdst + KT * C::ROW;
    const uint32_t live = __ballot_sync(0xffffffffu, r.live);
    if (lane == 0) valid[stage] = live;
    const bool col_ok = 8 * c < p.c.d;
#pragma unroll
    for (int s = 0; s < KT / RPI; ++s) {
      const int row = s * RPI + lane / CH;
      const long long ko = __shfl_sync(0xffffffffu, r.k, row);
      const long long vo = __shfl_sync(0xffffffffu, r.v, row);
      const bool ok = col_ok && ((live >> row) & 1u);
      const uint32_t at = row * C::ROW + ((c ^ (row & 7)) << 4);
      cp_async16(kdst + at, p.k + (ok ? ko + 8 * c : 0), ok);
      cp_async16(vdst + at, p.v + (ok ? vo + 8 * c : 0), ok);
    }
  };

  float o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int u = 0; u < 4; ++u) o[i][u] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // rows g, g + 8; l: this lane's part

  // tiles warp, warp + kWarps, ...
  int fill = warp;
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) {
    if (fill < tiles) load(s, locate(fill));
    cp_async_commit();
    fill += kWarps;
  }
  Row next = locate(fill);
  int stage = 0;
  for (int tile = warp; tile < tiles; tile += kWarps) {
    // the next free stage was read in the previous round
    __syncwarp();
    {
      const int into = stage == 0 ? STAGES - 1 : stage - 1;
      if (fill < tiles) load(into, next);
      cp_async_commit();
      fill += kWarps;
      next = locate(fill);
    }
    cp_async_wait<STAGES - 1>();
    __syncwarp();
    const uint32_t kbase = ring + stage * C::STAGE, vbase = kbase + KT * C::ROW;
    const uint32_t live = valid[stage];
    float s[KT / 8][4];
#pragma unroll
    for (int i = 0; i < KT / 8; ++i)
#pragma unroll
      for (int u = 0; u < 4; ++u) s[i][u] = 0.f;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
      for (int kt = 0; kt < KT / 16; ++kt) {
        uint32_t kb[4];
        const int row = kt * 16 + (lane & 7) + ((lane >> 4) & 1) * 8;
        const int ch = 2 * kk + ((lane >> 3) & 1);
        ldsm_x4(kbase + row * C::ROW + ((ch ^ (row & 7)) << 4), kb);
        mma16816(s[2 * kt], qa[kk], kb[0], kb[1]);
        mma16816(s[2 * kt + 1], qa[kk], kb[2], kb[3]);
      }
    constexpr uint32_t kAll = KT == 32 ? 0xffffffffu : (1u << (KT & 31)) - 1u;
    if ((live & kAll) != kAll) {
#pragma unroll
      for (int i = 0; i < KT / 8; ++i)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (((live >> (8 * i + 2 * q4 + (u & 1))) & 1u) == 0u) s[i][u] = -INFINITY;
    }
    float alpha[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < KT / 8; ++i) mx = fmax3(mx, s[i][2 * r], s[i][2 * r + 1]);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float m_new = fmaxf(m[r], mx * p.scale_log2);
      const float ref = m_new == -INFINITY ? 0.f : m_new;
      alpha[r] = fast_exp2(m[r] - ref);
      m[r] = m_new;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < KT / 8; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float e = fast_exp2(fmaf(s[i][2 * r + u], p.scale_log2, -ref));
          s[i][2 * r + u] = e;
          sum += e;
        }
      l[r] = l[r] * alpha[r] + sum;
    }
    if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][0] *= alpha[0];
        o[i][1] *= alpha[0];
        o[i][2] *= alpha[1];
        o[i][3] *= alpha[1];
      }
    }
    // P is rounded to bf16 for the second product, as in the other attention
    // kernels; the row sum keeps the unrounded values
#pragma unroll
    for (int kt = 0; kt < KT / 16; ++kt) {
      const uint32_t pa[4] = {pack_bf16(s[2 * kt][0], s[2 * kt][1]), pack_bf16(s[2 * kt][2], s[2 * kt][3]),
                              pack_bf16(s[2 * kt + 1][0], s[2 * kt + 1][1]),
                              pack_bf16(s[2 * kt + 1][2], s[2 * kt + 1][3])};
#pragma unroll
      for (int dd = 0; dd < D / 16; ++dd) {
        uint32_t vb[4];
        const int row = kt * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
        const int ch = 2 * dd + (lane >> 4);
        ldsm_x4_trans(vbase + row * C::ROW + ((ch ^ (row & 7)) << 4), vb);
        mma16816(o[2 * dd], pa, vb[0], vb[1]);
        mma16816(o[2 * dd + 1], pa, vb[2], vb[3]);
      }
    }
    stage = stage + 1 == STAGES ? 0 : stage + 1;
  }
  cp_async_wait<0>();
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
  }

  // The warps' parts meet in the (now idle) ring: [warp][16 rows] statistics
  // and [warp][16][D] fp32 sums.
  __syncthreads();
  float2* stat = reinterpret_cast<float2*>(smem);
  float* acc = reinterpret_cast<float*>(smem + kWarps * 16 * sizeof(float2));
  if (q4 == 0) {
    stat[warp * 16 + g] = make_float2(m[0], l[0]);
    stat[warp * 16 + g + 8] = make_float2(m[1], l[1]);
  }
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    float* a = acc + (warp * 16 + g) * D + 8 * i + 2 * q4;
    *reinterpret_cast<float2*>(a) = make_float2(o[i][0], o[i][1]);
    *reinterpret_cast<float2*>(a + 8 * D) = make_float2(o[i][2], o[i][3]);
  }
  __syncthreads();
  for (int x = threadIdx.x; x < hn * (D / 8); x += kWarps * 32) {
    const int r = x / (D / 8), col = 8 * (x % (D / 8));
    if (col >= p.c.d) continue;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, stat[w * 16 + r].x);
    const float ref = mm == -INFINITY ? 0.f : mm;
    float sum = 0.f, out[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 st = stat[w * 16 + r];
      const float f = fast_exp2(st.x - ref);
      sum += f * st.y;
#pragma unroll
      for (int e = 0; e < 8; ++e) out[e] = fmaf(f, acc[(w * 16 + r) * D + col + e], out[e]);
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    *reinterpret_cast<uint4*>(p.o + b * p.o_batch + (h0 + r) * p.o_head + col) =
        make_uint4(pack_bf16(out[0] * inv, out[1] * inv), pack_bf16(out[2] * inv, out[3] * inv),
                   pack_bf16(out[4] * inv, out[5] * inv), pack_bf16(out[6] * inv, out[7] * inv));
    if (col == 0)
      p.lse[static_cast<long long>(b) * p.heads + h0 + r] =
          sum > 0.f ? (mm + log2f(sum)) * kLn2 : -INFINITY;
  }
}

template <int D>
cudaError_t launch_attend(const AttendParams& p, cudaStream_t stream) {
  using C = DecodeCfg<D>;
  static_assert(kWarps * 16 * (8 + D * 4) <= C::OFF_VALID, "the warps' parts fit the ring");
  auto kern = attend_kernel<D>;
  static OncePerContext prepared;
  const cudaError_t e = prepared.run([&]() -> cudaError_t {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(C::SMEM));
  });
  if (e != cudaSuccess) return e;
  const long long units = static_cast<long long>(p.batch) * p.c.heads_kv * p.head_blocks;
  return launch_overlapped(kern, dim3(static_cast<unsigned>(units)), dim3(kWarps * 32), C::SMEM,
                           stream, p);
}

// Work units of a call: 0 if there are too many for a grid.
long long units_of(const Cache& c, int batch, int heads) {
  const int blocks = (heads / c.heads_kv + 15) / 16;
  const long long units = static_cast<long long>(batch) * c.heads_kv * blocks;
  return units <= 0x7FFFFFFF ? units : 0;
}

}  // namespace
}  // namespace fa

extern "C" {

size_t fa_cache_attend_workspace_size(const fa_cache_t* cache, int batch, int heads, int window,
                                      int sinks) {
  (void)cache, (void)batch, (void)heads, (void)window, (void)sinks;
  return 0;
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
  if (fa::units_of(p.c, batch, heads) == 0) return FA_ERR_UNSUPPORTED;
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
  p.head_blocks = (p.group + 15) / 16;
  p.scale_log2 = static_cast<float>(static_cast<double>(softmax_scale) * fa::kLog2e);
  p.window = window;
  p.sinks = sinks;
  (void)workspace, (void)workspace_bytes;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = p.c.d <= 64    ? fa::launch_attend<64>(p, s)
                        : p.c.d <= 128 ? fa::launch_attend<128>(p, s)
                                       : fa::launch_attend<256>(p, s);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
