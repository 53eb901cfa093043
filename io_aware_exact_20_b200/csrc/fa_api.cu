// C ABI of the attention library: argument validation, TMA descriptor set-up
// and kernel launch.  See include/fa.h for the contract of every entry point.
//
// Every entry point first turns its arguments into one validated Problem (the
// classic [B, H, N, d] calls are the padded layout with contiguous strides and
// N_q = N_k = N); the launches below only ever see a Problem.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "devctx.h"
#include "fa.h"
#include "kernels.h"
#include "tmap.h"

namespace {

// One status word per device, in the library's own device memory (a
// file-scope __device__ variable, so no allocation happens at run time).
__device__ int g_status_word;

fa::SymbolAddressCache g_status_cache;
std::atomic<uint64_t> g_timeout_ns{4000000000ull};
std::atomic<int> g_mask_bitmap{1};

// Device address of the status word in the current device's context.
int* status_word() {
  return static_cast<int*>(g_status_cache.get([]() -> void* {
    void* ptr = nullptr;
    if (cudaGetSymbolAddress(&ptr, g_status_word) != cudaSuccess) return nullptr;
    return ptr;
  }));
}

}  // namespace

int* fa::device_status() { return status_word(); }

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool tensor_ok(const void* p) { return p != nullptr && aligned(p, 16); }

struct Dropout {
  uint32_t threshold;
  float rscale;
};

// Keep test: a 16-bit uniform >= threshold = min(floor(p 2^16), 2^16 - 1);
// kept values are divided by the keep probability 1 - threshold / 2^16.
Dropout dropout_params(float p) {
  const double t = std::floor(static_cast<double>(p) * 65536.0);
  Dropout d;
  d.threshold = t >= 65535.0 ? 65535u : static_cast<uint32_t>(t);
  d.rscale = static_cast<float>(65536.0 / (65536.0 - static_cast<double>(d.threshold)));
  return d;
}

constexpr double kLog2e = 1.4426950408889634074;
constexpr int kMaxRows = 1 << 23;

// Kernel width for a head dimension (0 if unsupported): 32 and 96 run the 64-
// and 128-wide kernels, whose extra columns TMA fills with zeros.
int kernel_dim(int d) {
  if (d == 32 || d == 64) return 64;
  if (d == 96 || d == 128) return 128;
  if (d == 192 || d == 256) return 256;
  return 0;
}

// A validated request.
struct Problem {
  int B, H, d, D;
  int nq, nk;                  // padded: rows per entry; packed: longest sequence
  bool packed;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int total_q, total_k;        // packed: rows of the tensors
  const int32_t* seqlens;
  float scale;
  int causal;
  float dropout_p;
  uint64_t seed;
  const uint8_t* block_mask;
  fa_strides_t q, k, v, o, dout, dq, dk, dv;
  int64_t drop_row0, drop_key0;  // dropout positions of the first query row and key
  int Hkv;                       // K / V heads (H / Hkv query heads share each)
  int window, sinks;             // sliding window (0: none), first keys that stay visible
  bool own_key;                  // the call's window is the query's own key alone

  int rows_q() const { return packed ? total_q : nq; }
  int rows_k() const { return packed ? total_k : nk; }
  int tb() const { return packed ? 1 : B; }
};

bool strides_ok(const fa_strides_t& s, bool packed) {
  if (s.head < 0 || s.row < 0 || (!packed && s.batch < 0)) return false;
  if (s.head % 8 || s.row % 8 || (!packed && s.batch % 8)) return false;
  return s.head < (int64_t{1} << 36) && s.row < (int64_t{1} << 36) &&
         (packed || s.batch < (int64_t{1} << 36));
}

// The tensors a call uses: the forward reads Q, K, V and writes O; the
// backward (and its workspace size) uses all eight.  Strides of unused tensors
// are not looked at.
enum Uses { kForward, kBackward };

fa_status_t resolve(const fa_attention_desc_t* a, Problem* p, Uses uses) {
  if (a == nullptr) return FA_ERR_INVALID_ARG;
  if (a->batch < 1 || a->heads < 1 || a->seqlen_q < 1 || a->seqlen_k < 1)
    return FA_ERR_INVALID_ARG;
  if (!(a->softmax_scale > 0.f) || !std::isfinite(a->softmax_scale)) return FA_ERR_INVALID_ARG;
  if (!(a->dropout_p >= 0.f && a->dropout_p < 1.f)) return FA_ERR_INVALID_ARG;
  if ((a->cu_seqlens_q == nullptr) != (a->cu_seqlens_k == nullptr)) return FA_ERR_INVALID_ARG;
  const bool packed = a->cu_seqlens_q != nullptr;
  if (packed && (!aligned(a->cu_seqlens_q, 4) || !aligned(a->cu_seqlens_k, 4) ||
                 a->total_q < 1 || a->total_k < 1))
    return FA_ERR_INVALID_ARG;
  if (a->seqlens_k != nullptr && !aligned(a->seqlens_k, 4)) return FA_ERR_INVALID_ARG;
  const int D = kernel_dim(a->head_dim);
  if (D == 0) return FA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(a->batch) * a->heads > 65535) return FA_ERR_UNSUPPORTED;
  if (a->seqlen_q > kMaxRows || a->seqlen_k > kMaxRows) return FA_ERR_UNSUPPORTED;
  // one CTA per (b, h, 128-row tile) in a 1-D grid
  const int64_t tiles = (static_cast<int64_t>(a->seqlen_q > a->seqlen_k ? a->seqlen_q : a->seqlen_k) +
                         127) / 128;
  // (the d = 256 backward runs two CTAs per key tile)
  const int64_t per_tile = (uses == kBackward && D == 256) ? 2 : 1;
  if (static_cast<int64_t>(a->batch) * a->heads * tiles * per_tile > 0x7FFFFFFF)
    return FA_ERR_UNSUPPORTED;
  // grouped-query attention: heads_kv K / V heads, each shared by heads / heads_kv
  const int hkv = a->heads_kv == 0 ? a->heads : a->heads_kv;
  if (hkv < 1 || hkv > a->heads || a->heads % hkv != 0) return FA_ERR_INVALID_ARG;
  // the backward's walk packs (query head of the group, query tile) in 16 + 16 bits
  if (a->heads / hkv >= 32768) return FA_ERR_UNSUPPORTED;
  const fa_strides_t* all[8] = {&a->q, &a->k, &a->v, &a->o, &a->dout, &a->dq, &a->dk, &a->dv};
  const bool kv_side[8] = {false, true, true, false, false, false, true, true};
  for (int t = 0; t < (uses == kForward ? 4 : 8); ++t) {
    const fa_strides_t* s = all[t];
    if (!strides_ok(*s, packed)) return FA_ERR_INVALID_ARG;
    // a zero stride would make heads / entries / rows share memory
    const int heads_t = kv_side[t] ? hkv : a->heads;
    if ((heads_t > 1 && s->head == 0) || (!packed && a->batch > 1 && s->batch == 0) ||
        s->row == 0)
      return FA_ERR_INVALID_ARG;
  }
  // dropout positions: counter words are 32-bit, keys go in groups of 8
  if (a->dropout_row0 < 0 || a->dropout_key0 < 0 || a->dropout_key0 % 8 != 0 ||
      a->dropout_row0 > 0x7FFFFFFFll - a->seqlen_q || a->dropout_key0 > 0x7FFFFFFFll - a->seqlen_k)
    return FA_ERR_INVALID_ARG;
  if (a->window < 0 || a->sinks < 0 || (a->window > 0 && a->causal == 0)) return FA_ERR_INVALID_ARG;
  // a window as long as the keys hides nothing: the kernels without it run.
  // Positions are below kMaxRows, so longer windows and more first keys than
  // that change nothing either (and the kernels' sums stay inside 32 bits).
  p->window = a->window < a->seqlen_k ? a->window : 0;
  p->own_key = a->window == 1 && a->sinks == 0;  // (of one key, too)
  p->sinks = a->sinks < kMaxRows ? a->sinks : kMaxRows;
  p->drop_row0 = a->dropout_row0;
  p->drop_key0 = a->dropout_key0;
  p->Hkv = hkv;
  p->B = a->batch;
  p->H = a->heads;
  p->d = a->head_dim;
  p->D = D;
  p->nq = a->seqlen_q;
  p->nk = a->seqlen_k;
  p->packed = packed;
  p->cu_q = a->cu_seqlens_q;
  p->cu_k = a->cu_seqlens_k;
  p->total_q = packed ? a->total_q : 0;
  p->total_k = packed ? a->total_k : 0;
  p->seqlens = a->seqlens_k;
  p->scale = a->softmax_scale;
  p->causal = a->causal != 0;
  p->dropout_p = a->dropout_p;
  p->seed = a->seed;
  p->block_mask = a->block_mask;
  p->q = a->q;
  p->k = a->k;
  p->v = a->v;
  p->o = a->o;
  p->dout = a->dout;
  p->dq = a->dq;
  p->dk = a->dk;
  p->dv = a->dv;
  if (packed) {  // the batch coordinate is always 0
    for (fa_strides_t* s : {&p->q, &p->k, &p->v, &p->o, &p->dout, &p->dq, &p->dk, &p->dv})
      s->batch = 0;
  }
  return FA_OK;
}

// The classic contiguous [B, H, N, d] request.
fa_attention_desc_t classic_desc(int B, int H, int N, int d, float scale, int causal,
                                 const int32_t* seqlens, float dropout_p, uint64_t seed,
                                 const uint8_t* block_mask) {
  fa_attention_desc_t a{};
  a.batch = B;
  a.heads = H;
  a.head_dim = d;
  a.seqlen_q = N;
  a.seqlen_k = N;
  a.seqlens_k = seqlens;
  a.softmax_scale = scale;
  a.causal = causal;
  a.dropout_p = dropout_p;
  a.seed = seed;
  a.block_mask = block_mask;
  const fa_strides_t s{static_cast<int64_t>(H) * N * d, static_cast<int64_t>(N) * d, d};
  a.q = a.k = a.v = a.o = a.dout = a.dq = a.dk = a.dv = s;
  return a;
}

fa::Strides kstrides(const fa_strides_t& s) { return fa::Strides{s.batch, s.head, s.row}; }

fa::Rows kernel_rows(const Problem& p) {
  fa::Rows r;
  r.cu_q = p.cu_q;
  r.cu_k = p.cu_k;
  r.nq = p.nq;
  r.nk = p.nk;
  r.total_q = p.total_q;
  r.total_k = p.total_k;
  return r;
}

// TMA view {d, rows, H, batch} of a bf16 tensor; box 64 x 128 x 1 x 1.
bool tmap(CUtensorMap* m, const void* base, const Problem& p, const fa_strides_t& s, int rows,
          int heads) {
  fa::TmapDesc t = fa::tmap_desc_zero();
  t.base = base;
  t.dtype = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  t.rank = 4;
  t.dims[0] = static_cast<uint64_t>(p.d);
  t.dims[1] = static_cast<uint64_t>(rows);
  t.dims[2] = static_cast<uint64_t>(heads);
  t.dims[3] = static_cast<uint64_t>(p.tb());
  // a zero stride (a single head or batch entry) is described as the
  // smallest legal one; that coordinate is always 0
  t.strides[0] = static_cast<uint64_t>(s.row ? s.row : 8) * 2;
  t.strides[1] = static_cast<uint64_t>(s.head ? s.head : 8) * 2;
  t.strides[2] = static_cast<uint64_t>(s.batch ? s.batch : 8) * 2;
  t.box[0] = 64;
  t.box[1] = 128;
  t.box[2] = 1;
  t.box[3] = 1;
  return fa::tmap_cache().encode(t, m);
}

// LSE element strides of a batch entry and a head.
void lse_strides(const Problem& p, long long* sb, long long* sh) {
  if (p.packed) {
    *sb = 0;
    *sh = p.total_q;
  } else {
    *sb = static_cast<long long>(p.H) * p.nq;
    *sh = p.nq;
  }
}

// Rows of each workspace array (a multiple of 128), with the padded layout's
// rows per (b, h) or the packed layout's rows per head.
int64_t ws_rows(const Problem& p, int* npad, int64_t* rtot) {
  if (!p.packed) {
    *npad = (p.nq + 127) / 128 * 128;
    *rtot = 0;
    return static_cast<int64_t>(p.B) * p.H * *npad;
  }
  *npad = 0;
  *rtot = (static_cast<int64_t>(p.total_q) + 127) / 128 * 128 + 256ll * p.B;
  return static_cast<int64_t>(p.H) * *rtot;
}

// Parts per backward unit under grouped K / V heads: the smallest divisor of
// the group whose parts give about four units per SM of the 148 (every divisor
// up to the whole group when there are fewer); 1 without grouping.  A split
// unit adds its dK / dV into fp32 accumulators converted at the end.  Under a
// window the units are equally long, so one and a half per SM balance them, and
// short, so a part's set-up and fp32 slices weigh more (16K, 4 K / V heads of 4,
// d = 128, window 1024: 607 us in 512 whole units, 705 in 1024 halves; 4K, window
// 512: 135 us in 256 halves, 145 in 128 whole units, 169 in 512 quarters).
std::atomic<int> g_gqa_split{0};  // test support: forced parts, 0 = automatic

int split_of(const Problem& p) {
  if (p.Hkv <= 0 || p.Hkv == p.H) return 1;
  const int G = p.H / p.Hkv;
  const int forced = g_gqa_split.load();
  if (forced > 0 && G % forced == 0) return forced;
  const int64_t units = static_cast<int64_t>(p.B) * p.Hkv * ((p.nk + 127) / 128) *
                        (p.D == 256 ? 2 : 1);
  int s = 1;
  for (int c = 1; c <= G; ++c) {
    if (G % c) continue;
    s = c;
    if (units * c >= (p.window > 0 ? 3 * 148 / 2 : 4 * 148)) break;
  }
  return s;
}

// fp32 elements of each of the dK / dV areas of split units: one slice
// [tb][H_kv][key rows][D] per part
int64_t kv_acc_elems(const Problem& p) {
  const int s = split_of(p);
  if (s == 1) return 0;
  return static_cast<int64_t>(s) * p.tb() * p.Hkv * p.rows_k() * p.D;
}

// First keys under a sliding window, in the backward: see BwdParams.  A unit of
// a first key tile walks all later query tiles where the others walk the
// window, so its walk is cut into pieces of at least a window's length (and 8
// tiles), fewer where the first tiles' units alone would fill the GPU four
// times.  (16K sequence, 4 K / V heads of 4 query heads, d = 128, window 1024, 4
// first keys: 1430 us with whole walks, 627 without first keys.)
struct SinkCut {
  int tiles = 0, chunks = 0, len = 0;
  int64_t elems = 0;  // of each of the dK / dV slices
};

SinkCut sink_cut_of(const Problem& p) {
  SinkCut c;
  if (p.window == 0 || p.sinks == 0) return c;
  const int64_t key_tiles = (p.nk + 127) / 128, q_tiles = (p.nq + 127) / 128;
  const int64_t tiles = (p.sinks + 127) / 128 < key_tiles ? (p.sinks + 127) / 128 : key_tiles;
  const int64_t units = static_cast<int64_t>(p.B) * p.Hkv * split_of(p) * tiles;
  if (units >= 4 * 148) return c;
  int64_t len = p.window / 128 + 1;
  if (len < 8) len = 8;
  if (len < (q_tiles * units + 4 * 148 - 1) / (4 * 148)) len = (q_tiles * units + 4 * 148 - 1) / (4 * 148);
  if (q_tiles <= len) return c;
  c.tiles = static_cast<int>(tiles);
  c.len = static_cast<int>(len);
  c.chunks = static_cast<int>((q_tiles + len - 1) / len);
  c.elems = (1 + c.chunks) * units * 128 * p.D;
  return c;
}

size_t workspace_bytes_of(const Problem& p) {
  int npad = 0;
  int64_t rtot = 0;
  const uint64_t rows = static_cast<uint64_t>(ws_rows(p, &npad, &rtot));
  const uint64_t bytes = rows * (4ull + 4ull + 4ull * p.D) + 8ull * kv_acc_elems(p) +
                         8ull * sink_cut_of(p).elems;
  return static_cast<size_t>((bytes + 255) / 256 * 256);
}

#ifdef FA_DEBUG_BOUNDS
// Elements from a tensor's base to one past the last element a call may touch.
long long span(const fa_strides_t& s, int tb, int H, long long rows, int d) {
  return (tb - 1) * s.batch + (H - 1) * s.head + (rows - 1) * s.row + d;
}

// Extents of the buffers the kernels address directly, and the rows' offsets.
void set_extents(const Problem& pr, int* status, fa::Extents* e, fa::Rows* rows) {
  const int tb = pr.tb();
  e->o = span(pr.o, tb, pr.H, pr.rows_q(), pr.d);
  e->dout = span(pr.dout, tb, pr.H, pr.rows_q(), pr.d);
  e->dq = span(pr.dq, tb, pr.H, pr.rows_q(), pr.d);
  e->dk = span(pr.dk, tb, pr.Hkv, pr.rows_k(), pr.d);
  e->dv = span(pr.dv, tb, pr.Hkv, pr.rows_k(), pr.d);
  long long sb = 0, sh = 0;
  lse_strides(pr, &sb, &sh);
  e->lse = (tb - 1) * sb + (pr.H - 1) * sh + pr.rows_q();
  e->mask = pr.block_mask != nullptr
                ? static_cast<long long>((pr.nq + 127) / 128) * ((pr.nk + 127) / 128)
                : 0;
  e->seqlens = pr.seqlens != nullptr ? pr.B : 0;
  e->kvacc = kv_acc_elems(pr);
  e->sink = sink_cut_of(pr).elems;
  rows->n_cu = pr.packed ? pr.B + 1 : 0;
  rows->status = status;
}
#endif

fa_status_t run_fwd(const Problem& pr, const void* q, const void* k, const void* v, void* o,
                    float* lse, void* stream) {
  if (!tensor_ok(q) || !tensor_ok(k) || !tensor_ok(v) || !tensor_ok(o)) return FA_ERR_INVALID_ARG;
  if (lse == nullptr || !aligned(lse, 4)) return FA_ERR_INVALID_ARG;
  int* status = status_word();
  if (status == nullptr) return FA_ERR_CUDA;
  CUtensorMap tq, tk, tv;
  if (!tmap(&tq, q, pr, pr.q, pr.rows_q(), pr.H) || !tmap(&tk, k, pr, pr.k, pr.rows_k(), pr.Hkv) ||
      !tmap(&tv, v, pr, pr.v, pr.rows_k(), pr.Hkv))
    return FA_ERR_UNSUPPORTED;
  const Dropout dr = dropout_params(pr.dropout_p);
  fa::FwdParams p{};
  p.o = o;
  p.so = kstrides(pr.o);
  p.lse = lse;
  lse_strides(pr, &p.lse_sb, &p.lse_sh);
  p.seqlens = pr.seqlens;
  p.block_mask = pr.block_mask;
  p.nbq = (pr.nq + 127) / 128;
  p.nbk = (pr.nk + 127) / 128;
  p.status = status;
  p.rows = kernel_rows(pr);
  p.B = pr.B;
  p.H = pr.H;
  p.group = pr.H / pr.Hkv;
  p.window = pr.window;
  p.sinks = pr.sinks;
  p.d_real = pr.d;
  p.scale_log2 = static_cast<float>(static_cast<double>(pr.scale) * kLog2e);
  p.causal = pr.causal;
  p.group_heads = fa::order_group_heads(pr.B, pr.H, fa::fwd_head_bytes(pr.nk, pr.D), pr.causal);
  p.drop_threshold = dr.threshold;
  p.drop_rscale = dr.rscale;
  p.seed_lo = static_cast<uint32_t>(pr.seed & 0xFFFFFFFFull);
  p.seed_hi = static_cast<uint32_t>(pr.seed >> 32);
  p.rk = fa::philox_round_keys(pr.seed);
  p.drop_row0 = static_cast<uint32_t>(pr.drop_row0);
  p.drop_kgrp0 = static_cast<uint32_t>(pr.drop_key0 / 8);
  p.timeout_ns = g_timeout_ns.load();
  p.mask_bitmap = g_mask_bitmap.load();
#ifdef FA_DEBUG_BOUNDS
  set_extents(pr, status, &p.ext, &p.rows);
#endif
  const cudaError_t e =
      fa::launch_fwd(pr.D, dr.threshold != 0, tq, tk, tv, p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// Scalar and workspace fields shared by the three backward launches.
fa_status_t bwd_params(fa::BwdParams* p, const Problem& pr, const void* workspace,
                       size_t workspace_bytes) {
  if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < workspace_bytes_of(pr))
    return FA_ERR_WORKSPACE;
  int* status = status_word();
  if (status == nullptr) return FA_ERR_CUDA;
  const Dropout dr = dropout_params(pr.dropout_p);
  *p = fa::BwdParams{};
  int npad = 0;
  int64_t rtot = 0;
  const int64_t rows = ws_rows(pr, &npad, &rtot);
  if (rows > 0x7FFFFFFFll) return FA_ERR_UNSUPPORTED;  // TMA row coordinate of the dQ reduce
  p->ws_lse2 = static_cast<float*>(const_cast<void*>(workspace));
  p->ws_delta = p->ws_lse2 + rows;
  p->ws_dq = p->ws_delta + rows;
  p->ws_rows = rows;
  p->split = split_of(pr);
  p->rows_tb = pr.tb();
  p->ws_dk = p->split > 1 ? p->ws_dq + rows * pr.D : nullptr;
  p->ws_dv = p->split > 1 ? p->ws_dk + kv_acc_elems(pr) : nullptr;
  const SinkCut cut = sink_cut_of(pr);
  p->sink_tiles = cut.tiles;
  p->sink_chunks = cut.chunks;
  p->sink_len = cut.len;
  p->sink_units = static_cast<long long>(pr.B) * pr.Hkv * p->split * cut.tiles * cut.chunks;
  p->ws_sk = cut.tiles > 0 ? p->ws_dq + rows * pr.D + 2 * kv_acc_elems(pr) : nullptr;
  p->ws_sv = cut.tiles > 0 ? p->ws_sk + cut.elems : nullptr;
  p->Npad = npad;
  p->Rtot = rtot;
  lse_strides(pr, &p->lse_sb, &p->lse_sh);
  p->so = kstrides(pr.o);
  p->sdo = kstrides(pr.dout);
  p->sdq = kstrides(pr.dq);
  p->sdk = kstrides(pr.dk);
  p->sdv = kstrides(pr.dv);
  p->seqlens = pr.seqlens;
  p->block_mask = pr.block_mask;
  p->nbq = (pr.nq + 127) / 128;
  p->nbk = (pr.nk + 127) / 128;
  p->status = status;
  p->rows = kernel_rows(pr);
  p->B = pr.B;
  p->H = pr.H;
  p->group = pr.H / pr.Hkv;
  p->window = pr.window;
  p->sinks = pr.sinks;
  p->d_real = pr.d;
  // A window of the query's own key alone: its probability is 1 whatever the
  // score, so dQ and dK are exactly 0; dP - D would leave rounding noise there.
  // (This scale is only the final factor of dQ and dK.)
  p->scale = pr.own_key ? 0.f : pr.scale;
  p->scale_log2 = static_cast<float>(static_cast<double>(pr.scale) * kLog2e);
  p->causal = pr.causal;
  // the main kernel's units are (b, K / V head, key tile): its head groups are
  // of K / V heads, each sharing the Q / dO rows of H / Hkv query heads
  p->group_heads = fa::order_group_heads(pr.B, pr.Hkv,
                                         (pr.H / pr.Hkv) * fa::bwd_head_bytes(pr.nq, pr.D),
                                         pr.causal);
  p->drop_threshold = dr.threshold;
  p->drop_rscale = dr.rscale;
  p->seed_lo = static_cast<uint32_t>(pr.seed & 0xFFFFFFFFull);
  p->seed_hi = static_cast<uint32_t>(pr.seed >> 32);
  p->rk = fa::philox_round_keys(pr.seed);
  p->drop_row0 = static_cast<uint32_t>(pr.drop_row0);
  p->drop_kgrp0 = static_cast<uint32_t>(pr.drop_key0 / 8);
  p->timeout_ns = g_timeout_ns.load();
  p->mask_bitmap = g_mask_bitmap.load();
#ifdef FA_DEBUG_BOUNDS
  set_extents(pr, status, &p->ext, &p->rows);
#endif
  return FA_OK;
}

// Tensor maps of the main backward kernel.
struct BwdMaps {
  CUtensorMap q, k, v, dout, dq;
};

fa_status_t bwd_maps(BwdMaps* m, const Problem& pr, const fa::BwdParams& p, const void* q,
                     const void* k, const void* v, const void* dout) {
  if (!tmap(&m->q, q, pr, pr.q, pr.rows_q(), pr.H) ||
      !tmap(&m->k, k, pr, pr.k, pr.rows_k(), pr.Hkv) ||
      !tmap(&m->v, v, pr, pr.v, pr.rows_k(), pr.Hkv) ||
      !tmap(&m->dout, dout, pr, pr.dout, pr.rows_q(), pr.H))
    return FA_ERR_UNSUPPORTED;
  if (!fa::make_tmap_f32_2d(&m->dq, p.ws_dq, static_cast<uint64_t>(pr.D),
                            static_cast<uint64_t>(p.ws_rows), 128))
    return FA_ERR_CUDA;
  return FA_OK;
}

fa_status_t run_bwd(const Problem& pr, const void* q, const void* k, const void* v, const void* o,
                    const float* lse, const void* dout, void* dq, void* dk, void* dv,
                    void* workspace, size_t workspace_bytes, void* stream) {
  if (!tensor_ok(q) || !tensor_ok(k) || !tensor_ok(v) || !tensor_ok(o) || !tensor_ok(dout) ||
      !tensor_ok(dq) || !tensor_ok(dk) || !tensor_ok(dv))
    return FA_ERR_INVALID_ARG;
  if (lse == nullptr || !aligned(lse, 4)) return FA_ERR_INVALID_ARG;
  fa::BwdParams p;
  fa_status_t st = bwd_params(&p, pr, workspace, workspace_bytes);
  if (st != FA_OK) return st;
  BwdMaps m;
  st = bwd_maps(&m, pr, p, q, k, v, dout);
  if (st != FA_OK) return st;
  p.o = o;
  p.lse = lse;
  p.dout = dout;
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (fa::launch_bwd_pre(pr.D, p, s) != cudaSuccess) return FA_ERR_CUDA;
  if (fa::launch_bwd_main(pr.D, p.drop_threshold != 0, m.q, m.k, m.v, m.dout, m.dq, p, s) !=
      cudaSuccess)
    return FA_ERR_CUDA;
  const cudaError_t e = p.split > 1 || p.sink_tiles > 0 ? fa::launch_bwd_post_all(pr.D, p, s)
                                                       : fa::launch_bwd_post(pr.D, p, s);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

extern "C" {

const char* fa_status_string(fa_status_t s) {
  switch (s) {
    case FA_OK: return "ok";
    case FA_ERR_INVALID_ARG: return "invalid argument";
    case FA_ERR_UNSUPPORTED: return "unsupported configuration";
    case FA_ERR_CUDA: return "CUDA error";
    case FA_ERR_TIMEOUT: return "kernel pipeline wait timed out";
    case FA_ERR_WORKSPACE: return "workspace missing or too small";
    case FA_ERR_BOUNDS: return "a kernel index was out of bounds (bounds-checking build)";
  }
  return "unknown status";
}

void fa_set_wait_timeout_ns(uint64_t ns) { g_timeout_ns.store(ns < 1000000ull ? 1000000ull : ns); }

void fa_debug_set_block_mask_bitmap(int enabled) { g_mask_bitmap.store(enabled != 0 ? 1 : 0); }

void fa_debug_set_gqa_split(int parts) { g_gqa_split.store(parts > 0 ? parts : 0); }

int fa_debug_bounds_checking(void) {
#ifdef FA_DEBUG_BOUNDS
  return 1;
#else
  return 0;
#endif
}

fa_status_t fa_last_device_status(void* stream) {
  int* w = status_word();
  if (w == nullptr) return FA_ERR_CUDA;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return FA_ERR_CUDA;
  int v = 0;
  if (cudaMemcpy(&v, w, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return FA_ERR_CUDA;
  const int zero = 0;
  if (cudaMemcpy(w, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess) return FA_ERR_CUDA;
  if (v == fa::kStatusTimeout) return FA_ERR_TIMEOUT;
  if (v != 0) return FA_ERR_CUDA;
  return FA_OK;
}

fa_status_t fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                   int N, int d, float softmax_scale, int causal, const int32_t* seqlens,
                   float dropout_p, uint64_t seed, const uint8_t* block_mask, void* stream) {
  if (seqlens != nullptr && !aligned(seqlens, 4)) return FA_ERR_INVALID_ARG;
  const fa_attention_desc_t a =
      classic_desc(B, H, N, d, softmax_scale, causal, seqlens, dropout_p, seed, block_mask);
  Problem pr;
  const fa_status_t st = resolve(&a, &pr, kForward);
  if (st != FA_OK) return st;
  return run_fwd(pr, q, k, v, o, lse, stream);
}

fa_status_t fa_fwd_ex(const fa_attention_desc_t* desc, const void* q, const void* k,
                      const void* v, void* o, float* lse, void* stream) {
  Problem pr;
  const fa_status_t st = resolve(desc, &pr, kForward);
  if (st != FA_OK) return st;
  return run_fwd(pr, q, k, v, o, lse, stream);
}

size_t fa_bwd_workspace_size(int B, int H, int N, int d) {
  if (B < 1 || H < 1 || N < 1 || kernel_dim(d) == 0) return 0;
  const fa_attention_desc_t a = classic_desc(B, H, N, d, 1.f, 0, nullptr, 0.f, 0, nullptr);
  Problem pr;
  if (resolve(&a, &pr, kBackward) != FA_OK) {  // sizes beyond the kernels' limits: still report the bytes
    pr = Problem{};
    pr.B = B;
    pr.H = H;
    pr.nq = N;
    pr.D = kernel_dim(d);
  }
  return workspace_bytes_of(pr);
}

size_t fa_bwd_ex_workspace_size(const fa_attention_desc_t* desc) {
  Problem pr;
  if (resolve(desc, &pr, kBackward) != FA_OK) return 0;
  return workspace_bytes_of(pr);
}

fa_status_t fa_bwd_prepare(const void* o, const float* lse, const void* dout, int B, int H, int N,
                           int d, void* workspace, size_t workspace_bytes, void* stream) {
  if (!tensor_ok(o) || !tensor_ok(dout)) return FA_ERR_INVALID_ARG;
  if (lse == nullptr || !aligned(lse, 4)) return FA_ERR_INVALID_ARG;
  // scale and dropout do not enter this phase: validate with neutral values
  const fa_attention_desc_t a = classic_desc(B, H, N, d, 1.f, 0, nullptr, 0.f, 0, nullptr);
  Problem pr;
  fa_status_t st = resolve(&a, &pr, kBackward);
  if (st != FA_OK) return st;
  fa::BwdParams p;
  st = bwd_params(&p, pr, workspace, workspace_bytes);
  if (st != FA_OK) return st;
  p.o = o;
  p.lse = lse;
  p.dout = dout;
  return fa::launch_bwd_pre(pr.D, p, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

fa_status_t fa_bwd_main(const void* q, const void* k, const void* v, const void* dout, void* dk,
                        void* dv, int B, int H, int N, int d, float softmax_scale, int causal,
                        const int32_t* seqlens, float dropout_p, uint64_t seed,
                        const uint8_t* block_mask, void* workspace, size_t workspace_bytes,
                        void* stream) {
  if (!tensor_ok(q) || !tensor_ok(k) || !tensor_ok(v) || !tensor_ok(dout) || !tensor_ok(dk) ||
      !tensor_ok(dv))
    return FA_ERR_INVALID_ARG;
  if (seqlens != nullptr && !aligned(seqlens, 4)) return FA_ERR_INVALID_ARG;
  const fa_attention_desc_t a =
      classic_desc(B, H, N, d, softmax_scale, causal, seqlens, dropout_p, seed, block_mask);
  Problem pr;
  fa_status_t st = resolve(&a, &pr, kBackward);
  if (st != FA_OK) return st;
  fa::BwdParams p;
  st = bwd_params(&p, pr, workspace, workspace_bytes);
  if (st != FA_OK) return st;
  BwdMaps m;
  st = bwd_maps(&m, pr, p, q, k, v, dout);
  if (st != FA_OK) return st;
  p.dout = dout;
  p.dk = dk;
  p.dv = dv;
  const cudaError_t e = fa::launch_bwd_main(pr.D, p.drop_threshold != 0, m.q, m.k, m.v, m.dout,
                                            m.dq, p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status_t fa_bwd_finish(void* dq, int B, int H, int N, int d, float softmax_scale,
                          const void* workspace, size_t workspace_bytes, void* stream) {
  if (!tensor_ok(dq)) return FA_ERR_INVALID_ARG;
  const fa_attention_desc_t a =
      classic_desc(B, H, N, d, softmax_scale, 0, nullptr, 0.f, 0, nullptr);
  Problem pr;
  fa_status_t st = resolve(&a, &pr, kBackward);
  if (st != FA_OK) return st;
  fa::BwdParams p;
  st = bwd_params(&p, pr, workspace, workspace_bytes);
  if (st != FA_OK) return st;
  p.dq = dq;
  return fa::launch_bwd_post(pr.D, p, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

fa_status_t fa_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
                   const void* dout, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                   float softmax_scale, int causal, const int32_t* seqlens, float dropout_p,
                   uint64_t seed, const uint8_t* block_mask, void* workspace,
                   size_t workspace_bytes, void* stream) {
  if (seqlens != nullptr && !aligned(seqlens, 4)) return FA_ERR_INVALID_ARG;
  const fa_attention_desc_t a =
      classic_desc(B, H, N, d, softmax_scale, causal, seqlens, dropout_p, seed, block_mask);
  Problem pr;
  const fa_status_t st = resolve(&a, &pr, kBackward);
  if (st != FA_OK) return st;
  return run_bwd(pr, q, k, v, o, lse, dout, dq, dk, dv, workspace, workspace_bytes, stream);
}

fa_status_t fa_bwd_ex(const fa_attention_desc_t* desc, const void* q, const void* k,
                      const void* v, const void* o, const float* lse, const void* dout, void* dq,
                      void* dk, void* dv, void* workspace, size_t workspace_bytes, void* stream) {
  Problem pr;
  const fa_status_t st = resolve(desc, &pr, kBackward);
  if (st != FA_OK) return st;
  return run_bwd(pr, q, k, v, o, lse, dout, dq, dk, dv, workspace, workspace_bytes, stream);
}

fa_status_t fa_qkv_projection(const void* x, const void* w, const void* bias, void* q, void* k,
                              void* v, int B, int N, int H, int d, int d_model, void* stream) {
  if (!tensor_ok(x) || !tensor_ok(w) || !tensor_ok(q) || !tensor_ok(k) || !tensor_ok(v))
    return FA_ERR_INVALID_ARG;
  if (bias != nullptr && !aligned(bias, 16)) return FA_ERR_INVALID_ARG;
  if (B < 1 || N < 1 || H < 1 || d_model < 8 || d_model % 8) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if ((static_cast<int64_t>(H) * d) % 128) return FA_ERR_UNSUPPORTED;
  const int64_t T = static_cast<int64_t>(B) * N;
  if (T > 65535ll * 128 || static_cast<int64_t>(H) * d * 3 / 128 > 0x7FFFFFFF ||
      d_model > (1 << 24))
    return FA_ERR_UNSUPPORTED;
  int* status = status_word();
  if (status == nullptr) return FA_ERR_CUDA;
  const cudaError_t e = fa::launch_qkv_projection(x, w, bias, q, k, v, B, N, H, d, d_model, status,
                                                  g_timeout_ns.load(),
                                                  static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status_t fa_debug_dropout_mask(uint8_t* keep, int B, int H, int N, float dropout_p,
                                  uint64_t seed, void* stream) {
  if (keep == nullptr || B < 1 || H < 1 || N < 1) return FA_ERR_INVALID_ARG;
  if (!(dropout_p >= 0.f && dropout_p < 1.f)) return FA_ERR_INVALID_ARG;
  const Dropout dr = dropout_params(dropout_p);
  const cudaError_t e = fa::launch_dropout_mask(
      keep, B, H, N, dr.threshold, static_cast<uint32_t>(seed & 0xFFFFFFFFull),
      static_cast<uint32_t>(seed >> 32), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status_t fa_debug_wait_timeout(void* stream) {
  int* status = status_word();
  if (status == nullptr) return FA_ERR_CUDA;
  const cudaError_t e =
      fa::launch_wait_timeout_probe(status, g_timeout_ns.load(), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
