// kv.cuh -- what the paged cache's translation units share: host checks, the
// device view of a cache, and the layout of a plan.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "common.cuh"
#include "samspec.h"
#include "samspec_kv.h"

namespace samspec {

constexpr int kKvCtas = 152;   // persistent CTAs of kv_attend: one per SM of a GB300
constexpr int kRows = 128;     // query rows of a tile (a matrix instruction's)
constexpr int kTileRows = 256; // of a unit of attention work
constexpr int kKeyBlock = 128; // keys of one step of it

struct KvView {
  unsigned char* k;
  unsigned char* v;
  int32_t* table;
  int32_t* lens;
  int32_t* held;
  int32_t* refs;
  uint32_t* free_bits;
  int32_t layers, n_pages, page, log_page, kv_heads, head_dim, seqs, max_pages;
  int32_t elt;       // bytes of an element of k and v
  uint8_t* k_scale;  // of a cache of 8 bits
  uint8_t* v_scale;
};

// EINVAL / ESIZE / EDTYPE / EALIGN of a cache descriptor, else OK and its view
inline int kv_view(const kv_cache* c, KvView* o) {
  if (!c || !c->k || !c->v || !c->table || !c->lens || !c->held || !c->refs || !c->free_bits)
    return SAMSPEC_EINVAL;
  const bool eight = c->dtype == SAMSPEC_E4M3;
  if (!eight && c->dtype != SAMSPEC_BF16 && c->dtype != SAMSPEC_F16) return SAMSPEC_EDTYPE;
  if (eight && (!c->k_scale || !c->v_scale)) return SAMSPEC_EINVAL;
  if (eight && c->io_dtype != SAMSPEC_BF16 && c->io_dtype != SAMSPEC_F16) return SAMSPEC_EDTYPE;
  int lg = 4;
  while (lg < 8 && (1 << lg) != c->page) ++lg;
  if (lg == 8 || (c->head_dim != 64 && c->head_dim != 128)) return SAMSPEC_ESIZE;
  if (c->layers < 1 || c->n_pages < 1 || c->kv_heads < 1 || c->kv_heads > 1024 || c->seqs < 1 ||
      c->seqs > (1 << 20) || c->max_pages < 1 || c->max_pages > (1 << 20))
    return SAMSPEC_ESIZE;
  const int64_t lim = (int64_t)1 << 31;
  if ((int64_t)c->layers * c->n_pages >= lim || (int64_t)c->n_pages * c->kv_heads * c->page >= lim ||
      (int64_t)c->max_pages * c->page >= lim / 2)
    return SAMSPEC_ESIZE;
  if ((reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v)) % 16 != 0)
    return SAMSPEC_EALIGN;
  if (eight && (reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale)) % 16 != 0)
    return SAMSPEC_EALIGN;
  *o = {static_cast<unsigned char*>(c->k), static_cast<unsigned char*>(c->v), c->table, c->lens,
        c->held, c->refs, c->free_bits, c->layers, c->n_pages, c->page, lg, c->kv_heads,
        c->head_dim, c->seqs, c->max_pages, eight ? 1 : 2,
        eight ? static_cast<uint8_t*>(c->k_scale) : nullptr, eight ? static_cast<uint8_t*>(c->v_scale) : nullptr};
  return SAMSPEC_OK;
}
// the type of queries, new keys and values, and results
inline int32_t io_dtype(const kv_cache* c) { return c->dtype == SAMSPEC_E4M3 ? c->io_dtype : c->dtype; }

// the first slot of (layer, page, head) in a pool, which has a scale for each; its
// byte: page * head_dim elements follow.  64 bits: a pool passes 4 GB.
__host__ __device__ inline int64_t kv_slot(const KvView& c, int layer, int page, int head) {
  return (((int64_t)layer * c.n_pages + page) * c.kv_heads + head) * c.page;
}
__host__ __device__ inline int64_t kv_offset(const KvView& c, int layer, int page, int head) {
  return kv_slot(c, layer, page, head) * c.head_dim * c.elt;
}

// ---- a cache of 8 bits -------------------------------------------------------
// A code's bits s eeee mmm, moved into a 16-bit float's s and the low end of its
// exponent and mantissa, are its value times 2^-120 (bf16) or 2^-8 (fp16): the
// biases' difference, subnormal codes included.  One product with 2^(b - 127) times
// that puts it right, and rounds only where the type has no such value.  (cvt from
// e4m3 to fp16 has no bf16 form; by way of fp32 it would take 6 instructions a pair
// instead of 5.)  kScaleLow .. kScaleHigh keep that factor a number of the type.
constexpr int kScaleLow = 95, kScaleHigh = 134, kScaleNan = 255;
template <bool kBf16>
__device__ __forceinline__ uint32_t scale_word(uint32_t b) {
  const uint32_t x = min(max(b, (uint32_t)kScaleLow), (uint32_t)kScaleHigh);
  const uint32_t h = kBf16 ? (x + 120) << 7 : x >= 105 ? (x - 104) << 10 : 1u << (x - 95);
  return b == kScaleNan ? 0x7fff7fffu : h * 0x10001u;
}
template <bool kBf16>
__device__ __forceinline__ uint32_t expand_pair(uint32_t x, uint32_t scale) {  // x: a code in each half's upper byte
  const uint32_t y = kBf16 ? ((x >> 4) & 0x07f007f0u) : ((x >> 1) & 0x3f803f80u);
  uint32_t r = y | (x & 0x80008000u);
  if (kBf16) asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(scale));
  else asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(scale));
  return r;
}
// 16 codes to 16 values, in order
template <bool kBf16>
__device__ __forceinline__ void expand16(uint4 u, uint32_t scale, uint32_t* out) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    out[2 * k] = expand_pair<kBf16>(__byte_perm(w[k], 0, 0x1404), scale);
    out[2 * k + 1] = expand_pair<kBf16>(__byte_perm(w[k], 0, 0x3424), scale);
  }
}

// exclusive prefix sum over a block of 1024 threads; *total the block's sum.
// `part` is 32 words of shared memory.
__device__ __forceinline__ int block_scan(int v, int* part, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kFullMask, s, o);
    if (lane >= o) s += x;
  }
  __syncthreads();  // the last call's reads of part
  if (lane == 31) part[w] = s;
  __syncthreads();
  int q = part[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kFullMask, q, o);
    if (lane >= o) q += x;
  }
  const int before = w ? __shfl_sync(kFullMask, q, w - 1) : 0;
  *total = __shfl_sync(kFullMask, q, 31);
  return before + s - v;
}

// Programmatic dependent launch: a kernel may be started while the one before
// it in the stream still runs; nothing that one writes, or may still read, is
// touched before wait_for_previous().  (Launch gaps of about 2 us a kernel.)
// So the arguments of such kernels carry no __restrict__: with const it promises
// that what they point to does not change while the kernel runs, and allows loads
// that are not coherent, or moved before the wait.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <typename... A, typename... B>
cudaError_t launch_after(void (*kernel)(A...), unsigned grid, unsigned block, size_t smem, cudaStream_t s, B... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, A(args)...);
}
inline int launched() { return cudaGetLastError() == cudaSuccess ? SAMSPEC_OK : SAMSPEC_ECUDA; }

// ---- plan ------------------------------------------------------------------
// one sequence of the call
struct KvSeq {
  int32_t row;     // its row in the cache
  int32_t base;    // committed tokens
  int32_t ntok;    // new tokens (0: a status is set)
  int32_t leader;  // first sequence of its group that takes part (itself: none, or it takes none)
  int32_t lcp;     // tokens of the pages that it shares with the first that might
  int32_t shared;  // tokens that its group reads once (0: none; at every member that takes part)
  int32_t gsize;   // at the leader: sequences up to the last that takes part
  int32_t first;   // (of the plan's own)
};
// a unit of attention work, once for each key head: the queries of `toks`
// tokens (tokens of consecutive sequences follow one another, rep query heads
// each) against a range of keys.  Up to kRows / rep tokens make one tile of
// query rows, up to twice as many a unit of two.
struct KvTile {
  int32_t tok0, toks;  // first token of the call (i * N + node), how many
  int32_t two;         // two tiles of rows
  int32_t kbeg, kend;  // keys, in tokens
  int32_t ctx;         // every row sees the keys before this one; token t of a chain those before ctx + t
  int32_t seq_row;     // the cache row whose pages are read
  int32_t kind;        // 1: keys that the group shares, every row sees them all;
                       // 2: own keys of a sequence whose group shares others
  int32_t blocks;      // key blocks
  int32_t cost0;       // cost of all heads of the tiles before
  int32_t sinks;       // windows: every row sees the keys before this one; where kbeg > 0 their
                       // blocks come before those from kbeg on
  int32_t low;         // windows: not every row sees the keys before this one (0: no such keys)
};
// A unit's first blocks, of keys that stay visible before its window.
__host__ __device__ inline int sink_blocks(const KvTile& t) {
  return t.kbeg > 0 ? (t.sinks + kKeyBlock - 1) / kKeyBlock : 0;
}
// Block b of a unit: its first key.  (kWindow: of a plan with a window.)
template <bool kWindow>
__host__ __device__ inline int block_key(const KvTile& t, int b) {
  const int s = kWindow ? sink_blocks(t) : 0;
  return b < s ? b * kKeyBlock : t.kbeg + (b - s) * kKeyBlock;
}
// The key behind its last: block b's own (of the keys before `sinks`, where
// they have blocks), or the unit's.
template <bool kWindow>
__host__ __device__ inline int block_end(const KvTile& t, int b) {
  return kWindow && b < sink_blocks(t) ? t.sinks : t.kend;
}
// a unit that was cut among CTAs: at the CTA behind its first part's
struct KvJoin {
  int32_t tok0, toks;  // its tokens (0: no unit is first cut here)
  int32_t head, parts;
  int32_t first, rest;  // where its first part's rows lie, and the second's; the others 2 * slot_rows apart
  int32_t pad[2];
};
inline __host__ __device__ int tile_tokens(int rep) { return kRows / rep; }
// Do a pass's units have few enough rows for attend_few_kernel?  Its time goes by the
// rows, attend_kernel's hardly up to 128.  64 sequences of 4096 8-bit keys and 8 key heads of
// 128 (64) elements, us a call, L2 flushed before it: 16 rows 119 (90), by attend_kernel 197
// (145); 32 rows 150 (122), by attend_kernel 199 (147); 64 rows, by attend_kernel, 205
// (150), where an earlier attend_few_kernel took 351 (309).  In windows of 1024 keys 32 rows
// take 119, by attend_kernel 111, but 16 take 78 and 107.
inline bool few_rows(const KvView& c, int N, int rep, bool grouped) {
  return c.elt == 1 && !grouped && (int64_t)N * rep <= 32;
}
enum { kHdrCtas = 1, kHdrCost = 2, kHdrTree = 3, kHdrInts = 16 };

struct PlanLayout {
  size_t status, hdr, seq, node, suf0, pre0, tile, start, join, ml, o, bytes;
  int32_t max_tiles;
  int32_t slot_rows;  // rows of a cut unit's part
  int64_t store;      // rows of each of the two stores of whole units (grouped plans)
  int64_t part_rows;  // rows of partial results: two per CTA, then the stores
};

inline size_t kv_align(size_t x) { return (x + 255) / 256 * 256; }

// 0 bytes where the sizes are outside the limits
inline PlanLayout plan_layout(const KvView& c, int32_t n, int32_t N, int32_t q_heads, bool grouped) {
  PlanLayout p = {};
  if (n < 1 || n > (1 << 20) || N < 1 || N > (1 << 16) || q_heads < 1 || q_heads % c.kv_heads != 0 ||
      q_heads / c.kv_heads > 64 || (int64_t)n * N * q_heads >= ((int64_t)1 << (grouped ? 29 : 30)))
    return p;
  const int64_t rep = q_heads / c.kv_heads;
  const int64_t unit = 2 * tile_tokens((int)rep);  // tokens
  const int64_t suf = (N + unit - 1) / unit * n;
  const int64_t pre = grouped ? ((int64_t)n * N + unit - 1) / unit + n : 0;
  // costs are counted in 32 bits
  const int64_t blocks = ((int64_t)c.max_pages * c.page / kKeyBlock + 2) * 2 + 5;
  if ((suf + pre) * blocks * c.kv_heads >= ((int64_t)1 << 31)) return p;
  p.max_tiles = (int32_t)(suf + pre);
  p.store = grouped ? (int64_t)n * N * q_heads : 0;
  // a unit's rows: its first tile's from 0 on, its second's from kRows
  p.slot_rows = grouped || N > unit / 2 ? kTileRows : (int32_t)(N * rep);
  p.part_rows = (int64_t)2 * kKvCtas * p.slot_rows + 2 * p.store;
  size_t at = 0;
  auto take = [&](size_t bytes) { const size_t o = at; at = kv_align(at + bytes); return o; };
  p.status = take(4 * (size_t)n);
  p.hdr = take(4 * kHdrInts);
  p.seq = take(sizeof(KvSeq) * n);
  p.node = take(N <= 32 ? 8 * (size_t)n * N : 0);
  p.suf0 = take(4 * (size_t)n);
  p.pre0 = take(4 * (size_t)n);
  p.tile = take(sizeof(KvTile) * (size_t)p.max_tiles);
  p.start = take(16 * (kKvCtas + 1));
  p.join = take(sizeof(KvJoin) * kKvCtas);
  p.ml = take(8 * (size_t)p.part_rows);
  p.o = take(4 * (size_t)p.part_rows * c.head_dim);
  p.bytes = at;
  return p;
}

struct PlanView {
  int32_t* status;
  int32_t* hdr;
  KvSeq* seq;
  int2* node;      // depth, visible nodes (trees)
  int32_t* suf0;   // first tile of a sequence's own keys
  int32_t* pre0;   // first tile of a group's shared keys (at the leader)
  KvTile* tile;
  int4* start;     // where each CTA's share begins: tile, head, block; and the plan's window
  KvJoin* join;    // the cut units (plans without groups)
  float2* ml;      // partial results: running maximum (base 2) and sum ...
  float* o;        // ... and the sums of p v
  int32_t slot_rows;
  int64_t store;
};
inline PlanView plan_view(void* d_plan, const PlanLayout& p) {
  unsigned char* b = static_cast<unsigned char*>(d_plan);
  return {reinterpret_cast<int32_t*>(b + p.status), reinterpret_cast<int32_t*>(b + p.hdr),
          reinterpret_cast<KvSeq*>(b + p.seq),      reinterpret_cast<int2*>(b + p.node),
          reinterpret_cast<int32_t*>(b + p.suf0),   reinterpret_cast<int32_t*>(b + p.pre0),
          reinterpret_cast<KvTile*>(b + p.tile),    reinterpret_cast<int4*>(b + p.start),
          reinterpret_cast<KvJoin*>(b + p.join),    reinterpret_cast<float2*>(b + p.ml),
          reinterpret_cast<float*>(b + p.o),        p.slot_rows,
          p.store};
}

}  // namespace samspec
