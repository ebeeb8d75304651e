// attend_few.cu -- attention over a cache of 8 bits for units of up to 32 query rows
// (a decode step: N * rep of them), where HBM is to be the bound.
#include "attend.cuh"

namespace samspec {
namespace {

// Codes go to the matrix unit as they are; the keys stand for the rows of its tiles,
// and the queries for the columns, of which there are few:
//
//   S^T = K Q^T     [128 keys, rows]: K as it lies in its pages
//   O^T += V^T P^T  [D, rows]: V as it lies in its pages
//
// e4m3 has four significant bits, queries and weights have 8 or 11, so those are sums
// of parts: x = x0 + x1 / 16 (+ x2 / 256), each the nearest code to 16 times what is
// left by the one before.  Two parts are a bf16 number, three an fp16 one, exactly but
// for half a step of the last part, 2^-14 (2^-18), where a head's largest has a code of
// at least 224.  Parts are columns of their own, added up in fp32.
//
// Weights (times their value's scale) become parts too, each off by 2^-8 (2^-11 in fp16,
// as they pass through it) of itself; or, of small ones, by what the last part's smallest
// step leaves, 2^-13 (2^-17).  Were small weights rounded to the nearest, all keys with
// like scores would be off the same way, and their errors add up while the sum that
// divides has them in full: one key with 2^20 times the weight of 131072 others, and
// those came out 11% short.  So a number that runs evenly through a step from key to key
// is added before the last rounding (in place of the product that it follows, a fused one:
// no instruction), and another before that to fp16, whose smallest step is 2^-24: each
// weight goes up as often as it has parts of a step, and errors of n keys add up like
// sqrt(n) of them, without a direction.
//
// A thread has a key: the key's two scales are its own, its scores are R numbers.  Weights
// are 2^(s + c) for a row's reference c, moved only when a weight would pass 2^8.5: then
// (all rows for the first block, later single ones) the warpgroup takes those rows'
// maxima, and what is there is scaled.  Where they are put: high, and small weights have
// more steps left; low, and fewer maxima to come move the reference (2500 clocks; a call,
// L2 flushed before it, over 64 sequences of 4096 keys with 32 rows of random queries:
// always at 2^8 222 us, at 2^6 169, at 2^4 150; fp16, 32 sequences of 16k to 32k keys,
// 232 at 2^8, 197 at 2^6, 159 at 2^4, 140 at 2^2).  A row whose four warps' maxima lie
// together has many keys to share its weight, and can have it low; where they lie apart
// one key may have all of it, few are still to exceed it, and it goes high.  Else a step
// needs one vote of 128 threads.  The values' scale multiplies the weights on their way
// to the product, not those of the sum.
//
// Two streams of steps, blocks in turn, as in attend_kernel; warps 8 and 12 load keys
// with the scales, and values (one warp for both, or the scales with a warp of their
// own: no faster), warps 9 and 10 issue the two products (one thread for both takes
// 1800 clocks a step, most of them its waits and addresses), warp 11 splits the next
// unit's queries into parts.  Scores and weights have kS places, scores are computed as
// far ahead, into the next unit too: a stream's chain is its softmax alone.
//
// What bounds it.  A block is 128 keys * (D + 1) * 2 bytes: at D 128 1400 clocks of an
// SM's share of HBM.  64 sequences of 4096 keys, 8 heads of 128, 16 rows: 100 us for this
// kernel, 5.4 TB/s of 6.8; the rest are units' starts and ends.  At D 64 a block comes in
// 700 clocks, and fp16 has three parts to make: 32 sequences of 16k to 32k keys, 4 heads
// of 64, 32 rows: 124 us for it, 3.2 TB/s.  There the softmax bounds it, of 128 * 32
// weights a block at 10 instructions each: half of the issue slots are taken, and a warp
// that could issue waits for its instructions as often as not (the loops' code is 30 KB).
constexpr float kReach = 8.5f;  // log2 of the largest weight (e4m3 has 448)
constexpr float kEven = 4.f;    // how far apart (log2) maxima of 32 keys may lie for a reference put low
constexpr int kMaxStages = 12;

struct FewRow {
  int32_t lim, low;  // the keys that it sees: before lim, of a window those from low on
  uint32_t see;      // and a tree's nodes
  int32_t pad;
};
template <int R>
struct FewCtl {
  uint64_t k_full[kMaxStages], v_full[kMaxStages], k_empty[kMaxStages], v_empty[kMaxStages];
  uint64_t s_full[4], p_full[4], p_free[4], q_full[2], q_empty[2], o_free, drain;
  uint32_t tmem;
  int32_t abort;
  int32_t asked_k, asked_v;  // tiles that the loader has requested, once it has ended
  Segment seg[2];
  alignas(16) FewRow row[2][R];
  alignas(16) float scale[2][R];  // of the rows' parts, times the scores'
  int32_t to[2][R];              // a row's place among the unit's in the output
  alignas(16) float c[2][R];     // the streams' references
  alignas(16) float by[2][R];    // by how much they have moved
  alignas(16) float move[2][R];  // what that makes of earlier weights; at the end the streams' factors
  alignas(16) float red[2][4][R];
  uint32_t bits[2][4];  // rows that a warp finds to move; [0] then those that have
};
template <typename T, int D, int R>
struct Few {
  static constexpr int kParts = Type16<T>::kFormat == 1 ? 2 : 3;
  static constexpr int kCols = kParts * R;  // columns of both products
  // log2 of a row's largest weight when its reference is set
  static constexpr float kTopLow = kParts == 2 ? 4.f : 2.f, kTopHigh = 8.f;
  static_assert(R == 16 || R == 32, "a row a bit, a lane's sum");
  static constexpr int kS = 512 / kCols - 2 < 4 ? 512 / kCols - 2 : 4;  // places of scores, and of weights
  static constexpr int kTile = 128 * D, kScales = 2 * kKeyBlock;
  static constexpr int kQ = kCols * D, kP = 128 * kCols;
  static constexpr int kRest = 2 * kQ + kS * kP + (int)((sizeof(FewCtl<R>) + 127) / 128 * 128);
  static constexpr int kFit = (232448 - kRest) / (2 * kTile + kScales);
  static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
  // from a 1024-byte boundary: a stage's keys and values, the stages' scales, ...
  static constexpr int kScale0 = kStages * 2 * kTile, kQ0 = kScale0 + kStages * kScales, kP0 = kQ0 + 2 * kQ,
                       kCtl = kP0 + kS * kP, kBytes = kCtl + (int)((sizeof(FewCtl<R>) + 127) / 128 * 128);
  static_assert(kBytes <= 232448 && kStages >= 3, "227 KB of a CTA");
};

// Matrix descriptors: address and strides in units of 16 bytes.
__device__ __forceinline__ uint64_t matrix(const void* p, uint32_t lead, uint32_t stride, uint32_t layout) {
  const uint32_t lo = (smem_u32(p) >> 4) | (lead >> 4) << 16, hi = (stride >> 4) | (1u << 14) | layout << 29;
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t further(uint64_t matrix, uint32_t bytes) { return matrix + (bytes >> 4); }
__device__ __forceinline__ void mma_codes(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t addr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tmem_wait_ld8(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_ld1(uint32_t addr, uint32_t& r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_wait_ld1(uint32_t& r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r) : : "memory");
}
__device__ __forceinline__ void tmem_st1(uint32_t addr, uint32_t r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%1], {%0};" ::"r"(r), "r"(addr) : "memory");
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float warp_max(float v) {  // NaN only where all are
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}
// fp16 pairs and codes
__device__ __forceinline__ uint32_t half_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint16_t code_pair(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t code_values(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
// 16 times what a pair of codes leaves of a pair (exact), and `more` besides
__device__ __forceinline__ uint32_t left16(uint32_t h, uint16_t c, uint32_t more) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(code_values(c)));
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(r), "r"(0x4c004c00u), "r"(more));
  return r;
}
// What key `th` of a unit's block b adds to a weight before it is rounded: of a step of
// size 1 a number in (-1/2, 1/2), 11 bits and none of them 1/2, so that a weight of zero
// stays one.  A block's 128 keys have 128 numbers evenly apart, in an order (by `turn`, odd)
// in which any few neighbours lie well apart too, and all move on from block to block (by
// `shift`).  The two that a weight meets go by 1 / g and 1 / g^2, g^3 = g + 1, of 128 and of
// 2^16, whose multiples fill a square evenly, not only a line.
__device__ __forceinline__ float dither(int th, int b, uint32_t turn, uint32_t shift) {
  return (float)(int)(((uint32_t)th * (turn << 9) + (uint32_t)b * shift) >> 5 & 2047) * 0x1p-11f - 0.5f + 0x1p-12f;
}

// Values of key `row` of a block that not every query sees: zeros where it is no key of
// the unit; and no NaN, since 0 * NaN would reach the queries that do not see it.
template <int D>
__device__ __forceinline__ void clean_row(unsigned char* tile, int row, bool none) {
  const int turn = D == 128 ? row & 7 : (row >> 1) & 3;
  uint4* at = reinterpret_cast<uint4*>(tile + row * D);
#pragma unroll 2
  for (int p = 0; p < D / 16; ++p) {
    uint4 u = none ? uint4{0, 0, 0, 0} : at[p ^ turn];
    uint32_t* a = reinterpret_cast<uint32_t*>(&u);
    bool hit = none;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t nan = ((a[k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
      hit |= nan != 0;
      a[k] &= ~((nan >> 7) * 0xffu);
    }
    if (hit) at[p ^ turn] = u;
  }
  fence_async_smem();
}

// A unit's queries as parts: columns part * R + row, 16 bytes of them beside one another.
// A warp, D / 8 lanes to a row.  `scale` gets each row's.
template <typename T, int D, int R>
__device__ __forceinline__ void split_queries(const AttendParams& P, const KvTile& t, int head, unsigned char* q,
                                              float* scale, int th) {
  using F = Few<T, D, R>;
  using H = Type16<T>;
  constexpr int kVec = D / 8, kStep = 32 / kVec;
  const int rows = t.toks * P.rep, e = th % kVec;
#pragma unroll 2
  for (int r0 = 0; r0 < R; r0 += kStep) {
    const int r = r0 + th / kVec, lt = P.rep_div(r);
    uint4 u = {0, 0, 0, 0};
    if (r < rows)
      u = *reinterpret_cast<const uint4*>(
          P.q + (((int64_t)t.tok0 + lt) * P.q_stride + (int64_t)(head * P.rep + r - lt * P.rep) * D + e * 8) * 2);
    const uint32_t a[4] = {u.x, u.y, u.z, u.w};
    float x[8];
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = H::lo(a[k]);
      x[2 * k + 1] = H::hi(a[k]);
      top = max(top, max(__float_as_uint(x[2 * k]) & 0x7fffffffu, __float_as_uint(x[2 * k + 1]) & 0x7fffffffu));
    }
#pragma unroll
    for (int o = 1; o < kVec; o <<= 1) top = max(top, __shfl_xor_sync(kFullMask, top, o));
    // the smallest power of two of which 448 times is not exceeded
    const int ex = max((int)(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u), -126);
    const float inv = __uint_as_float((uint32_t)(127 - ex) << 23);
    if (e == 0)
      scale[r] = top >= 0x7f800000u ? NAN : P.scale_log2 * __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] *= inv;
#pragma unroll
    for (int p = 0; p < F::kParts; ++p) {
      uint32_t w[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[4 * k + 1]), "f"(x[4 * k]));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[4 * k + 3]), "f"(x[4 * k + 2]));
        w[k] = lo | (uint32_t)hi << 16;
        const float2 b0 = __half22float2(*reinterpret_cast<const __half2*>(&(const uint32_t&)code_values(lo)));
        const float2 b1 = __half22float2(*reinterpret_cast<const __half2*>(&(const uint32_t&)code_values(hi)));
        x[4 * k] = (x[4 * k] - b0.x) * 16.f;
        x[4 * k + 1] = (x[4 * k + 1] - b0.y) * 16.f;
        x[4 * k + 2] = (x[4 * k + 2] - b1.x) * 16.f;
        x[4 * k + 3] = (x[4 * k + 3] - b1.y) * 16.f;
      }
      *reinterpret_cast<uint2*>(q + (e / 2 * F::kCols + p * R + r) * 16 + (e & 1) * 8) = uint2{w[0], w[1]};
    }
  }
}

// R numbers of each lane, summed over the warp: row r's sum in lane r (R 32), or lanes
// 2r and 2r + 1 (R 16).
template <int R>
__device__ __forceinline__ void sum_rows(float* l, int lane) {
  int o = 16;
#pragma unroll
  for (int n = R; n > 1; n >>= 1, o >>= 1) {
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float send = lane & o ? l[i] : l[i + n / 2], keep = lane & o ? l[i + n / 2] : l[i];
      l[i] = keep + __shfl_xor_sync(kFullMask, send, o);
    }
  }
  if (R == 16) l[0] += __shfl_xor_sync(kFullMask, l[0], 1);
}

// The keys of a CTA's blocks with the scales, or their values.
template <typename T, int D, int R, bool kWindow, bool kValues>
__device__ __forceinline__ void load_blocks(const AttendParams& P, unsigned char* smem, const CUtensorMap& map,
                                         int lane) {
  using F = Few<T, D, R>;
  FewCtl<R>* ctl = reinterpret_cast<FewCtl<R>*>(smem + F::kCtl);
  const KvView& c = P.c;
  uint64_t* const full = kValues ? ctl->v_full : ctl->k_full;
  uint64_t* const empty = kValues ? ctl->v_empty : ctl->k_empty;
  unsigned char* const to = smem + (kValues ? F::kTile : 0) + lane * c.page * D;
  unsigned char* const scales = smem + F::kScale0 + lane * c.page;
  int asked = 0, st = 0, par = 1;
  bool ok = true;
#pragma unroll 1
  for (Walk wk(P, kWindow); ok && wk.more(); wk.next(P)) {
    Pages<kWindow> of(c, wk.t);
    const int x = P.layer * c.n_pages, y = wk.head;
#pragma unroll 1
    for (int b = 0; b < wk.nb; ++b) {
      const int page = of.of(c, wk.t, wk.blk + b, lane);
      const int pages = __popc(__ballot_sync(kFullMask, page >= 0));
      ok = __all_sync(kFullMask, wait_for(&empty[st], par, ctl, P.wait_ns));
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)(pages << c.log_page) * (kValues ? D : D + 2));
      __syncwarp();
      if (page >= 0) {
        tma_load3(to + st * 2 * F::kTile, &map, 0, y << c.log_page, x + page, &full[st]);
        if (!kValues) {
          // (16 to 128 bytes: a tensor's copy would want its place on a 128-byte boundary)
          const int64_t slot = kv_slot(c, P.layer, page, wk.head);
          bulk_g2s(scales + st * F::kScales, c.k_scale + slot, c.page, &full[st]);
          bulk_g2s(scales + st * F::kScales + kKeyBlock, c.v_scale + slot, c.page, &full[st]);
        }
      }
      ++asked;
      if (++st == F::kStages) st = 0, par ^= 1;
    }
  }
  if (lane == 0) (kValues ? ctl->asked_v : ctl->asked_k) = asked;
}

template <typename T, int D, int R, bool kWindow>
__global__ void __launch_bounds__(512, 1)
    attend_few_kernel(const __grid_constant__ AttendParams P, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v) {
  using F = Few<T, D, R>;
  using H = Type16<T>;
  extern __shared__ __align__(1024) unsigned char smem[];
  FewCtl<R>* ctl = reinterpret_cast<FewCtl<R>*>(smem + F::kCtl);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (smem_u32(smem) & 1023) {  // (as in attend_kernel)
    wait_for_previous();
    let_next_start();
    for (int i = blockIdx.x * 512 + tid; i < P.n; i += kKvCtas * 512) P.plan.status[i] = SAMSPEC_ST_TIMEOUT;
    return;
  }
  if (warp == 9) tmem_alloc(&ctl->tmem, 512);
  if (tid == 0) {
    for (int s = 0; s < F::kStages; ++s) {
      mbar_init(&ctl->k_full[s], 1);
      mbar_init(&ctl->v_full[s], 1);
      mbar_init(&ctl->k_empty[s], 4);
      mbar_init(&ctl->v_empty[s], 1);
    }
    for (int w = 0; w < 4; ++w) {
      mbar_init(&ctl->s_full[w], 1);
      mbar_init(&ctl->p_full[w], 4);
      mbar_init(&ctl->p_free[w], 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&ctl->q_full[w], 1);
      mbar_init(&ctl->q_empty[w], 8);
    }
    mbar_init(&ctl->o_free, 8);
    mbar_init(&ctl->drain, 2);
    ctl->abort = 0;
    mbar_fence_init();
  }
  tc_fence_before();
  wait_for_previous();
  let_next_start();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  const uint32_t tO = tmem + 512 - 2 * F::kCols;  // the streams' sums, behind the scores
  constexpr uint32_t kLayout = D == 128 ? 2 : 4;  // 128- or 64-byte swizzle of keys and values
  constexpr uint32_t kGroup = 8 * D;              // bytes of 8 of them

  // registers: 512 * 128 at launch = 256 * 200 + 256 * 56
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 8 || warp >= 12) {
      // ---- pages ----
      if (warp == 8) load_blocks<T, D, R, kWindow, false>(P, smem, map_k, lane);
      else if (warp == 12) load_blocks<T, D, R, kWindow, true>(P, smem, map_v, lane);
    } else if (warp == 9) {
      // ---- scores ----
      if (lane == 0) {
        const uint32_t id = (1u << 4) | ((128 >> 4) << 24) | ((F::kCols >> 3) << 17);
        const uint64_t k0 = matrix(smem, 16, kGroup, kLayout), q0 = matrix(smem + F::kQ0, F::kCols * 16, 128, 0);
        bool ok = true, last = !Walk(P, kWindow).more();
        int st = 0, par = 0, at = 0, at_par = 1;  // the step's stage and place, with their phases
#pragma unroll 1
        for (int seg = 0; ok && !last; ++seg) {
          ok = wait_for(&ctl->q_full[seg & 1], (seg >> 1) & 1, ctl, P.wait_ns);
          if (!ok) break;
          const int nb = ctl->seg[seg & 1].nb;
          last = ctl->seg[seg & 1].last;
          const uint64_t q = further(q0, (seg & 1) * F::kQ);
#pragma unroll 1
          for (int x = 0; ok && x < nb; ++x) {
            // The step that had the place is done, its product with the values too: the
            // place of its weights is free as well, and who waits for these scores need not ask.
            ok = wait_for(&ctl->p_free[at], at_par, ctl, P.wait_ns);
            ok = ok && wait_for(&ctl->k_full[st], par, ctl, P.wait_ns);
            if (!ok) break;
            tc_fence_after();
            const uint64_t k = further(k0, st * 2 * F::kTile);
#pragma unroll
            for (int e = 0; e < D / 32; ++e)  // 32 elements along a row
              mma_codes(tmem + at * F::kCols, further(k, e * 32), further(q, e * 2 * F::kCols * 16), id, e > 0);
            mma_commit(&ctl->s_full[at]);
            if (++st == F::kStages) st = 0, par ^= 1;
            if (++at == F::kS) at = 0, at_par ^= 1;
          }
        }
      }
      __syncwarp();
    } else if (warp == 10) {
      // ---- weights times values ----
      if (lane == 0) {
        const uint32_t across = (1u << 15) | (1u << 16);  // both operands
        const uint32_t id = (1u << 4) | ((128 >> 4) << 24) | ((F::kCols >> 3) << 17) | across;
        const uint64_t v0 = matrix(smem + F::kTile, kGroup, kGroup, kLayout), p0 = matrix(smem + F::kP0, 128, 2048, 0);
        bool ok = true, last = !Walk(P, kWindow).more();
        int st = 0, par = 0, at = 0, at_par = 0;  // the step's stage, and its weights' place
        uint32_t to = 0;
#pragma unroll 1
        for (int seg = 0; ok && !last; ++seg) {
          ok = wait_for(&ctl->q_full[seg & 1], (seg >> 1) & 1, ctl, P.wait_ns);
          if (!ok) break;
          const int nb = ctl->seg[seg & 1].nb;
          last = ctl->seg[seg & 1].last;
#pragma unroll 1
          for (int x = 0; ok && x < nb; ++x, to ^= F::kCols) {
            ok = wait_for(&ctl->p_full[at], at_par, ctl, P.wait_ns);
            ok = ok && wait_for(&ctl->v_full[st], par, ctl, P.wait_ns);
            // the last unit's O has to be read before this one's begins
            if (x == 0 && seg > 0) ok = ok && wait_for(&ctl->o_free, (seg - 1) & 1, ctl, P.wait_ns);
            if (!ok) break;
            tc_fence_after();
            const uint64_t v = further(v0, st * 2 * F::kTile), p = further(p0, at * F::kP);
#pragma unroll
            for (int k = 0; k < 4; ++k)  // 32 keys; (at D 64 the tile's upper 64 rows are others' values, unused)
              mma_codes(tO + to, further(v, k * 4 * kGroup), further(p, k * 512), id, x >= 2 || k > 0);
            mma_commit(&ctl->v_empty[st]);
            mma_commit(&ctl->p_free[at]);
            if (++st == F::kStages) st = 0, par ^= 1;
            if (++at == F::kS) at = 0, at_par ^= 1;
          }
        }
      }
      __syncwarp();
    } else {
      // ---- queries ----
      const int th = lane;
      const bool tree = P.plan.hdr[kHdrTree] != 0;
      bool ok = true;
      int seg = 0;
#pragma unroll 1
      for (Walk wk(P, kWindow); ok && wk.more(); wk.next(P), ++seg) {
        ok = __all_sync(kFullMask, wait_for(&ctl->q_empty[seg & 1], ((seg >> 1) & 1) ^ 1, ctl, P.wait_ns));
        if (!ok) break;
        if (th == 0) ctl->seg[seg & 1] = {wk.t, wk.head, wk.blk, wk.nb, wk.final_one(P)};
        FewRow* info = ctl->row[seg & 1];
#pragma unroll 1
        for (int r = th; r < R; r += 32) {
          const int lt = P.rep_div(r);
          int lim = wk.t.kend, low = 0;
          uint32_t see = 0;
          if (lt < wk.t.toks) {
            if (tree) {
              const int2 node = P.plan.node[wk.t.tok0 + lt];
              see = (uint32_t)node.y;
              lim = wk.t.ctx - 1;
              low = wk.t.ctx + node.x - wk.window;
            } else {
              lim = min(lim, wk.t.ctx + lt);
              low = wk.t.ctx + lt - wk.window;
            }
          }
          ctl->to[seg & 1][r] = lt * P.q_heads + r - lt * P.rep;
          info[r].lim = lim;
          info[r].low = low;
          info[r].see = see;
        }
        split_queries<T, D, R>(P, wk.t, wk.head, smem + F::kQ0 + (seg & 1) * F::kQ, ctl->scale[seg & 1], th);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->q_full[seg & 1]);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ---- softmax ----  (a thread that gives up: as in attend_kernel)
    const int w = warp >> 2, th = tid & 127;  // stream; the key of a block
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t mO = tO + F::kCols * w + lanes;
    bool last, ok = true;
    {
      const Walk share(P, kWindow);
      last = !share.more();
      if (share.other && blockIdx.x == 0)
        for (int i = tid; i < P.n; i += 256) P.plan.status[i] = SAMSPEC_ST_BADPARAM;
    }
    int g0 = 0, seg = 0;  // steps and segments before
    // this stream's next step (every second one): its stage and the place of its scores and
    // weights, with their phases; and the place before
    int st = w, st_par = 0, at = w, at_par = 0, was = 0, was_par = 0;
    auto next_segment = [&](int s) {
      const bool came = wait_for(&ctl->q_full[s & 1], (s >> 1) & 1, ctl, P.wait_ns);
      return !named_any(4, 256, !came);
    };
    if (th < R) ctl->c[w][th] = 0.f;
    if (!last) ok = next_segment(0);
#pragma unroll 1
    for (; ok && !last; ++seg) {
      const Segment& sg = ctl->seg[seg & 1];
      const FewRow* info = ctl->row[seg & 1];
      const float* scale = ctl->scale[seg & 1];
      const int items = sg.nb, rows = sg.t.toks * P.rep;
      const int x0 = (w - g0) & 1;  // this stream's first step of the segment
      const int first = sg.blk - (kWindow ? sink_blocks(sg.t) : 0);
      const int before = sg.t.ctx - sg.t.kbeg - first * kKeyBlock;
      const int x_edge = before > 0 ? before / kKeyBlock : 0;
      const int x_low = kWindow && sg.t.low > 0 ? (sg.t.low - sg.t.kbeg + kKeyBlock - 1) / kKeyBlock - first : 0;
      // sums; up to 16 rows' scales and references are held, more are read in each step (held for
      // 32, 64-wide heads over 16k-32k keys took 191 us a call where they took 175 read)
      constexpr int kHeld = R <= 16 ? R : 1;
      float l[R], sr[kHeld], cr[kHeld];
      uint32_t unset = first_bits(rows);  // rows without a reference
#pragma unroll
      for (int r = 0; r < R; ++r) l[r] = 0.f;
      // (rows behind the unit's have queries and scales of zero: finite scores, no reference)
      if constexpr (R <= 16) {
#pragma unroll
        for (int r = 0; r < R; r += 4) {
          *reinterpret_cast<float4*>(sr + r) = *reinterpret_cast<const float4*>(scale + r);
          *reinterpret_cast<float4*>(cr + r) = float4{0.f, 0.f, 0.f, 0.f};
        }
      }
#pragma unroll 1
      for (int x = x0; x < items; x += 2) {
        const bool edge = x >= x_edge || (kWindow && x < x_low);
        if (ok) ok = wait_for(&ctl->s_full[at], at_par, ctl, P.wait_ns);
        if (ok) ok = wait_for(&ctl->k_full[st], st_par, ctl, P.wait_ns);  // (the scales)
        ok = __all_sync(kFullMask, ok);
        tc_fence_after();
        float ks = 1.f, vs = 1.f, ve = 0.f;  // this key's scales; the values' exponent
        if (ok) {
          const unsigned char* scales = smem + F::kScale0 + st * F::kScales + th;
          const int kb = scales[0], vb = scales[kKeyBlock];
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->k_empty[st]);  // (its product is done too)
          const int k1 = min(max(kb, kScaleLow), kScaleHigh), v1 = min(max(vb, kScaleLow), kScaleHigh);
          // (a head of NaN makes the weights of the rows that see it NaN)
          ks = kb == kScaleNan || vb == kScaleNan ? NAN : __uint_as_float((uint32_t)k1 << 23);
          vs = __uint_as_float((uint32_t)v1 << 23);
          ve = (float)(v1 - 127);
        }
        uint32_t vis = 0xffffffffu;  // rows that see the key
        const int b = sg.blk + x;
        if (edge) {
          const int key = block_key<kWindow>(sg.t, b) + th, d = key - (sg.t.ctx - 1);
          vis = 0;
#pragma unroll 1
          for (int r = 0; r < rows; r += P.rep) {  // a token's rows see alike
            const FewRow ri = info[r];
            if ((key < ri.lim && (!(kWindow && x < x_low) || key >= ri.low || key < sg.t.sinks)) ||
                ((unsigned)d < 32 && ((ri.see >> d) & 1)))
              vis |= first_bits(r + P.rep) & ~first_bits(r);
          }
        }
        const uint32_t mS = tmem + at * F::kCols + lanes;
        unsigned char* pw = smem + F::kP0 + at * F::kP + th * 16;
        const uint64_t ks2 = pack2(ks, ks), vs2 = pack2(vs, vs), part2 = pack2(0.0625f, 0.0625f);
        const float d_half = dither(th, b, 73, 37345) * 0x1p-24f, d_code = dither(th, b, 97, 49471) * 0x1p-9f;
        const uint64_t by_half = pack2(d_half, d_half);
        const uint32_t by_code = half_pair(d_code, d_code);
        float s[R];
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < R; i += 16) {
          uint32_t a[F::kParts][16];
#pragma unroll
          for (int p = 0; p < F::kParts; ++p) tmem_ld16(mS + p * R + i, a[p]);
#pragma unroll
          for (int p = 0; p < F::kParts; ++p) tmem_wait_ld16(a[p]);
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const int r = i + e;
            uint64_t v = pack2(__uint_as_float(a[F::kParts - 1][e]), __uint_as_float(a[F::kParts - 1][e + 1]));
#pragma unroll
            for (int p = F::kParts - 2; p >= 0; --p)
              v = fma2(v, part2, pack2(__uint_as_float(a[p][e]), __uint_as_float(a[p][e + 1])));
            float2 f, c2;
            if constexpr (R <= 16) {
              f = {sr[r], sr[r + 1]};
              c2 = {cr[r], cr[r + 1]};
            } else {
              f = *reinterpret_cast<const float2*>(scale + r);
              c2 = *reinterpret_cast<const float2*>(ctl->c[w] + r);
            }
            const float2 z = unpack2(fma2(mul2(v, ks2), pack2(f.x, f.y), pack2(c2.x, c2.y)));
            s[i + e] = z.x;
            s[i + e + 1] = z.y;
          }
        }
        if (edge) {
#pragma unroll
          for (int e = 0; e < R; ++e)
            if (!((vis >> e) & 1)) s[e] = -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < R; e += 2) mx = max3(mx, s[e], s[e + 1]);
        const bool start = x == x0;  // (no vote: all of them are to be set)
        if (start || named_any(1 + w, 128, !ok || unset || mx + ve > kReach)) {
          // references are set or moved: of which rows, ...
          uint32_t want = first_bits(R);
          if (!start) {
            want = 0;
#pragma unroll
            for (int e = 0; e < R; ++e)
              if (s[e] + ve > kReach) want |= 1u << e;
            want = __reduce_or_sync(kFullMask, want) | unset;
            if (lane == 0) ctl->bits[w][warp & 3] = want;
            named_sync(1 + w, 128);
            want = ctl->bits[w][0] | ctl->bits[w][1] | ctl->bits[w][2] | ctl->bits[w][3];
          }
          // ... their maxima over the block, ...
          float top = -INFINITY;
#pragma unroll
          for (int e = 0; e < R; ++e)
            if ((want >> e) & 1) {
              const float m = warp_max(s[e] + ve);
              if (lane == e) top = m;
            }
          if (lane < R) ctl->red[w][warp & 3][lane] = top;
          named_sync(1 + w, 128);
          if (th < 32) {
            bool move = false;
            if (lane < R) {
              float a[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) a[k] = ctl->red[w][k][lane];
              const float m = fmaxf(max3(a[0], a[1], a[2]), a[3]);
              move = m > -INFINITY && (((unset >> lane) & 1) || m > kReach);
              const float apart = m - fminf(fminf(a[0], a[1]), fminf(a[2], a[3]));
              const float by = move ? fminf(F::kTopLow + fmaxf(apart - kEven, 0.f), F::kTopHigh) - m : 0.f;
              // (a row that is set for the first time has no earlier weights)
              ctl->move[w][lane] = ex2_approx(fminf(by, 0.f));
              ctl->by[w][lane] = by;
              ctl->c[w][lane] += by;
            }
            const uint32_t moved = __ballot_sync(kFullMask, move);
            if (lane == 0) ctl->bits[w][0] = moved;
          }
          // (what the products have added up is scaled: the last one has to be done)
          if (x >= 2 && ok) ok = wait_for(&ctl->p_free[was], was_par, ctl, P.wait_ns);
          named_sync(1 + w, 128);
          const uint32_t moved = ctl->bits[w][0];
#pragma unroll
          for (int e = 0; e < R; e += 4) {
            const float4 by = *reinterpret_cast<const float4*>(ctl->by[w] + e);
            const float b4[4] = {by.x, by.y, by.z, by.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              s[e + k] += b4[k];
              if constexpr (R <= 16) cr[e + k] += b4[k];
            }
          }
          if (!start) {
            tc_fence_after();
#pragma unroll
            for (int e = 0; e < R; e += 4) {
              const float4 f = *reinterpret_cast<const float4*>(ctl->move[w] + e);
              l[e] *= f.x;
              l[e + 1] *= f.y;
              l[e + 2] *= f.z;
              l[e + 3] *= f.w;
            }
#pragma unroll 1
            for (uint32_t todo = moved; todo; todo &= todo - 1) {
              const int e = __ffs(todo) - 1;
              const float f = ctl->move[w][e];
              uint32_t o[F::kParts];
#pragma unroll
              for (int p = 0; p < F::kParts; ++p) tmem_ld1(mO + p * R + e, o[p]);
#pragma unroll
              for (int p = 0; p < F::kParts; ++p) {
                tmem_wait_ld1(o[p]);
                tmem_st1(mO + p * R + e, __float_as_uint(__uint_as_float(o[p]) * f));
              }
            }
            tmem_wait_st();
          }
          unset &= ~moved;
        }
#pragma unroll
        for (int i = 0; i < R; i += 16) {
          uint32_t codes[F::kParts][4];
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const uint64_t ab = pack2(ex2_approx(s[i + e]), ex2_approx(s[i + e + 1]));
            const float2 sum = unpack2(add2(pack2(l[i + e], l[i + e + 1]), ab));
            l[i + e] = sum.x;
            l[i + e + 1] = sum.y;
            const float2 z = unpack2(fma2(ab, vs2, by_half));
            uint32_t h = half_pair(z.x, z.y);
#pragma unroll
            for (int p = 0; p < F::kParts; ++p) {
              const uint16_t cp = code_pair(h);
              if (e % 4 == 0) codes[p][e / 4] = cp;
              else codes[p][e / 4] |= (uint32_t)cp << 16;
              if (p + 1 < F::kParts) h = left16(h, cp, p + 2 < F::kParts ? 0u : by_code);
            }
          }
          if (ok) {
#pragma unroll
            for (int p = 0; p < F::kParts; ++p)
              *reinterpret_cast<uint4*>(pw + (p * R + i) / 16 * 2048) =
                  uint4{codes[p][0], codes[p][1], codes[p][2], codes[p][3]};
          }
        }
        if (edge && ok) {
          ok = wait_for(&ctl->v_full[st], st_par, ctl, P.wait_ns);
          if (ok)
            clean_row<D>(smem + st * 2 * F::kTile + F::kTile, th,
                         block_key<kWindow>(sg.t, b) + th >= block_end<kWindow>(sg.t, b));
        }
        fence_async_smem();
        tc_fence_before();
        ok = __all_sync(kFullMask, ok);
        if (ok && lane == 0) mbar_arrive(&ctl->p_full[at]);
        was = at, was_par = at_par;
        if ((st += 2) >= F::kStages) st -= F::kStages, st_par ^= 1;
        if ((at += 2) >= F::kS) at -= F::kS, at_par ^= 1;
      }
      // both streams' products are done
      const bool both = items > 1;
      const int wa = g0 & 1;  // the stream of the segment's first step
#pragma unroll 1
      for (int t = g0 + items - (both ? 2 : 1); t < g0 + items; ++t)
        if (ok) ok = wait_for(&ctl->p_free[t % F::kS], (t / F::kS) & 1, ctl, P.wait_ns);
      sum_rows<R>(l, lane);
      if (R == 16) {
        if (!(lane & 1)) ctl->red[w][warp & 3][lane >> 1] = l[0];
      } else {
        ctl->red[w][warp & 3][lane] = l[0];
      }
      ok = !named_any(4, 256, !ok);
      if (!ok) break;
      tc_fence_after();
      const bool direct = sg.nb == sg.t.blocks;
      const int64_t slot0 = (int64_t)(2 * blockIdx.x + (seg > 0)) * P.plan.slot_rows;
      if (tid < R) {
        float m[2], sum[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          sum[z] = ctl->red[z][0][tid] + ctl->red[z][1][tid] + ctl->red[z][2][tid] + ctl->red[z][3][tid];
          m[z] = sum[z] == 0.f ? -INFINITY : -ctl->c[z][tid];
        }
        const float top = fmaxf(m[0], m[1]);
        const float f0 = m[0] == -INFINITY ? 0.f : ex2_approx(m[0] - top);
        const float f1 = m[1] == -INFINITY ? 0.f : ex2_approx(m[1] - top);
        const float all = sum[0] * f0 + sum[1] * f1;
        const float f = !direct ? 1.f : all > 0.f || all != all ? 1.f / all : 0.f;
        ctl->move[0][tid] = f0 * f;
        ctl->move[1][tid] = f1 * f;
        if (!direct && tid < rows) P.plan.ml[slot0 + tid] = {top, all};
      }
      named_sync(4, 256);
      if (th < R) ctl->c[w][th] = 0.f;  // (of the next unit)
      // a warpgroup half of the rows, a lane of tensor memory an element of a head
      const bool mine = th < D;
      const int64_t row0 = (int64_t)sg.t.tok0 * P.q_heads + sg.head * P.rep;
      T* const out = reinterpret_cast<T*>(P.out) + row0 * D + th;
      float* const part = P.plan.o + slot0 * D + th;
      const int* places = ctl->to[seg & 1];
#pragma unroll 1
      for (int r = w * (R / 2); r < (w + 1) * (R / 2); r += 8) {
        if (r >= rows) break;
        uint32_t a[F::kParts][8], b[F::kParts][8];
#pragma unroll
        for (int p = 0; p < F::kParts; ++p) {
          tmem_ld8(tO + lanes + F::kCols * wa + p * R + r, a[p]);
          if (both) tmem_ld8(tO + lanes + F::kCols * (wa ^ 1) + p * R + r, b[p]);
        }
#pragma unroll
        for (int p = 0; p < F::kParts; ++p) {
          tmem_wait_ld8(a[p]);
          if (both) tmem_wait_ld8(b[p]);
        }
        auto whole = [&](uint32_t (&v)[F::kParts][8], int e) {
          float z = __uint_as_float(v[F::kParts - 1][e]);
#pragma unroll
          for (int p = F::kParts - 2; p >= 0; --p) z = z * 0.0625f + __uint_as_float(v[p][e]);
          return z;
        };
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float o = whole(a, e) * ctl->move[wa][r + e];
          if (both) o += whole(b, e) * ctl->move[wa ^ 1][r + e];
          if (!mine || r + e >= rows) continue;
          if (direct) out[places[r + e] * D] = (T)o;
          else part[(r + e) * D] = o;
        }
      }
      last = sg.last;  // (before the segment's place is given back)
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ctl->o_free);
        mbar_arrive(&ctl->q_empty[seg & 1]);
      }
      g0 += items;
      if (!last) {
        ok = next_segment(seg + 1);
        if (!ok) ++seg;
      }
      if (!ok) break;
    }
    if (!ok) {
      // the sequences of this and the following units have no result
      int k = 0;
#pragma unroll 1
      for (Walk wk(P, kWindow); wk.more(); wk.next(P), ++k)
        if (k >= seg) {
          const int end = (wk.t.tok0 + wk.t.toks - 1) / P.N;
#pragma unroll 1
          for (int j = wk.t.tok0 / P.N + tid; j <= end; j += 256) P.plan.status[j] = SAMSPEC_ST_TIMEOUT;
        }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (vload(&ctl->abort)) {  // what is in flight lands first, as in attend_kernel
    if (warp == 8) {  // (both loaders' copies)
      for (int t = max(ctl->asked_k - F::kStages, 0); t < ctl->asked_k; ++t)
        drain_wait(&ctl->k_full[t % F::kStages], (t / F::kStages) & 1);
      for (int t = max(ctl->asked_v - F::kStages, 0); t < ctl->asked_v; ++t)
        drain_wait(&ctl->v_full[t % F::kStages], (t / F::kStages) & 1);
    } else if (tid == 9 * 32 || tid == 10 * 32) {  // (each waits for its own products)
      mma_commit(&ctl->drain);
      drain_wait(&ctl->drain, 0);
    }
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 9) tmem_free(tmem, 512);
}

// a pool of codes as [layers * n_pages][kv_heads * page][head_dim], in boxes of one
// page and head
int code_map(const KvView& c, void* pool, CUtensorMap* map) {
  const EncodeTiled enc = encode_tiled();
  if (!enc) return SAMSPEC_ECUDA;
  const cuuint64_t D = c.head_dim, slots = (cuuint64_t)c.kv_heads * c.page;
  const cuuint64_t dims[3] = {D, slots, (cuuint64_t)c.layers * c.n_pages};
  const cuuint64_t strides[2] = {D, slots * D};
  const cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)c.page, 1}, one[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, pool, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? SAMSPEC_OK
             : SAMSPEC_ECUDA;
}

template <typename T, int D, int R>
int launch(const AttendParams& P, bool window, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s) {
  const auto kernel = window ? attend_few_kernel<T, D, R, true> : attend_few_kernel<T, D, R, false>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Few<T, D, R>::kBytes) != cudaSuccess ||
      launch_after(kernel, kKvCtas, 512, Few<T, D, R>::kBytes, s, P, mk, mv) != cudaSuccess)
    return SAMSPEC_ECUDA;
  return SAMSPEC_OK;
}
template <typename T, int D>
int launch_rows(const AttendParams& P, bool window, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s) {
  const int rows = P.N * P.rep;
  if (rows <= 16) return launch<T, D, 16>(P, window, mk, mv, s);
  return launch<T, D, 32>(P, window, mk, mv, s);
}

}  // namespace

int attend_few(const AttendParams& P, bool bf16, bool window, cudaStream_t s) {
  CUtensorMap mk, mv;
  if (code_map(P.c, P.c.k, &mk) != SAMSPEC_OK || code_map(P.c, P.c.v, &mv) != SAMSPEC_OK) return SAMSPEC_ECUDA;
  if (bf16)
    return P.c.head_dim == 64 ? launch_rows<__nv_bfloat16, 64>(P, window, mk, mv, s)
                              : launch_rows<__nv_bfloat16, 128>(P, window, mk, mv, s);
  return P.c.head_dim == 64 ? launch_rows<__half, 64>(P, window, mk, mv, s)
                            : launch_rows<__half, 128>(P, window, mk, mv, s);
}

}  // namespace samspec
