// attend.cuh -- what the attention kernels share: their parameters, tensor memory
// and matrix instructions, bounded waits, and the walk along a CTA's work.
#pragma once

#include "common.cuh"
#include "kv.cuh"

#include <atomic>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace samspec {

// x / d for 0 <= x < 2^31 by a multiplication: ceil(2^(31 + s) / d), s the
// bits of d - 1, is off by less than d / 2^s <= 1, so the quotient by less
// than x / 2^31 < 1 part of 1 / d
struct Divider {
  uint32_t mul, shift;
  explicit Divider(uint32_t d = 1) {
    uint32_t s = 0;
    while ((1ull << s) < d) ++s;
    shift = 31 + s;
    mul = (uint32_t)(((1ull << shift) + d - 1) / d);
  }
  __device__ __forceinline__ int operator()(int x) const { return (int)(((uint64_t)(uint32_t)x * mul) >> shift); }
};

struct AttendParams {
  KvView c;
  PlanView plan;
  int layer, n, N, q_heads, rep;
  Divider rep_div;
  const unsigned char* q;
  int64_t q_stride;
  float scale_log2;  // scale * log2(e), positive
  float lazy;        // kLazy in units of raw scores
  unsigned char* out;
  uint64_t wait_ns;
};

// Attention over a cache of 8 bits for few rows (attend_few.cu), without the join.
int attend_few(const AttendParams& P, bool bf16, bool window, cudaStream_t s);

// Tensor memory and matrix instructions (tcgen05), as inline PTX.
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// waits for this thread's loads; the 32 registers cannot be used before it
__device__ __forceinline__ void tmem_wait_ld(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                 "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// arrives on `bar` once every matrix product this thread has issued is done
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
// D (tensor memory) = A B (+ D): A and B in shared memory
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// the same with A in tensor memory
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// 32 columns of this warp's 32 lanes, one lane a thread
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tma_load3(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load4(void* dst, const CUtensorMap* map, int x, int y, int z, int u, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(u), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void named_sync(int id, int threads) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// true for all where any thread says so
__device__ __forceinline__ bool named_any(int id, int threads, bool v) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
      "bar.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ uint64_t global_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

template <typename T>
struct Type16;
template <>
struct Type16<__nv_bfloat16> {
  static constexpr uint32_t kFormat = 1, kExponent = 0x7f80;
  // probabilities relative to a maximum that may lie this many powers of two back
  static constexpr float kLazy = 8.f, kOffset = 0.f;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&x);
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return bf16_lo(w); }
  static __device__ __forceinline__ float hi(uint32_t w) { return bf16_hi(w); }
};
template <>
struct Type16<__half> {
  static constexpr uint32_t kFormat = 0, kExponent = 0x7c00;
  // fp16 probabilities are held times 2^8: 2^-32 of the largest is still
  // represented, and 2^15 (a maximum 7 behind) still below its limit
  static constexpr float kLazy = 7.f, kOffset = 8.f;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 x = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&x);
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return __half2float(__ushort_as_half(w & 0xffff)); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __half2float(__ushort_as_half(w >> 16)); }
};

struct Segment {  // what the loader hands on of a segment
  KvTile t;
  int32_t head, blk, nb, last;
};

// A bounded wait: false once the CTA gives up.  The first thread whose wait
// exceeds the limit raises the flag for all.  Flag and clock (in units of 1024 ns)
// are read only every 1024 tries, and the loop is kept small: a kernel has a dozen
// of them between the code of its roles, which is read through a cache (unrolled, with
// the clock in 64 bits, 64-wide heads over 16k-32k 8-bit keys took 188 us a call instead of
// 158).  kAhead: a try before the loop, which the kernel for 16 bits is better off with
// (64-wide heads over 16k-32k keys 160 us instead of 163).
template <bool kAhead = false, typename C>
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, C* ctl, uint64_t limit) {
  if (kAhead && mbar_try_wait(bar, parity)) return true;
  const uint32_t mask = limit < 1000000 ? 0 : 1023;  // (short limits are a test's)
  uint32_t t0 = 0;
#pragma unroll 1
  for (uint32_t k = 1; !mbar_try_wait(bar, parity); ++k) {
    if (k & mask) continue;
    if (vload(&ctl->abort)) return false;
    const uint32_t t = (uint32_t)(global_ns() >> 10) | 1;
    if (t0 == 0) t0 = t;
    if (t - t0 >= (uint32_t)(limit >> 10)) {
      vstore(&ctl->abort, 1);
      return false;
    }
  }
  return true;
}
// the same without the flag, for what is in flight when a CTA has given up
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait(bar, parity) && global_ns() - t0 < 2000000000ull) {
  }
}

// A CTA's share of the work: blocks of consecutive units (tile, key head), up
// to where the next one's begins.
struct Walk {
  int tile, head, blk;
  int window;  // of the plan
  bool other;  // the plan is not of the kernel's kind: no work
  int4 end;
  KvTile t;
  int nb;  // blocks of the segment in hand
  __device__ __forceinline__ Walk(const AttendParams& P, bool windowed) {
    const int4 a = P.plan.start[blockIdx.x];
    end = P.plan.start[blockIdx.x + 1];
    tile = a.x;
    head = a.y;
    blk = a.z;
    window = a.w;
    other = (window != 0) != windowed;
    if (other) end = a;
    load(P);
  }
  __device__ __forceinline__ void load(const AttendParams& P) {
    if (more()) {
      const int4* s = reinterpret_cast<const int4*>(P.plan.tile + tile);
      const int4 a = s[0], b = s[1], c = s[2];
      t = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
      nb = (tile == end.x && head == end.y ? end.z : t.blocks) - blk;
    }
  }
  __device__ __forceinline__ bool more() const {
    return tile < end.x || (tile == end.x && (head < end.y || (head == end.y && blk < end.z)));
  }
  // is the segment in hand the last?
  __device__ __forceinline__ bool final_one(const AttendParams& P) const {
    const bool wrap = head + 1 == P.c.kv_heads;
    return (tile == end.x && head == end.y) ||
           (end.z == 0 && tile + wrap == end.x && (wrap ? 0 : head + 1) == end.y);
  }
  __device__ __forceinline__ void next(const AttendParams& P) {
    blk = 0;
    if (++head == P.c.kv_heads) {
      head = 0;
      ++tile;
    }
    load(P);
  }
};

// a word whose lowest n bits are set (none of them, or all, where n is outside 0 .. 32)
__device__ __forceinline__ uint32_t first_bits(int n) { return n >= 32 ? 0xffffffffu : n > 0 ? (1u << n) - 1 : 0; }
// The pages of a unit's blocks, for a warp that copies them: the table's entries are
// read 32 at a time, the next 32 while these are used (a read for each block, and the
// wait for it, are a thousand clocks of one).  Entries outside the pool, should the
// table have changed since it was planned, are no pages: copies by address have no
// bounds of their own.
template <bool kWindow>
struct Pages {
  const int32_t* table;
  int end, p0 = -64, now = -1, next = -1;  // entries p0 + lane, and 32 further
  __device__ __forceinline__ Pages(const KvView& c, const KvTile& t)
      : table(c.table + (int64_t)t.seq_row * c.max_pages), end((t.kend + c.page - 1) >> c.log_page) {}
  __device__ __forceinline__ int entry(const KvView& c, int p) const {
    const int page = p < end ? table[p] : -1;
    return page >= c.n_pages ? -1 : page;
  }
  // lane x: block b's page x, -1 where it has none
  __device__ __forceinline__ int of(const KvView& c, const KvTile& t, int b, int lane) {
    const int p = block_key<kWindow>(t, b) >> c.log_page, per = kKeyBlock >> c.log_page;
    if (p >= p0 + 32) {
      // (both anew for the unit's first, or behind the keys that stay visible)
      now = p >= p0 + 64 ? entry(c, p + lane) : next;
      p0 = p >= p0 + 64 ? p : p0 + 32;
      next = entry(c, p0 + 32 + lane);
    }
    const int at = p - p0 + lane;
    int page = __shfl_sync(kFullMask, now, at & 31);
    if (p0 + 32 < p + per) {
      const int page2 = __shfl_sync(kFullMask, next, at & 31);
      if (at >= 32) page = page2;
    }
    return lane >= per || (p + lane) << c.log_page >= block_end<kWindow>(t, b) ? -1 : page;
  }
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Two floats in one instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 32 bytes a thread: a whole sector
__device__ __forceinline__ void store32(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// cuTensorMapEncodeTiled, looked up once: the library links no driver
typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiled encode_tiled() {
  static std::atomic<void*> cached{nullptr};
  void* f = cached.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    cached.store(f, std::memory_order_release);
  }
  return reinterpret_cast<EncodeTiled>(f);
}

}  // namespace samspec
