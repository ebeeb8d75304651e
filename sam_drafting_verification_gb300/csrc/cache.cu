// cache.cu -- the paged cache's bookkeeping (reserve, fork, commit, truncate)
// and the rotary append.
//
// Free pages are a bitmap and a count of references: giving pages back is a
// sum of independent atomics (the result does not depend on their order), and
// taking them is the lowest free numbers in the order of the call's
// sequences, so every call's outcome is a function of the cache's state alone.
#include "common.cuh"
#include "kv.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace samspec {
namespace {

__device__ __forceinline__ void release_page(const KvView& c, int page) {
  if (atomicSub(&c.refs[page], 1) == 1) atomicOr(&c.free_bits[page >> 5], 1u << (page & 31));
}

// ---- reserve ---------------------------------------------------------------
struct ReserveWs {
  int32_t* first;  // [n] its first page's rank among the call's
  int32_t* need;   // [n] pages behind those held; bit 30: the last page is copied; -1: refused
  int32_t* claim;  // [seqs] the call's first sequence that names the row
  int32_t* list;   // [n_pages] the free pages in order, as far as they are needed
  int32_t* cow;    // [0]: copies; then {from, to, filled slots} of each
};

constexpr int kCowBit = 1 << 30;

// One CTA: the whole outcome hangs on prefix sums over the sequences (a few
// thousand at most) and over the bitmap, each read once; latency is its cost.
__global__ void __launch_bounds__(1024) reserve_kernel(KvView c, const int32_t* rows, int n, int N,
                                                       const int32_t* n_tok, int32_t* status, ReserveWs w) {
  __shared__ int part[32];
  const int tid = threadIdx.x;
  wait_for_previous();
  let_next_start();
  for (int i = tid; i < n; i += 1024) {
    const int row = rows ? rows[i] : i;
    if (row >= 0 && row < c.seqs) w.claim[row] = 0x7fffffff;
  }
  __syncthreads();
  for (int i = tid; i < n; i += 1024) {
    const int row = rows ? rows[i] : i;
    if (row >= 0 && row < c.seqs) atomicMin(&w.claim[row], i);
  }
  __syncthreads();
  int total = 0;
  for (int i0 = 0; i0 < n; i0 += 1024) {
    const int i = i0 + tid;
    int st = SAMSPEC_ST_OK, need = 0;
    if (i < n) {
      const int row = rows ? rows[i] : i;
      const int nt = n_tok ? n_tok[i] : N;
      if (row < 0 || row >= c.seqs || atomicAdd(&w.claim[row], 0) != i) {
        st = SAMSPEC_ST_ROW;
      } else if (nt < 0 || nt > N) {
        st = SAMSPEC_ST_BADDRAFT;
      } else {
        const int len = c.lens[row], held = c.held[row];
        const int full = len >> c.log_page;
        if (len < 0 || held < 0 || held > c.max_pages || (int64_t)held << c.log_page < len) {
          st = SAMSPEC_ST_PAGE;
        } else {
          const int64_t want = ((int64_t)len + nt + c.page - 1) >> c.log_page;
          if (want > c.max_pages) {
            st = SAMSPEC_ST_CAPACITY;
          } else {
            need = want > held ? (int)want - held : 0;
            if (len & (c.page - 1)) {
              const int tail = c.table[(int64_t)row * c.max_pages + full];
              if (tail < 0 || tail >= c.n_pages) {
                st = SAMSPEC_ST_PAGE;
                need = 0;
              } else if (c.refs[tail] > 1) {
                need |= kCowBit;
              }
            }
          }
        }
      }
      if (st != SAMSPEC_ST_OK) need = -1;
      if (status) status[i] = st;
    }
    const int pages = need > 0 ? (need & ~kCowBit) + (need & kCowBit ? 1 : 0) : 0;
    int sum;
    const int at = block_scan(pages, part, &sum);  // at most 1024 * (2^20 + 1)
    const int64_t first = (int64_t)total + at;
    if (i < n) {
      w.first[i] = (int)(first < c.n_pages ? first : c.n_pages);
      w.need[i] = need;
    }
    const int64_t t = (int64_t)total + sum;
    total = (int)(t < c.n_pages ? t : c.n_pages);
  }
  // the lowest `total` free pages, four words of the bitmap a thread and round
  const int words = (c.n_pages + 31) / 32;
  int found = 0;
  for (int w0 = 0; w0 < words && found < total; w0 += 4096) {
    uint32_t b[4];
    int cnt = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int x = w0 + 4 * tid + k;
      b[k] = x < words ? c.free_bits[x] : 0;
      if (x == words - 1 && (c.n_pages & 31)) b[k] &= (1u << (c.n_pages & 31)) - 1;
      cnt += __popc(b[k]);
    }
    int sum;
    int at = found + block_scan(cnt, part, &sum);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      for (uint32_t m = b[k]; m && at < total; m &= m - 1)
        w.list[at++] = (w0 + 4 * tid + k) * 32 + __ffs(m) - 1;
    found += sum;
  }
  if (found > total) found = total;
  __syncthreads();
  int copies = 0;
  for (int i0 = 0; i0 < n; i0 += 1024) {
    const int i = i0 + tid;
    int need = i < n ? w.need[i] : -1;
    const int first = i < n ? w.first[i] : 0;
    bool cow = need >= 0 && (need & kCowBit);
    const int more = need >= 0 ? need & ~kCowBit : 0;
    if (need > 0 && (int64_t)first + more + cow > found) {
      if (status) status[i] = SAMSPEC_ST_CAPACITY;
      cow = false;
      need = -1;
    }
    int sum;
    const int slot = copies + block_scan(cow, part, &sum);
    copies += sum;
    if (need > 0) {
      const int row = rows ? rows[i] : i;
      int32_t* t = c.table + (int64_t)row * c.max_pages;
      const int len = c.lens[row], held = c.held[row];
      if (cow) {
        const int full = len >> c.log_page, old = t[full], fresh = w.list[first];
        t[full] = fresh;
        c.refs[fresh] = 1;
        atomicAnd(&c.free_bits[fresh >> 5], ~(1u << (fresh & 31)));
        release_page(c, old);
        w.cow[1 + 3 * slot] = old;
        w.cow[2 + 3 * slot] = fresh;
        w.cow[3 + 3 * slot] = len & (c.page - 1);
      }
      for (int k = 0; k < more; ++k) {
        const int fresh = w.list[first + cow + k];
        t[held + k] = fresh;
        c.refs[fresh] = 1;
        atomicAnd(&c.free_bits[fresh >> 5], ~(1u << (fresh & 31)));
      }
      if (more) c.held[row] = held + more;
    }
  }
  if (tid == 0) w.cow[0] = copies;
}

// Filled slots of shared pages to their new pages: a warp takes one (copy,
// layer, pool, head) at a time, filled * head_dim * 2 contiguous bytes.
__global__ void __launch_bounds__(256) copy_pages_kernel(KvView c, const int32_t* cow) {
  const int lane = threadIdx.x & 31;
  const int64_t per = (int64_t)c.layers * 2 * c.kv_heads;
  wait_for_previous();
  let_next_start();
  const int64_t items = cow[0] * per;
  const int64_t warps = (int64_t)gridDim.x * 8;
  for (int64_t x = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); x < items; x += warps) {
    const int e = (int)(x / per);
    int r = (int)(x % per);
    const int head = r % c.kv_heads;
    r /= c.kv_heads;
    unsigned char* pool = r & 1 ? c.v : c.k;
    const int layer = r >> 1;
    const int from = cow[1 + 3 * e], to = cow[2 + 3 * e];
    const int vecs = cow[3 + 3 * e] * c.head_dim / 8;
    const uint4* src = reinterpret_cast<const uint4*>(pool + kv_offset(c, layer, from, head));
    uint4* dst = reinterpret_cast<uint4*>(pool + kv_offset(c, layer, to, head));
    int k = lane;
    for (; k + 96 < vecs; k += 128) {
      const uint4 a = src[k], b = src[k + 32], d = src[k + 64], f = src[k + 96];
      dst[k] = a;
      dst[k + 32] = b;
      dst[k + 64] = d;
      dst[k + 96] = f;
    }
    for (; k < vecs; k += 32) dst[k] = src[k];
  }
}

// ---- fork --------------------------------------------------------------------
__global__ void __launch_bounds__(256) fork_kernel(KvView c, const int32_t* src, const int32_t* dst, int n,
                                                   int32_t* status) {
  const int i = blockIdx.x, tid = threadIdx.x;
  wait_for_previous();
  let_next_start();
  const int s = src[i], d = dst[i];
  int st = SAMSPEC_ST_OK;
  if (s < 0 || s >= c.seqs || d < 0 || d >= c.seqs) st = SAMSPEC_ST_ROW;
  // d may not be another's target or anyone's source; s may not be a target
  bool clash = false;
  for (int j = tid; j < n; j += 256) {
    const int dj = dst[j];
    clash |= (dj == d && j != i) || src[j] == d || dj == s;
  }
  if (__syncthreads_or(clash)) st = SAMSPEC_ST_ROW;
  int len = 0, pages = 0;
  if (st == SAMSPEC_ST_OK) {
    len = c.lens[s];
    if (c.lens[d] != 0 || c.held[d] != 0) st = SAMSPEC_ST_ROW;
    else if (len < 0 || c.held[s] > c.max_pages || (int64_t)c.held[s] << c.log_page < len)
      st = SAMSPEC_ST_PAGE;
    else
      pages = (len + c.page - 1) >> c.log_page;
  }
  const int32_t* ts = c.table + (int64_t)(st ? 0 : s) * c.max_pages;
  bool bad = false;
  for (int k = tid; k < pages; k += 256) {
    const int p = ts[k];
    bad |= p < 0 || p >= c.n_pages;
  }
  // also orders every thread's reads of d's length before they are written
  if (__syncthreads_or(bad)) {
    st = SAMSPEC_ST_PAGE;
    pages = 0;
  }
  if (tid == 0 && status) status[i] = st;
  if (st != SAMSPEC_ST_OK) return;
  int32_t* td = c.table + (int64_t)d * c.max_pages;
  for (int k = tid; k < c.max_pages; k += 256) {
    if (k < pages) {
      const int p = ts[k];
      td[k] = p;
      atomicAdd(&c.refs[p], 1);
    } else {
      td[k] = -1;
    }
  }
  if (tid == 0) {
    c.lens[d] = len;
    c.held[d] = pages;
  }
}

// ---- commit and truncate -----------------------------------------------------
// One warp's judgement of call sequence i: its status, and its new length.
// Every lane returns the same.  `path`: lane t holds the t-th accepted node.
struct Judged {
  int st, row, len, new_len, held, accept, path;
};
__device__ __forceinline__ Judged judge(const KvView& c, const int32_t* rows, int n, int i, int N,
                                        const int32_t* accept, const int32_t* path, const int32_t* new_len,
                                        int lane) {
  Judged j = {SAMSPEC_ST_OK, rows ? rows[i] : i, 0, 0, 0, 0, -1};
  bool twice = false;
  if (rows)
#pragma unroll 8
    for (int k = lane; k < n; k += 32) twice |= k != i && rows[k] == j.row;
  if (__any_sync(kFullMask, twice) || j.row < 0 || j.row >= c.seqs) {
    j.st = SAMSPEC_ST_ROW;
    return j;
  }
  j.len = c.lens[j.row];
  j.held = c.held[j.row];
  if (j.len < 0 || j.held < 0 || j.held > c.max_pages || (int64_t)j.held << c.log_page < j.len) {
    j.st = SAMSPEC_ST_PAGE;
    return j;
  }
  if (!accept) {
    const int want = new_len ? new_len[i] : 0;
    if (want < 0) j.st = SAMSPEC_ST_BADDRAFT;
    j.new_len = want < j.len ? want : j.len;
    return j;
  }
  j.accept = accept[i];
  if (j.accept < -1 || j.accept >= N) {
    j.st = SAMSPEC_ST_BADDRAFT;
    return j;
  }
  int64_t last = j.accept;  // highest node that is kept
  if (path && j.accept > 0) {
    j.path = lane < j.accept ? path[(int64_t)i * N + lane] : -1;
    const int before = __shfl_up_sync(kFullMask, j.path, 1);
    const bool bad = lane < j.accept && (j.path <= (lane ? before : 0) || j.path >= N);
    if (__any_sync(kFullMask, bad)) {
      j.st = SAMSPEC_ST_BADDRAFT;
      return j;
    }
    last = __shfl_sync(kFullMask, j.path, j.accept - 1);
  }
  if (j.len + last + 1 > (int64_t)j.held << c.log_page) {
    j.st = SAMSPEC_ST_CAPACITY;
    return j;
  }
  j.new_len = j.len + 1 + j.accept;
  if (path) {
    // slots that are written have to lie in pages that no one else holds
    const int32_t* t = c.table + (int64_t)j.row * c.max_pages;
    bool bad = false, lent = false;
    for (int k = (j.len >> c.log_page) + lane; k << c.log_page < j.new_len; k += 32) {
      const int p = t[k];
      const bool out = p < 0 || p >= c.n_pages;
      bad |= out;
      lent |= !out && c.refs[p] > 1;
    }
    if (__any_sync(kFullMask, bad)) j.st = SAMSPEC_ST_PAGE;
    else if (__any_sync(kFullMask, lent)) j.st = SAMSPEC_ST_CAPACITY;
  }
  return j;
}

// Accepted nodes' keys and values to the front of their slots.  A CTA takes
// one sequence and 64 of its (layer, pool, head), judges it once (the judging
// is a chain of a dozen reads, as long as all the moves), and gives its warps
// one after the other.  Targets may be sources of nodes before them, so a warp
// reads all of its rows into registers before it writes; no other warp touches
// them.
constexpr int kMoveItems = 64;
template <int D>
__global__ void __launch_bounds__(256) move_path_kernel(KvView c, const int32_t* rows, int n, int N,
                                                        const int32_t* accept, const int32_t* path,
                                                        int32_t* status) {
  constexpr int kLanes = D / 8;           // 16-byte pieces of a row
  constexpr int kRows = 32 / kLanes;      // rows at a time
  constexpr int kSteps = 32 / kRows;      // 31 rows at most
  __shared__ int accepted;
  __shared__ int64_t from[32], to[32];    // bytes from (layer, head) 0 of a pool
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int items = c.layers * 2 * c.kv_heads;
  const int parts = (items + kMoveItems - 1) / kMoveItems;
  const int i = blockIdx.x / parts, part = blockIdx.x % parts;
  wait_for_previous();
  let_next_start();
  if (warp == 0) {
    const Judged j = judge(c, rows, n, i, N, accept, path, nullptr, lane);
    if (lane == 0 && part == 0) status[i] = j.st;  // set_len_kernel goes by it
    const bool moves = lane < j.accept && j.path != lane + 1;
    const bool any = __any_sync(kFullMask, moves);
    int a = j.st == SAMSPEC_ST_OK && any ? j.accept : 0;
    bool bad = false;
    if (lane < a) {
      const int32_t* t = c.table + (int64_t)j.row * c.max_pages;
      const int s = j.len + j.path, d = j.len + 1 + lane;
      const int ps = t[s >> c.log_page], pd = t[d >> c.log_page];
      bad = ps < 0 || ps >= c.n_pages || pd < 0 || pd >= c.n_pages;
      from[lane] = kv_offset(c, 0, ps, 0) + (int64_t)(s & (c.page - 1)) * D * 2;
      to[lane] = kv_offset(c, 0, pd, 0) + (int64_t)(d & (c.page - 1)) * D * 2;
    }
    if (__any_sync(kFullMask, bad)) a = 0;
    if (lane == 0) accepted = a;
  }
  __syncthreads();
  const int a = accepted;
  if (a == 0) return;
  const int col = lane % kLanes * 16;
  for (int x = part * kMoveItems + warp; x < min(items, (part + 1) * kMoveItems); x += 8) {
    const int head = x % c.kv_heads, r = x / c.kv_heads;
    unsigned char* pool = (r & 1 ? c.v : c.k) + kv_offset(c, r >> 1, 0, head) + col;
    uint4 buf[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int e = s * kRows + lane / kLanes;
      if (e < a) buf[s] = *reinterpret_cast<const uint4*>(pool + from[e]);
    }
    __syncwarp();
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int e = s * kRows + lane / kLanes;
      if (e < a) *reinterpret_cast<uint4*>(pool + to[e]) = buf[s];
    }
  }
}

// Lengths set, pages behind them released: one warp a sequence.  Of a commit
// with a path the status is move_path_kernel's: references change here.
__global__ void __launch_bounds__(256) set_len_kernel(KvView c, const int32_t* rows, int n, int N,
                                                      const int32_t* accept, const int32_t* path,
                                                      const int32_t* new_len, int32_t* status) {
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
  wait_for_previous();
  let_next_start();
  if (i >= n) return;
  Judged j = judge(c, rows, n, i, N, accept, nullptr, new_len, lane);
  if (path) j.st = status[i];
  int32_t* t = c.table + (int64_t)(j.st ? 0 : j.row) * c.max_pages;
  const int keep = j.st ? 0 : (j.new_len + c.page - 1) >> c.log_page;
  if (j.st == SAMSPEC_ST_OK) {
    bool bad = false;
    for (int k = keep + lane; k < j.held; k += 32) {
      const int p = t[k];
      bad |= p < 0 || p >= c.n_pages;
    }
    if (__any_sync(kFullMask, bad)) j.st = SAMSPEC_ST_PAGE;
  }
  if (lane == 0 && status) status[i] = j.st;
  if (j.st != SAMSPEC_ST_OK) return;
  for (int k = keep + lane; k < j.held; k += 32) {
    release_page(c, t[k]);
    t[k] = -1;
  }
  if (lane == 0) {
    c.lens[j.row] = j.new_len;
    if (keep < j.held) c.held[j.row] = keep;
  }
}

// ---- rotary append -----------------------------------------------------------
struct AppendParams {
  KvView c;
  PlanView plan;
  int layer, n, N, q_heads, rot, parts;
  const unsigned char* q;
  unsigned char* q_out;
  const unsigned char* k;
  const unsigned char* v;
  int64_t q_stride, k_stride, v_stride;  // elements
  const double* inv_freq;
  float mscale;
};

template <typename T>
__device__ __forceinline__ float2 unpack(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack<__nv_bfloat16>(uint32_t w) {
  return {bf16_lo(w), bf16_hi(w)};
}
template <>
__device__ __forceinline__ float2 unpack<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<__half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}
template <>
__device__ __forceinline__ uint32_t pack<__half>(float a, float b) {
  const __half2 x = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}

// Angles: pair j turns by position * f_j.  f_j / 2 pi, without its whole
// turns, is held as a 64-bit fraction of a turn; the position times that, in
// 64-bit arithmetic that wraps, is the angle with whole turns gone, exact to
// position * 2^-53 turns whatever the position.  Its top bits go to fp32 half
// turns in [-1, 1) for sincospif.
//
// A warp takes a token (for few tokens, a part of its heads): its sines and
// cosines, then its heads, eight 16-byte loads of a lane in flight.  A lane's
// place in a head is the same for all of them, and so are its sines and
// cosines; in the half layout the other elements of its pairs come from the
// lane that has loaded them.  Reads q, k, v and writes q', K, V once: bound by
// HBM for prompts, by latency for a decode step.
template <typename T, int D, bool kInterleaved>
__global__ void __launch_bounds__(256, 2) append_kernel(AppendParams P) {
  constexpr int kVec = D / 8, kStep = 32 / kVec;  // vectors of a head, heads at a time
  constexpr int kDeep = 8;
  __shared__ uint64_t turn[64];
  __shared__ float2 cs[8][64];  // each warp's cosines and sines
  const KvView& c = P.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, half = P.rot / 2;
  wait_for_previous();
  let_next_start();
  for (int j = tid; j < half; j += 256) {
    double f = P.inv_freq[j] * 0.15915494309189533577;  // 1 / (2 pi)
    f -= floor(f);
    turn[j] = (uint64_t)(f * 18446744073709551616.0);
  }
  __syncthreads();
  const bool tree = P.plan.hdr[kHdrTree] != 0;
  const int head_bytes = c.page * D * 2;
  const int q_heads = P.q ? P.q_heads : 0;
  const bool vectors = kInterleaved || half % 8 == 0;
  // this lane's vector: the first of its pairs, and in the half layout whether
  // it holds their lower (1) or upper (2) elements, and who the others
  const int e = lane % kVec;
  int first = 0, role = 0, other = lane;
  if (kInterleaved) {
    first = 4 * e;
    role = 8 * e < P.rot;
  } else if (e < half / 8) {
    first = 8 * e;
    role = 1;
    other = lane + half / 8;
  } else if (e < half / 4) {
    first = 8 * e - half;
    role = 2;
    other = lane - half / 8;
  }

  const int items = P.n * P.N * P.parts;
#pragma unroll 1
  for (int item = blockIdx.x * 8 + warp; item < items; item += gridDim.x * 8) {
    const int tok = item / P.parts, part = item % P.parts, i = tok / P.N, node = tok % P.N;
    const int q0 = q_heads * part / P.parts, q1 = q_heads * (part + 1) / P.parts;
    const int k0 = c.kv_heads * part / P.parts, k1 = c.kv_heads * (part + 1) / P.parts;
    const KvSeq& s = P.plan.seq[i];
    unsigned char* q_out = P.q_out + (int64_t)tok * P.q_heads * D * 2;
    // (the page was checked when the pass was planned; a plan used after the
    // table has changed must not write outside the pool)
    const int z = s.base + node;
    const int page = node < s.ntok ? c.table[(int64_t)s.row * c.max_pages + (z >> c.log_page)] : -1;
    if (page < 0 || page >= c.n_pages) {
      for (int x = q0 * kVec + lane; x < q1 * kVec; x += 32) reinterpret_cast<uint4*>(q_out)[x] = uint4{0, 0, 0, 0};
      continue;
    }
    const int64_t at = kv_offset(c, P.layer, page, 0) + (int64_t)(z & (c.page - 1)) * D * 2;
    const int64_t pos = (int64_t)s.base + (tree ? P.plan.node[tok].x : node);
    const unsigned char* q = P.q + (int64_t)tok * P.q_stride * 2;
    const unsigned char* k = P.k + (int64_t)tok * P.k_stride * 2;
    const unsigned char* v = P.v + (int64_t)tok * P.v_stride * 2;
    __syncwarp();  // the last token's values are read
#pragma unroll 1
    for (int j = lane; j < half; j += 32) {
      const uint64_t a = (uint64_t)pos * turn[j];
      float sn, cn;
      sincospif((float)(int64_t)a * 1.0842021724855044e-19f, &sn, &cn);  // 2^-63
      cs[warp][j] = {cn * P.mscale, sn * P.mscale};
    }
    __syncwarp();
    // heads [h0, h1) from src to dst (heads dst_head bytes apart), turned or not
    auto heads = [&](const unsigned char* src, unsigned char* dst, int dst_head, int h0, int h1, bool turned) {
      src += ((h0 + lane / kVec) * D + e * 8) * 2;
      dst += (int64_t)(h0 + lane / kVec) * dst_head + e * 16;
#pragma unroll 1
      for (int h = h0; h < h1; h += kDeep * kStep) {
        const int left = h1 - h - lane / kVec;
        uint4 x[kDeep];
#pragma unroll
        for (int y = 0; y < kDeep; ++y)
          if (y * kStep < left) x[y] = *reinterpret_cast<const uint4*>(src + y * (kStep * D * 2));
#pragma unroll
        for (int y = 0; y < kDeep; ++y) {
          if (h + y * kStep >= h1) break;  // (the whole warp)
          uint32_t* a = reinterpret_cast<uint32_t*>(&x[y]);
          if (turned) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              if (kInterleaved) {
                const float2 f = unpack<T>(a[w]), g = cs[warp][(first + w) & 63];
                if (first + w < half) a[w] = pack<T>(f.x * g.x - f.y * g.y, f.x * g.y + f.y * g.x);
              } else {
                const float2 f = unpack<T>(a[w]), o = unpack<T>(__shfl_sync(kFullMask, a[w], other & 31));
                const float2 g0 = cs[warp][(first + 2 * w) & 63], g1 = cs[warp][(first + 2 * w + 1) & 63];
                if (role == 1) a[w] = pack<T>(f.x * g0.x - o.x * g0.y, f.y * g1.x - o.y * g1.y);
                if (role == 2) a[w] = pack<T>(o.x * g0.y + f.x * g0.x, o.y * g1.y + f.y * g1.x);
              }
            }
          }
          if (y * kStep < left) *reinterpret_cast<uint4*>(dst) = x[y];
          dst += (int64_t)kStep * dst_head;
        }
        src += kDeep * kStep * D * 2;
      }
    };
    if (vectors) {
      heads(q, q_out, D * 2, q0, q1, half > 0);
      heads(k, c.k + at, head_bytes, k0, k1, half > 0);
    } else {
      // halves that do not begin on a vector: single elements
      auto singles = [&](const unsigned char* src, unsigned char* dst, int dst_head, int h0, int h1) {
#pragma unroll 1
        for (int x = h0 * D + lane; x < h1 * D; x += 32) {
          const int h = x / D, d = x % D;
          const T* from = reinterpret_cast<const T*>(src) + h * D;
          T* to = reinterpret_cast<T*>(dst + (int64_t)h * dst_head);
          if (d >= P.rot) {
            to[d] = from[d];
          } else if (d < half) {
            const float a = (float)from[d], b = (float)from[d + half];
            const float2 g = cs[warp][d];
            to[d] = (T)(a * g.x - b * g.y);
            to[d + half] = (T)(a * g.y + b * g.x);
          }
        }
      };
      singles(q, q_out, D * 2, q0, q1);
      singles(k, c.k + at, head_bytes, k0, k1);
    }
    heads(v, c.v + at, head_bytes, k0, k1, false);
  }
}

template <typename T>
void (*append_for(int D, bool interleaved))(AppendParams) {
  if (D == 64) return interleaved ? append_kernel<T, 64, true> : append_kernel<T, 64, false>;
  return interleaved ? append_kernel<T, 128, true> : append_kernel<T, 128, false>;
}

inline bool bad_rows(const KvView& c, const int32_t* d_rows, int32_t n) {
  return n < 1 || n > (1 << 20) || (!d_rows && n > c.seqs);
}

size_t reserve_layout(const KvView& c, int32_t n, void* ws, ReserveWs* w) {
  size_t at = 0;
  unsigned char* b = static_cast<unsigned char*>(ws);
  auto take = [&](size_t ints) {
    int32_t* p = reinterpret_cast<int32_t*>(b + at);
    at += (4 * ints + 15) / 16 * 16;
    return p;
  };
  w->first = take(n);
  w->need = take(n);
  w->claim = take(c.seqs);
  w->list = take(c.n_pages);
  w->cow = take(1 + 3 * (size_t)n);
  return at;
}

}  // namespace
}  // namespace samspec

using namespace samspec;

extern "C" {

size_t kv_reserve_workspace_bytes(const kv_cache* cache, int32_t n) {
  KvView c;
  ReserveWs w;
  if (kv_view(cache, &c) != SAMSPEC_OK || n < 1 || n > (1 << 20)) return 0;
  return reserve_layout(c, n, nullptr, &w);
}

int kv_reserve(const kv_cache* cache, const int32_t* d_rows, int32_t n, int32_t N,
               const int32_t* d_n_tok, int32_t* d_status, void* d_workspace, size_t ws_bytes,
               samspec_stream_t stream) {
  KvView c;
  const int rc = kv_view(cache, &c);
  if (rc != SAMSPEC_OK) return rc;
  if (!d_workspace) return SAMSPEC_EINVAL;
  if (bad_rows(c, d_rows, n) || N < 0 || N > (1 << 30)) return SAMSPEC_ESIZE;
  if (reinterpret_cast<uintptr_t>(d_workspace) % 16 != 0) return SAMSPEC_EALIGN;
  ReserveWs w;
  if (ws_bytes < reserve_layout(c, n, d_workspace, &w)) return SAMSPEC_ESIZE;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int64_t items = (int64_t)n * c.layers * 2 * c.kv_heads;
  const int64_t ctas = (items + 7) / 8;
  if (launch_after(reserve_kernel, 1, 1024, 0, s, c, d_rows, n, N, d_n_tok, d_status, w) != cudaSuccess ||
      launch_after(copy_pages_kernel, (unsigned)(ctas < kKvCtas * 8 ? ctas : kKvCtas * 8), 256, 0, s, c, w.cow) !=
          cudaSuccess)
    return SAMSPEC_ECUDA;
  return launched();
}

int kv_fork(const kv_cache* cache, const int32_t* d_src, const int32_t* d_dst, int32_t n,
            int32_t* d_status, samspec_stream_t stream) {
  KvView c;
  const int rc = kv_view(cache, &c);
  if (rc != SAMSPEC_OK) return rc;
  if (!d_src || !d_dst) return SAMSPEC_EINVAL;
  if (n < 1 || n > (1 << 20)) return SAMSPEC_ESIZE;
  if (launch_after(fork_kernel, n, 256, 0, reinterpret_cast<cudaStream_t>(stream), c, d_src, d_dst, n, d_status) !=
      cudaSuccess)
    return SAMSPEC_ECUDA;
  return launched();
}

int kv_commit(const kv_cache* cache, const int32_t* d_rows, int32_t n, int32_t N,
              const int32_t* d_accept_len, const int32_t* d_path, int32_t* d_status,
              samspec_stream_t stream) {
  KvView c;
  const int rc = kv_view(cache, &c);
  if (rc != SAMSPEC_OK) return rc;
  if (!d_accept_len || (d_path && !d_status)) return SAMSPEC_EINVAL;
  if (bad_rows(c, d_rows, n) || N < 1 || N > (d_path ? 32 : 1 << 30)) return SAMSPEC_ESIZE;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (d_path) {
    const int64_t ctas = (int64_t)n * (((int64_t)c.layers * 2 * c.kv_heads + kMoveItems - 1) / kMoveItems);
    if (ctas >= ((int64_t)1 << 31)) return SAMSPEC_ESIZE;
    if (launch_after(c.head_dim == 64 ? move_path_kernel<64> : move_path_kernel<128>, (unsigned)ctas, 256, 0, s, c,
                     d_rows, n, N, d_accept_len, d_path, d_status) != cudaSuccess)
      return SAMSPEC_ECUDA;
  }
  if (launch_after(set_len_kernel, (n + 7) / 8, 256, 0, s, c, d_rows, n, N, d_accept_len, d_path, nullptr, d_status) !=
      cudaSuccess)
    return SAMSPEC_ECUDA;
  return launched();
}

int kv_truncate(const kv_cache* cache, const int32_t* d_rows, int32_t n, const int32_t* d_new_len,
                int32_t* d_status, samspec_stream_t stream) {
  KvView c;
  const int rc = kv_view(cache, &c);
  if (rc != SAMSPEC_OK) return rc;
  if (bad_rows(c, d_rows, n)) return SAMSPEC_ESIZE;
  if (launch_after(set_len_kernel, (n + 7) / 8, 256, 0, reinterpret_cast<cudaStream_t>(stream), c, d_rows, n, 0,
                   nullptr, nullptr, d_new_len, d_status) != cudaSuccess)
    return SAMSPEC_ECUDA;
  return launched();
}

int kv_append(const kv_cache* cache, int32_t layer, const void* d_plan, int32_t n, int32_t N,
              int32_t q_heads, const void* d_q, int64_t q_stride, void* d_q_out, const void* d_k,
              int64_t k_stride, const void* d_v, int64_t v_stride, const double* d_inv_freq,
              int32_t rot, int32_t layout, float mscale, samspec_stream_t stream) {
  AppendParams P;
  const int rc = kv_view(cache, &P.c);
  if (rc != SAMSPEC_OK) return rc;
  if (!d_plan || !d_k || !d_v || !d_q != !d_q_out || (rot > 0 && !d_inv_freq)) return SAMSPEC_EINVAL;
  if (layer < 0 || layer >= P.c.layers || (layout != SAMSPEC_ROPE_HALF && layout != SAMSPEC_ROPE_INTERLEAVED))
    return SAMSPEC_EINVAL;
  const PlanLayout l = plan_layout(P.c, n, N, q_heads, false);
  if (!l.bytes || rot < 0 || rot % 2 != 0 || rot > P.c.head_dim) return SAMSPEC_ESIZE;
  const int64_t D = P.c.head_dim;
  if (k_stride < P.c.kv_heads * D || v_stride < P.c.kv_heads * D || (d_q && q_stride < q_heads * D))
    return SAMSPEC_EINVAL;
  if (d_q && d_q == d_q_out && q_stride != q_heads * D) return SAMSPEC_EINVAL;
  const uintptr_t all = reinterpret_cast<uintptr_t>(d_q) | reinterpret_cast<uintptr_t>(d_q_out) |
                        reinterpret_cast<uintptr_t>(d_k) | reinterpret_cast<uintptr_t>(d_v);
  if (all % 16 != 0 || (k_stride | v_stride | (d_q ? q_stride : 0)) % 8 != 0 ||
      reinterpret_cast<uintptr_t>(d_plan) % 256 != 0)
    return SAMSPEC_EALIGN;
  P.plan = plan_view(const_cast<void*>(d_plan), l);
  P.layer = layer;
  P.n = n;
  P.N = N;
  P.q_heads = q_heads;
  P.rot = rot;
  P.q = static_cast<const unsigned char*>(d_q);
  P.q_out = static_cast<unsigned char*>(d_q_out);
  P.k = static_cast<const unsigned char*>(d_k);
  P.v = static_cast<const unsigned char*>(d_v);
  P.q_stride = q_stride;
  P.k_stride = k_stride;
  P.v_stride = v_stride;
  P.inv_freq = d_inv_freq;
  P.mscale = mscale;
  // few tokens: a warp takes a part of a token's heads, as long as all warps run
  // at once (16 an SM; a second wave of 2048 tokens in quarters took 14.5 us, one
  // wave of whole ones 8)
  const int64_t toks = (int64_t)n * N;
  P.parts = toks * 4 <= kKvCtas * 16 ? 4 : toks * 2 <= kKvCtas * 16 ? 2 : 1;
  const int64_t ctas = (toks * P.parts + 7) / 8;
  const unsigned grid = (unsigned)(ctas < kKvCtas * 8 ? ctas : kKvCtas * 8);
  const bool inter = layout == SAMSPEC_ROPE_INTERLEAVED;
  void (*kernel)(AppendParams) = cache->dtype == SAMSPEC_BF16 ? append_for<__nv_bfloat16>(P.c.head_dim, inter)
                                                              : append_for<__half>(P.c.head_dim, inter);
  if (launch_after(kernel, grid, 256, 0, reinterpret_cast<cudaStream_t>(stream), P) != cudaSuccess) return SAMSPEC_ECUDA;
  return launched();
}

}  // extern "C"
