// attend.cu -- the plan of a verification pass and its attention over the
// paged cache.
#include "attend.cuh"

#include <cmath>

namespace samspec {
namespace {

std::atomic<uint64_t> g_kv_wait_ns{2000000000ull};

// ---- plan --------------------------------------------------------------------
struct PlanParams {
  KvView c;
  PlanView plan;
  const int32_t* rows;
  const int32_t* n_tok;
  const int32_t* first_child;
  const int32_t* next_sibling;
  const int32_t* group;
  int n, N, rep;
  int window, sinks;  // (window 0: none)
};

// A warp: its sequence's lengths and pages checked, the tree's depths and
// ancestors, the pages that it shares with the first sequence of its group.
__device__ __forceinline__ void plan_sequence(const PlanParams& P, int i, int lane) {
  const KvView& c = P.c;
  int st = SAMSPEC_ST_OK;
  int first = -1, next = -1;  // (read before the lengths are known)
  if (P.first_child && lane < P.N) {
    first = P.first_child[(int64_t)i * P.N + lane];
    next = P.next_sibling[(int64_t)i * P.N + lane];
  }
  const int row = P.rows ? P.rows[i] : i;
  const int nt = P.first_child ? P.N : P.n_tok ? P.n_tok[i] : P.N;
  bool twice = false;
  if (P.rows)
    for (int k = lane; k < P.n; k += 32) twice |= k != i && P.rows[k] == row;
  if (__any_sync(kFullMask, twice) || row < 0 || row >= c.seqs)
    st = SAMSPEC_ST_ROW;
  else if (nt < 0 || nt > P.N)
    st = SAMSPEC_ST_BADDRAFT;
  int base = 0;
  if (st == SAMSPEC_ST_OK) {
    base = c.lens[row];
    const int held = c.held[row];
    if (base < 0 || held < 0 || held > c.max_pages || (int64_t)held << c.log_page < base)
      st = SAMSPEC_ST_PAGE;
    else if ((int64_t)held << c.log_page < (int64_t)base + nt)
      st = SAMSPEC_ST_CAPACITY;
  }
  if (P.first_child && st == SAMSPEC_ST_OK) {
    // lane p walks its children (links only point to larger numbers, so each
    // walk ends) and is every child's parent
    const int N = P.N;
    bool bad = lane < N && ((first != -1 && (first <= lane || first >= N)) ||
                            (next != -1 && (next <= lane || next >= N)) || (lane == 0 && next != -1));
    if (__any_sync(kFullMask, bad)) {
      st = SAMSPEC_ST_BADDRAFT;
    } else {
      int parent = -1, links = 0;
      for (int p = 0; p < N; ++p) {
        // a child is linked by its parent or by the sibling before it
        const int f = __shfl_sync(kFullMask, first, p), x = __shfl_sync(kFullMask, next, p);
        const int pp = __shfl_sync(kFullMask, parent, p);
        if (lane == f) {
          parent = p;
          ++links;
        }
        if (lane == x) {
          parent = pp;
          ++links;
        }
      }
      if (__any_sync(kFullMask, lane > 0 && lane < N && links != 1)) {
        st = SAMSPEC_ST_BADDRAFT;
      } else {
        int depth = 0;
        uint32_t see = 1u << lane;
        for (int p = 1; p < N; ++p) {  // parents come first
          const int pp = __shfl_sync(kFullMask, parent, p);
          const int d = __shfl_sync(kFullMask, depth, pp);
          const uint32_t m = __shfl_sync(kFullMask, see, pp);
          if (lane == p) {
            depth = d + 1;
            see |= m;
          }
        }
        if (P.window && P.window < N) {  // ancestors behind the window, unless they stay visible
          uint32_t out = 0;
          for (int p = 0; p < N; ++p) {
            const int d = __shfl_sync(kFullMask, depth, p);
            if (depth - d >= P.window && base + d >= P.sinks) out |= 1u << p;
          }
          see &= ~out;
        }
        if (lane < N) P.plan.node[(int64_t)i * N + lane] = {depth, (int)see};
      }
    }
  }
  int leader = i, lcp = 0;
  if (st == SAMSPEC_ST_OK) {
    const int32_t* t = c.table + (int64_t)row * c.max_pages;
    const int pages = (int)(((int64_t)base + nt + c.page - 1) >> c.log_page);
    const int full = base >> c.log_page;
    bool bad = false, lent = false;
    for (int k0 = lane; k0 < pages; k0 += 128) {  // four reads of a lane in flight
      int p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = k0 + 32 * e < pages ? t[k0 + 32 * e] : 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = k0 + 32 * e;
        const bool out = p[e] < 0 || p[e] >= c.n_pages;
        bad |= out;
        // a page that is written has to be the sequence's alone
        if (!out && k >= full && k < pages && nt > 0) lent |= c.refs[p[e]] > 1;
      }
    }
    if (__any_sync(kFullMask, bad)) st = SAMSPEC_ST_PAGE;
    else if (__any_sync(kFullMask, lent)) st = SAMSPEC_ST_CAPACITY;
    if (st == SAMSPEC_ST_OK && P.group && nt > 0) {
      const int g = P.group[i];
      for (int k = i - 1; k >= 0; k -= 32) {
        const int j = k - lane;
        const uint32_t other = __ballot_sync(kFullMask, j < 0 || P.group[j] != g);
        if (other) {
          leader = k - (__ffs(other) - 1) + 1;
          break;
        }
        leader = k - 31;
      }
      // The first of them that may take part, as far as its counts say: one
      // without tokens, or whose row is empty by now, has no pages to share.
      // (Where that one is refused for its table or its tree, what follows holds
      // all the same: equal entries of this sequence's own checked table.)
      for (int k0 = leader; k0 < i; k0 += 32) {
        const int j = k0 + lane;
        bool may = j >= i;
        if (!may) {
          const int r = P.rows ? P.rows[j] : j, t = P.first_child ? P.N : P.n_tok ? P.n_tok[j] : P.N;
          if (r >= 0 && r < c.seqs && t > 0 && t <= P.N) {
            const int b = c.lens[r], held = c.held[r];
            may = b >= 0 && held >= 0 && held <= c.max_pages && (int64_t)held << c.log_page >= (int64_t)b + t;
          }
        }
        const uint32_t found = __ballot_sync(kFullMask, may);
        leader = i;
        if (found) {
          leader = min(k0 + __ffs(found) - 1, i);
          break;
        }
      }
      if (leader != i) {
        const int lrow = P.rows ? P.rows[leader] : leader;
        const int lfull = c.lens[lrow] >> c.log_page;
        const int m = min(full, lfull);
        const int32_t* tl = c.table + (int64_t)lrow * c.max_pages;
        int same = m;
        for (int k0 = 0; k0 < m && same == m; k0 += 128) {
          bool d[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k = k0 + 32 * e + lane;
            d[e] = k < m && t[k] != tl[k];
          }
#pragma unroll
          for (int e = 3; e >= 0; --e) {  // the first that differs stays
            const uint32_t differ = __ballot_sync(kFullMask, d[e]);
            if (differ) same = k0 + 32 * e + __ffs(differ) - 1;
          }
        }
        lcp = same << c.log_page;
      } else {
        lcp = full << c.log_page;
      }
    }
  }
  if (lane == 0) {
    P.plan.status[i] = st;
    P.plan.seq[i] = {row, base, st ? 0 : nt, leader, lcp, 0, 0, 0};
  }
}
__global__ void __launch_bounds__(256) plan_sequences_kernel(PlanParams P) {
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
  wait_for_previous();
  let_next_start();
  if (i < P.n) plan_sequence(P, i, threadIdx.x & 31);
}

// One CTA: what a group reads once, the units of work and their order, and
// each persistent CTA's equal share of the key blocks.
constexpr int kMinShared = 128;  // tokens: less is read by each sequence for itself
// Costs, in blocks of a unit of one row tile (2800 clocks, by HBM): a block of
// two row tiles, and what a unit costs besides its blocks (the start and end of
// its streams; more where its results are partial, in fp32, or two tiles').
// Measured: 256 trees over short histories 52 us with 4 for every unit and 46
// with 2; groups of 16 with 880 own keys each 437 us with 2 and 418 with 4;
// prompt chunks (1000 tokens and up to 4000 before, 4 sequences) 114 us with 4
// for a unit of two tiles, 110 with 5 and 106 with 6, 256-token chunks of 16
// sequences 67.3, 66.9 and 71.
constexpr int kBlockCost2 = 2;
__device__ __forceinline__ int block_cost(const KvTile& t) { return t.two ? kBlockCost2 : 1; }
__device__ __forceinline__ int unit_cost(const KvTile& t) { return t.two ? 5 : t.kind ? 4 : 2; }

// The CTAs [c0, c1] that hold the blocks of unit (tile t, head h): those of its
// first and its last block, each the last that begins at or before it.
__device__ __forceinline__ int2 unit_ctas(const KvTile& t, int h, int ctas, int cost) {
  const int bc = block_cost(t), uc = unit_cost(t);
  const int64_t b0 = t.cost0 + h * (t.blocks * bc + uc) + uc + 1;
  return {(int)((b0 * ctas - 1) / cost), (int)(((b0 + (t.blocks - 1) * bc) * ctas - 1) / cost)};
}

__global__ void __launch_bounds__(1024, 1) plan_units_kernel(PlanParams P, bool sequences) {
  constexpr int kTilesHere = 8192;
  __shared__ int part[32];
  __shared__ int costs[kTilesHere];
  __shared__ int4 starts[kKvCtas];
  const KvView& c = P.c;
  const int tid = threadIdx.x, n = P.n;
  wait_for_previous();
  let_next_start();
  if (sequences) {
    if (tid >> 5 < n) plan_sequence(P, tid >> 5, tid & 31);
    __syncthreads();
  }
  const int tt = tile_tokens(P.rep);
  KvSeq* seq = P.plan.seq;
  if (P.group) {
    // only members that take part count: the others bring no rows, set no limit
    // and take none away from those behind them
    for (int i = tid; i < n; i += 1024) {
      seq[i].shared = 0x7fffffff;
      seq[i].gsize = 0;
      seq[i].first = 0x7fffffff;
    }
    __syncthreads();
    for (int i = tid; i < n; i += 1024)
      if (seq[i].ntok > 0) {
        KvSeq& led = seq[seq[i].leader];
        atomicMin(&led.shared, seq[i].lcp);
        atomicMax(&led.gsize, i - seq[i].leader + 1);
        atomicMin(&led.first, i);
      }
    __syncthreads();
    // what two or more share, from a length on
    for (int i = tid; i < n; i += 1024)
      if (seq[i].leader == i && (seq[i].first == i + seq[i].gsize - 1 || seq[i].shared < kMinShared)) seq[i].shared = 0;
    __syncthreads();
    // the first that takes part leads, where the one that the pages were compared
    // with was refused
    for (int i = tid; i < n; i += 1024)
      if (seq[i].ntok > 0) {
        const int led = seq[i].leader, first = seq[led].first;
        seq[i].leader = first;
        if (i == led) continue;
        seq[i].shared = seq[led].shared;
        if (i == first) seq[i].gsize = seq[led].gsize - (first - led);
      }
    __syncthreads();
  }
  // tiles of the groups' shared keys, then of each sequence's own; the costs
  // before each are kept in shared memory too, where the shares are looked up
  auto tile_of = [&](const KvSeq& q, int i, int k, bool own) {
    KvTile t = {};
    const int t0 = 2 * tt * k;
    t.tok0 = i * P.N + t0;
    t.seq_row = q.row;
    if (!own) {
      t.toks = min(2 * tt, q.gsize * P.N - t0);
      t.kend = t.ctx = q.shared;
      t.kind = 1;
    } else {
      t.toks = min(2 * tt, q.ntok - t0);
      t.kbeg = q.shared;
      // a chain's tile sees no further than its last token, and all of it up
      // to its first; a tree's nodes all see the root
      t.kend = q.base + (P.first_child ? q.ntok : t0 + t.toks);
      t.ctx = q.base + 1 + (P.first_child ? 0 : t0);
      t.kind = t.kbeg > 0 ? 2 : 0;
      if (P.window) {
        // From the page of the first key that its first token sees on; the keys
        // that stay visible have blocks of their own, unless those reach that page.
        const int first = q.base + (P.first_child ? 0 : t0) + 1 - P.window;
        const int low = q.base + (P.first_child ? q.ntok : t0 + t.toks) - P.window;
        const int page0 = first > 0 ? first >> c.log_page << c.log_page : 0;
        t.kbeg = page0 / kKeyBlock * kKeyBlock >= P.sinks ? page0 : 0;
        t.sinks = P.sinks;
        t.low = low > P.sinks ? low : 0;
      }
    }
    t.two = t.toks > tt;
    t.blocks = sink_blocks(t) + (t.kend - t.kbeg + kKeyBlock - 1) / kKeyBlock;
    return t;
  };
  // As many threads a sequence as it may have tiles, up to a warp: a prompt of
  // 32768 tokens has 512 of them (the plan took 99 us with one thread, 16 with a
  // warp); where a sequence has one, more threads cost 1 us.
  int lanes = 32;
  while (lanes > 1 && (n * lanes > 1024 || lanes * tt >= P.N)) lanes >>= 1;
  const int sub = tid & (lanes - 1);
  int tiles = 0, cost = 0;
  for (int own = P.group ? 0 : 1; own < 2; ++own)
    for (int i0 = 0; i0 < n; i0 += 1024 / lanes) {
      const int i = i0 + tid / lanes;
      int cnt = 0, sum = 0;
      KvSeq q = {};
      if (i < n) {
        q = seq[i];
        if (own) cnt = (q.ntok + 2 * tt - 1) / (2 * tt);
        else if (q.ntok > 0 && q.leader == i && q.shared > 0) cnt = (q.gsize * P.N + 2 * tt - 1) / (2 * tt);
      }
      auto cost_of = [&](const KvTile& t) { return (t.blocks * block_cost(t) + unit_cost(t)) * c.kv_heads; };
      for (int k = sub; k < cnt; k += lanes) sum += cost_of(tile_of(q, i, k, own));
      int all, all_cost;
      int at = tiles + block_scan(sub == 0 ? cnt : 0, part, &all);
      int before = cost + block_scan(sum, part, &all_cost);
      at = __shfl_sync(kFullMask, at, 0, lanes);
      before = __shfl_sync(kFullMask, before, 0, lanes);
      if (i < n && sub == 0) (own ? P.plan.suf0 : P.plan.pre0)[i] = at;
      const int most = __reduce_max_sync(kFullMask, cnt);
      for (int k0 = 0; k0 < most; k0 += lanes) {
        const int k = k0 + sub;
        KvTile t = {};
        if (k < cnt) t = tile_of(q, i, k, own);
        const int mine = k < cnt ? cost_of(t) : 0;
        int upto = mine;
        for (int o = 1; o < lanes; o <<= 1) {
          const int x = __shfl_up_sync(kFullMask, upto, o, lanes);
          if (sub >= o) upto += x;
        }
        if (k < cnt) {
          t.cost0 = before + upto - mine;
          P.plan.tile[at + k] = t;
          if (at + k < kTilesHere) costs[at + k] = t.cost0;
        }
        before += __shfl_sync(kFullMask, upto, lanes - 1, lanes);
      }
      tiles += all;
      cost += all_cost;
    }
  __syncthreads();
  // at least a block's cost lies between two shares, so no two begin in one block
  const int ctas = cost ? min(kKvCtas, max(1, cost / kBlockCost2)) : 0;
  int4 start = {tiles, 0, 0, P.window};
  KvTile at;
  if (tid < ctas) {
    const int b = (int)((int64_t)tid * cost / ctas);
    int lo = 0, hi = tiles - 1;  // the last tile that begins at or before b
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if ((mid < kTilesHere ? costs[mid] : P.plan.tile[mid].cost0) <= b) lo = mid;
      else hi = mid - 1;
    }
    // the share begins in unit (lo, y) at block z: the first of which no cost
    // lies before b
    at = P.plan.tile[lo];
    const int bc = block_cost(at), uc = unit_cost(at), u = at.blocks * bc + uc;
    start.x = lo;
    start.y = (b - at.cost0) / u;
    start.z = max(((b - at.cost0) % u - uc + bc - 1) / bc, 0);
    if (start.z == at.blocks) {  // behind the unit's last block
      start.z = 0;
      if (++start.y == c.kv_heads) {
        start.y = 0;
        ++start.x;
      }
    }
    starts[tid] = start;
  }
  if (tid <= ctas) P.plan.start[tid] = start;
  __syncthreads();
  if (tid < kKvCtas) {
    KvJoin j = {};
    if (tid < ctas && start.z > 0) {
      // inside a unit: CTA tid - 1 holds what is before, all of it unless its
      // share begins inside the same one
      const int4 before = starts[tid - 1];
      const bool same = before.x == start.x && before.y == start.y;
      if (!same || before.z == 0)
        j = {at.tok0, at.toks, start.y, unit_ctas(at, start.y, ctas, cost).y - tid + 2,
             (2 * (tid - 1) + !same) * P.plan.slot_rows, 2 * tid * P.plan.slot_rows, {0, 0}};
    }
    P.plan.join[tid] = j;
  }
  // CTAs without a share begin where the last one ends
  for (int x = ctas + 1 + tid; x <= kKvCtas; x += 1024) P.plan.start[x] = {tiles, 0, 0, P.window};
  if (tid == 0) {
    P.plan.hdr[kHdrCtas] = ctas;
    P.plan.hdr[kHdrCost] = cost;
    P.plan.hdr[kHdrTree] = P.first_child != nullptr;
  }
}

// ---- attention ---------------------------------------------------------------
// Shared memory of the attention kernel, from a 1024-byte boundary: two tiles
// of 128 queries, a ring of 128-key tiles (keys and values in turn), control.
// Every tile is D / 64 slabs of 128 rows of 128 bytes in the 128-byte swizzle
// (16-byte piece c of row r lies at piece c ^ (r % 8)), which TMA writes and
// the matrix instructions read.  With a cache of 8 bits there is a second ring before
// it, of codes row by row and their scales.
struct Ctl {
  uint64_t s_full[2], p_full[2], q_full[2], q_empty[2], o_done, o_free, drain;
  uint32_t tmem;
  int32_t abort, bad;
  int32_t asked, asked_q;  // tiles that the loader has requested, once it has ended
  float2 ml[2][128];  // running maxima and sums that the streams exchange
  alignas(16) Segment seg[4];
};
template <int kStages>
struct Stages : Ctl {
  uint64_t full[kStages], empty[kStages];
};
template <int kStages, int kStages8>
struct Stages8 : Stages<kStages> {
  uint64_t full8[kStages8], empty8[kStages8];
  int32_t last8[kStages8];  // the CTA's last tile
};
template <int D, bool kEight>
struct Ring {
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kStages = D == 128 ? 5 : 11;
  static constexpr int kCtl = (2 + kStages) * kTile;
  static constexpr int kThreads = 384;
  using Control = Stages<kStages>;
  static constexpr int kBytes = kCtl + (int)((sizeof(Control) + 127) / 128 * 128);
  static_assert(kBytes <= 232448, "227 KB of a CTA");
};
// Three tiles of 16 bits are what the products need (keys of the next block while a
// block's values wait for its softmax); the codes behind them cover HBM's latency.
template <int D>
struct Ring<D, true> {
  static constexpr int kTile = 128 * D * 2, kTile8 = 128 * D;
  static constexpr int kStages = D == 128 ? 3 : 5, kStages8 = D == 128 ? 4 : 12;
  static constexpr int kCodes = (2 + kStages) * kTile;
  static constexpr int kScales = kCodes + kStages8 * kTile8;
  static constexpr int kCtl = kScales + kStages8 * kKeyBlock;
  static constexpr int kThreads = 512;
  using Control = Stages8<kStages, kStages8>;
  static constexpr int kBytes = kCtl + (int)((sizeof(Control) + 127) / 128 * 128);
  static_assert(kBytes <= 232448, "227 KB of a CTA");
};

// Matrix descriptor of a tile: address and strides in units of 16 bytes,
// 16384 bytes between slabs (keys across, for the values), 1024 between groups
// of 8 rows, 128-byte swizzle.  Only the low word depends on the address.
constexpr uint32_t kDescHigh = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(const void* p) { return (smem_u32(p) >> 4) | ((16384u >> 4) << 16); }
__device__ __forceinline__ uint64_t desc(uint32_t low) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(low), "r"(kDescHigh));
  return r;
}

// Values of a block from row `lo` on (the keys that not every query sees):
// those of no key of the unit (from row `hi` on) become zeros, and so do
// infinities and NaN, since 0 * NaN would reach the queries that do not see
// them; those that do add them at the end.  `th` of `threads` threads.
template <typename T, int D>
__device__ __forceinline__ void clean_values(unsigned char* v, int lo, int hi, int th, int threads, Ctl* ctl) {
  using H = Type16<T>;
  constexpr int kPer = D / 8;
  bool found = false;
  for (int e = th; e < (kKeyBlock - lo) * kPer; e += threads) {
    const int r = lo + e / kPer, pc = e % kPer;
    uint4* at = reinterpret_cast<uint4*>(v + (pc >> 3) * 16384 + r * 128 + (((pc & 7) ^ (r & 7)) << 4));
    if (r >= hi) {
      *at = uint4{0, 0, 0, 0};
    } else {
      uint4 u = *at;
      uint32_t* a = reinterpret_cast<uint32_t*>(&u);
      bool hit = false;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t lo16 = (a[k] & H::kExponent) == H::kExponent ? 0xffffu : 0u;
        const uint32_t hi16 = ((a[k] >> 16) & H::kExponent) == H::kExponent ? 0xffff0000u : 0u;
        hit |= (lo16 | hi16) != 0;
        a[k] &= ~(lo16 | hi16);
      }
      if (hit) *at = u;
      found |= hit;
    }
  }
  if (found) ctl->bad = 1;
  fence_async_smem();
}

// Infinities and NaN among the values of keys [from, to) that a row sees (keys
// before lim, with a window those of them from `low` on, and a tree's nodes),
// added to its stored result (out: 16 bits, else fp32 sums), columns d0 on.
template <typename T, bool kWindow, bool kEight>
__device__ __forceinline__ void add_unclean(const AttendParams& P, int seq_row, int head, int base, int lim, int low,
                                         uint32_t see, int from, int to, int d0, int cols, unsigned char* out,
                                         float* sums) {
  using H = Type16<T>;
  const KvView& c = P.c;
#pragma unroll 1
  for (int key = from; key < to; ++key) {
    if (!((key < lim && (!kWindow || key >= low)) || (key >= base && key - base < 32 && ((see >> (key - base)) & 1))))
      continue;
    const int pg = c.table[(int64_t)seq_row * c.max_pages + (key >> c.log_page)];
    if (pg < 0 || pg >= c.n_pages) continue;
    if (kEight) {  // a head that is NaN as a whole
      if (c.v_scale[kv_slot(c, P.layer, pg, head) + (key & (c.page - 1))] != kScaleNan) continue;
      if (out)
        for (int e = 0; e < cols / 2; ++e) reinterpret_cast<uint32_t*>(out)[e] = 0x7fff7fffu;
      else
        for (int e = 0; e < cols; ++e) sums[e] = NAN;
      continue;
    }
    const uint32_t* v = reinterpret_cast<const uint32_t*>(
        c.v + kv_offset(c, P.layer, pg, head) + ((int64_t)(key & (c.page - 1)) * c.head_dim + d0) * 2);
#pragma unroll 1
    for (int e = 0; e < cols / 2; ++e) {
      const uint32_t z = v[e];
      const bool lo = (z & H::kExponent) == H::kExponent, hi = ((z >> 16) & H::kExponent) == H::kExponent;
      if (!lo && !hi) continue;
      if (out) {
        uint32_t* o = reinterpret_cast<uint32_t*>(out) + e;
        *o = H::pack(H::lo(*o) + (lo ? H::lo(z) : 0.f), H::hi(*o) + (hi ? H::hi(z) : 0.f));
      } else {
        if (lo) sums[2 * e] += H::lo(z);
        if (hi) sums[2 * e + 1] += H::hi(z);
      }
    }
  }
}

// The warps that turn tiles of codes into tiles of 16 bits, in the order of the copies:
// six of them (64 sequences of 4096 keys, 64 rows, us a call: 230 when that was chosen, with
// five 243, four 254, three 306), in one place of the code (in two, 310: it is read through
// a cache).  A warp takes 32 of the 16-byte pieces of codes at a time, each 2 pieces of a
// row (2 pc, 2 pc + 1), reading the next 32 meanwhile (230 -> 212, all of them beforehand
// 219; now 205, L2 flushed before the call); the upper half of a
// 128-wide row's lanes writes the odd one first, so that eight lanes meet eight groups of
// banks.  A lane makes the factor of one of the warp's rows, the lanes of a row take it
// from there.
constexpr int kExpandWarps = 6;
template <typename T, int D, bool kWindow>
__device__ __forceinline__ void expand_tiles(const AttendParams& P, unsigned char* smem, int who, int lane) {
  using R = Ring<D, true>;
  constexpr bool kBf16 = Type16<T>::kFormat == 1;
  auto* ctl = reinterpret_cast<typename R::Control*>(smem + R::kCtl);
  constexpr int kPer = D / 16, kRowsAt = 32 / kPer;       // pieces of a row; rows of 32 pieces
  constexpr int kAll = 128 / kRowsAt, kMost = (kAll + kExpandWarps - 1) / kExpandWarps;  // groups of rows
  const int pc = lane % kPer, flip = (pc >> 2) & 1;
  // this lane's row among a group's, and the row that it makes the factor of (that of
  // the warp's group lane / kRowsAt)
  const int sub = lane / kPer, made = min((who + lane / kRowsAt * kExpandWarps) * kRowsAt + lane % kRowsAt, 127);
  bool ok = true, last = !Walk(P, kWindow).more();
  int st = 0, par = 1, s8 = 0, par8 = 0;
#pragma unroll 1
  while (!last) {
    ok = wait_for(&ctl->full8[s8], par8, ctl, P.wait_ns);
    ok = ok && wait_for(&ctl->empty[st], par, ctl, P.wait_ns);
    if (!__all_sync(kFullMask, ok)) break;
    last = ctl->last8[s8];
    const uint32_t factor = scale_word<kBf16>(smem[R::kScales + s8 * kKeyBlock + made]);
    const uint4* from = reinterpret_cast<const uint4*>(smem + R::kCodes + s8 * R::kTile8) + who * 32 + lane;
    unsigned char* to = smem + (2 + st) * R::kTile + pc / 4 * 16384 + (who * kRowsAt + sub) * 128;
    uint4 ahead = from[0];
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      const uint32_t scale = __shfl_sync(kFullMask, factor, i * kRowsAt + sub);
      if (kAll % kExpandWarps != 0 && i == kMost - 1 && who + i * kExpandWarps >= kAll) break;
      uint4 u = ahead;
      if (i + 1 < kMost) ahead = from[(who + (i + 1) * kExpandWarps < kAll ? i + 1 : i) * kExpandWarps * 32];
      if (D == 128) u = flip ? uint4{u.z, u.w, u.x, u.y} : u;
      uint32_t w[8];
      expand16<kBf16>(u, scale, w);
      uint4* row = reinterpret_cast<uint4*>(to + i * (kExpandWarps * kRowsAt * 128));
      const int a = ((2 * pc + flip) & 7) ^ (((who + i * kExpandWarps) * kRowsAt + sub) & 7);
      row[a] = uint4{w[0], w[1], w[2], w[3]};
      row[a ^ 1] = uint4{w[4], w[5], w[6], w[7]};
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&ctl->full[st]);
      mbar_arrive(&ctl->empty8[s8]);
    }
    if (++st == R::kStages) st = 0, par ^= 1;
    if (++s8 == R::kStages8) s8 = 0, par8 ^= 1;
  }
}

// One persistent CTA an SM.  Warp 8 loads queries and pages by TMA, warp 9
// issues matrix products, two warpgroups do the softmax, a thread a row.
//
// A step is one block of 128 keys against 128 query rows: S = Q K^T (both in
// shared memory, S in tensor memory), P = exp2(S - m) rounded to 16 bits over
// S's columns, O += P V.  Two streams of steps run at once, each with its own
// S, running maximum, sum and O, so that the matrix unit works on one while
// the other's softmax runs: a unit of more than 128 rows has a stream for each
// half of its rows (both use a block of keys and values while it is in shared
// memory), a smaller one gives its blocks to the two in turn and adds them up
// at the end.  O is rescaled only when the maximum has moved by 2^kLazy.
// Steps are numbered through all of a CTA's segments, step g in stream g % 2,
// so the next segment's first scores are computed while this one's last are
// worked on; only its first product into O waits until O has been read.
//
// P is rounded to the cache's type, as the product takes it: half a step of
// each weight, which the 64-bit tests' bounds count; sums (of the weights before
// that), maxima and O stay in fp32.  Exponentials are ex2.approx, within 2^-22 of
// the value, far below that rounding: half of the softmax's clocks even so.
//
// What bounds it.  One tile of rows: HBM.  A block is 128 keys * D * 4 bytes,
// 2800 clocks of an SM's share, against 1090 for the two products and 1500 for
// a warp's softmax with two in flight; few rows (a decode step has N * rep of
// 128) waste the matrix unit but no time.  16 sequences of 32768 keys, 8 key
// heads of 128, 32 rows each: 322 us, 6.7 TB/s of 6.8.  Two tiles: a step of
// each stream takes 2000 clocks, half of it the matrix unit (1130 TFLOP/s over
// 32768 keys); what is left is the chain S, softmax, P, product, S of a stream,
// of which the softmax is 1470 (reading S 340, maximum 150, exponentials 750).
// A unit's start and end cost about 5000 clocks.
//
// Registers decide that chain.  What is spilled goes to L2, since shared memory
// leaves no L1: 100 bytes a thread cost 5%, 300 bytes twice the time.  So a
// thread holds a row's 128 scores (216 registers), and the sums are read 16
// columns at a time.  Two warpgroups a stream with 64 keys each (104 registers)
// had to read the scores twice, and took 256 us where this takes 241; giving
// the product its first 64 keys early took 252; spinning instead of waiting 270.
//
// kWindow: of a plan with a window.  A kernel of its own: what windows add to the
// softmax's steps costs 2-3% where those are the bound, used or not (groups of 16
// 442 -> 452 us, prompt chunks 122 -> 126), and both bodies in one kernel spill.
//
// What bounds a window: units' starts and ends.  64 sequences, trees' or chains' 4
// tokens, windows of 1024 keys, 8 heads of 128: 66 us for this kernel, 4.6 TB/s, for units
// of 9 to 10 blocks; 4 chunks of 1000 tokens in windows of 512: 59 us for units of 5 to 7.
//
// kEight: of a cache of 8 bits, for what attend_few_kernel does not take.  TMA brings
// codes and scales as they lie in their pages; warps 10 to 15 turn each tile into 16
// bits in the layout that the products take, two 16-byte pieces from one, so all that
// follows is the same, and results are those of a 16-bit cache that holds the codes'
// values.  A block is 128 keys * (D + 1) * 2 bytes, 1400 clocks of an SM's share of
// HBM.  What bounds it: the six warps for one tile of rows, as they take 3600 clocks for
// a block; the softmax's chain, which they share the issue slots with, for two.  So it
// saves memory, not time: 64 sequences of 4096 keys, 8 heads of 128 (64), 64 rows, 205 (150)
// us a call, L2 flushed before it, over a cache of 16 bits 190 (127); groups of 8 with
// 4096 keys shared 103 and 93; 4 chunks of 1000 tokens behind 0 to 4000 keys, 32 heads
// on 8 of 128, 136 and 122.
template <typename T, int D, bool kWindow, bool kEight>
__global__ void __launch_bounds__(Ring<D, kEight>::kThreads, 1)
    attend_kernel(const __grid_constant__ AttendParams P, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_q) {
  using R = Ring<D, kEight>;
  using H = Type16<T>;
  extern __shared__ __align__(1024) unsigned char smem[];
  auto* ctl = reinterpret_cast<typename R::Control*>(smem + R::kCtl);
  unsigned char* ring = smem + 2 * R::kTile;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const KvView& c = P.c;
  if (smem_u32(smem) & 1023) {
    // The swizzle counts from there, and the linker sees to it.  Were it not so,
    // nothing is computed, and every sequence says so.
    wait_for_previous();
    let_next_start();
    for (int i = blockIdx.x * R::kThreads + tid; i < P.n; i += kKvCtas * R::kThreads)
      P.plan.status[i] = SAMSPEC_ST_TIMEOUT;
    return;
  }
  if (warp == 9) tmem_alloc(&ctl->tmem, 512);
  if (tid == 0) {
    for (int s = 0; s < R::kStages; ++s) {
      mbar_init(&ctl->full[s], kEight ? kExpandWarps : 1);
      mbar_init(&ctl->empty[s], 1);
    }
    if constexpr (kEight)
      for (int s = 0; s < R::kStages8; ++s) {
        mbar_init(&ctl->full8[s], 1);
        mbar_init(&ctl->empty8[s], kExpandWarps);
      }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&ctl->s_full[w], 1);
      mbar_init(&ctl->p_full[w], 4);
      mbar_init(&ctl->q_full[w], 1);
      mbar_init(&ctl->q_empty[w], 1);
    }
    mbar_init(&ctl->o_done, 1);
    mbar_init(&ctl->o_free, 8);
    mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    ctl->bad = 0;
    mbar_fence_init();
  }
  tc_fence_before();
  wait_for_previous();
  let_next_start();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  // (a CTA without a share finds its first segment at its end)
  const uint32_t tS = tmem, tO = tmem + 256;  // streams 128 columns apart

  const int tt = tile_tokens(P.rep);
  // registers: 384 * 168 at launch = 256 * 216 + 128 * 72, or 512 * 128 = 256 * 200 + 256 * 56
  if (warp >= 8) {
    if (kEight) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 8) {
      // ---- queries and pages ----
      int kt = 0, qt = 0, seg = 0;  // tiles requested, of keys and values and of queries; segments
      bool ok = true;
      constexpr int kSlabs = D / 64;
      const int x = lane / kSlabs, slab = lane % kSlabs;
      const int per = kKeyBlock >> c.log_page;  // pages of a block
      for (Walk wk(P, kWindow); ok && wk.more(); wk.next(P), ++seg) {
        for (int h = 0; ok && h <= wk.t.two; ++h) {
          uint64_t* bar = &ctl->q_full[qt & 1];
          ok = wait_for<!kEight>(&ctl->q_empty[qt & 1], ((qt >> 1) & 1) ^ 1, ctl, P.wait_ns);
          ok = __all_sync(kFullMask, ok);
          if (!ok) break;
          if (lane == 0) {
            if (h == 0) ctl->seg[seg & 3] = {wk.t, wk.head, wk.blk, wk.nb, wk.final_one(P)};
            mbar_arrive_expect_tx(bar, (uint32_t)(tt * P.rep) * D * 2);
          }
          __syncwarp();
          if (lane < kSlabs)
            tma_load4(smem + (qt & 1) * R::kTile + lane * 16384, &map_q, lane * 64, 0, wk.head, wk.t.tok0 + h * tt, bar);
          ++qt;
        }
        if constexpr (kEight) {
          Pages<kWindow> of(c, wk.t);
          const bool final_one = wk.final_one(P);
#pragma unroll 1
          for (int b2 = 0; ok && b2 < 2 * wk.nb; ++b2) {  // keys and values in turn
            const int page = of.of(c, wk.t, wk.blk + (b2 >> 1), lane);
            const int pages = __popc(__ballot_sync(kFullMask, page >= 0));
            const int st = kt % R::kStages8;
            ok = wait_for<!kEight>(&ctl->empty8[st], ((kt / R::kStages8) & 1) ^ 1, ctl, P.wait_ns);
            ok = __all_sync(kFullMask, ok);
            if (!ok) break;
            if (lane == 0) {
              ctl->last8[st] = b2 + 1 == 2 * wk.nb && final_one;
              mbar_arrive_expect_tx(&ctl->full8[st], (uint32_t)pages * c.page * (D + 1));
            }
            __syncwarp();
            if (page >= 0) {
              const int64_t slot = kv_slot(c, P.layer, page, wk.head);
              bulk_g2s(smem + R::kCodes + st * R::kTile8 + lane * c.page * D, (b2 & 1 ? c.v : c.k) + slot * D, c.page * D,
                       &ctl->full8[st]);
              bulk_g2s(smem + R::kScales + st * kKeyBlock + lane * c.page, (b2 & 1 ? c.v_scale : c.k_scale) + slot, c.page,
                       &ctl->full8[st]);
            }
            ++kt;
          }
          continue;
        }
        const int32_t* table = c.table + (int64_t)wk.t.seq_row * c.max_pages;
        auto fetch = [&](int b) {
          const int p = (block_key<kWindow>(wk.t, b) >> c.log_page) + x;
          return x < per && p << c.log_page < block_end<kWindow>(wk.t, b) ? table[p] : -1;
        };
        int page = fetch(wk.blk);
        for (int b = 0; ok && b < wk.nb; ++b) {
          const int ahead = b + 1 < wk.nb ? fetch(wk.blk + b + 1) : -1;
          const int pages = __popc(__ballot_sync(kFullMask, page >= 0 && slab == 0));
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const int st = kt % R::kStages;
            ok = ok && wait_for<!kEight>(&ctl->empty[st], ((kt / R::kStages) & 1) ^ 1, ctl, P.wait_ns);
            ok = __all_sync(kFullMask, ok);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&ctl->full[st], (uint32_t)pages * c.page * D * 2);
            __syncwarp();
            if (page >= 0)
              tma_load3(ring + st * R::kTile + slab * (128 * 128) + x * c.page * 128, kv ? &map_v : &map_k, slab * 64,
                        wk.head * c.page, P.layer * c.n_pages + page, &ctl->full[st]);
            ++kt;
          }
          page = ahead;
        }
      }
      if (lane == 0) {
        ctl->asked = kt;
        ctl->asked_q = qt;
      }
    } else if (warp == 9) {
      // ---- matrix products ----
      if (lane == 0) {
        const uint32_t id = (1u << 4) | (H::kFormat << 7) | (H::kFormat << 10) | ((128 >> 4) << 24);
        const uint32_t id_s = id | ((128 >> 3) << 17), id_o = id | ((D >> 3) << 17) | (1u << 16);
        const uint32_t q_low = desc_low(smem), ring_low = desc_low(ring);
        bool ok = true, last = !Walk(P, kWindow).more();
        // the step whose product with V is still to be issued: its ring stage
        // (-1: none), the parity of that, and what goes with it
        enum { kFirst = 1, kAwaitV = 2, kRelease = 4, kEnd = 8, kAwaitO = 16, kParityO = 32, kParityV = 64 };
        int v_stage = -1;
        uint32_t v_what = 0;
        int g = 0;               // steps issued
        int st = 0, par = 0;     // ring stage of the block's keys, its parity
        auto product = [&] {
          const int w = (g - 1) & 1;
          ok = wait_for<!kEight>(&ctl->p_full[w], ((g - 1) >> 1) & 1, ctl, P.wait_ns);
          if (v_what & kAwaitV) ok = ok && wait_for<!kEight>(&ctl->full[v_stage], (v_what & kParityV) != 0, ctl, P.wait_ns);
          // the last segment's O has to be read before this one's begins
          if (v_what & kAwaitO) ok = ok && wait_for<!kEight>(&ctl->o_free, (v_what & kParityO) != 0, ctl, P.wait_ns);
          if (!ok) return;
          tc_fence_after();
          const uint32_t vl = ring_low + v_stage * (R::kTile >> 4);
#pragma unroll
          for (int k = 0; k < 8; ++k)  // 16 keys: two groups of 8 rows
            mma_ts(tO + 128 * w, tS + 128 * w + 8 * k, desc(vl + k * (2048 >> 4)), id_o,
                   !(v_what & kFirst) || k > 0);
          if (v_what & kRelease) mma_commit(&ctl->empty[v_stage]);
          if (v_what & kEnd) mma_commit(&ctl->o_done);
          v_stage = -1;
        };
        for (int seg = 0, qt = 0; ok && !last; ++seg) {
          ok = wait_for<!kEight>(&ctl->q_full[qt & 1], (qt >> 1) & 1, ctl, P.wait_ns);
          if (!ok) break;
          const int nb = ctl->seg[seg & 3].nb;
          const bool rows2 = ctl->seg[seg & 3].t.two;
          last = ctl->seg[seg & 3].last;
          if (rows2) ok = wait_for<!kEight>(&ctl->q_full[(qt + 1) & 1], ((qt + 1) >> 1) & 1, ctl, P.wait_ns);
          const int items = rows2 ? 2 * nb : nb;
          for (int x = 0; ok && x < items; ++x, ++g) {
            const int w = g & 1, half = rows2 ? x & 1 : 0;
            const bool done = !rows2 || half == 1;  // with the block's keys
            if (half == 0) ok = wait_for<!kEight>(&ctl->full[st], par, ctl, P.wait_ns);
            if (!ok) break;
            tc_fence_after();
            const uint32_t ql = q_low + ((qt + half) & 1) * (R::kTile >> 4), kl = ring_low + st * (R::kTile >> 4);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t at = (k / 4) * (16384 >> 4) + (k % 4) * 2;  // 16 elements along a row
              mma_ss(tS + 128 * w, desc(ql + at), desc(kl + at), id_s, k > 0);
            }
            mma_commit(&ctl->s_full[w]);
            if (v_stage >= 0) product();
            int vs = st + 1, vp = par;
            if (vs == R::kStages) vs = 0, vp ^= 1;
            v_stage = vs;
            v_what = (x < 2 ? kFirst | (seg > 0 ? kAwaitO | ((seg - 1) & 1 ? kParityO : 0) : 0) : 0) |
                     (half == 0 ? kAwaitV : 0) | (done ? kRelease : 0) | (x == items - 1 ? kEnd : 0) |
                     (vp ? kParityV : 0);
            if (done) {
              st = vs + 1, par = vp;
              if (st == R::kStages) st = 0, par ^= 1;
            }
          }
          qt += rows2 ? 2 : 1;
        }
        if (ok && v_stage >= 0) product();
      }
      __syncwarp();
    } else {
      // (by the loader's warp, in its code: groups of 16 446 us instead of 442)
      if (warp == 10 && blockIdx.x == 0 && (P.plan.start[0].w != 0) != kWindow)  // a plan of the other kind
        for (int i = lane; i < P.n; i += 32) P.plan.status[i] = SAMSPEC_ST_BADPARAM;
      if constexpr (kEight) expand_tiles<T, D, kWindow>(P, smem, warp - 10, lane);
    }
  } else {
    if (kEight) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // ---- softmax ----
    // A thread that gives up keeps taking part in every bar.sync of its segment,
    // without work, so that no other waits for it there.  It arrives on no
    // mbarrier any more: that would hand on what it has not seen (a ring stage
    // whose copy is still on its way would be asked for again, and its barrier's
    // counts would run ahead); those who wait for it see the flag.
    const int w = warp >> 2;                 // stream
    const int row = (warp & 3) * 32 + lane;  // its lane of tensor memory
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t mS = tS + 128 * w + lanes, mO = tO + 128 * w + lanes;
    const float sc = P.scale_log2;
    const bool tree = P.plan.hdr[kHdrTree] != 0;
    int g0 = 0, kb = 0, qt = 0, seg = 0;  // steps, blocks, query tiles and segments before
    const int window = kWindow ? P.plan.start[blockIdx.x].w : 0;
    bool last = !Walk(P, kWindow).more();
    bool ok = true;
    // a segment has come: all threads of both streams decide alike whether to
    // go on, and are done with the last one's exchange and flag
    auto next_segment = [&](int q) {
      const bool came = wait_for<!kEight>(&ctl->q_full[q & 1], (q >> 1) & 1, ctl, P.wait_ns);
      return !named_any(4, 256, !came);
    };
    if (!last) ok = next_segment(0);
    for (; ok && !last; ++seg) {
      const Segment& sg = ctl->seg[seg & 3];  // the loader is two segments ahead at most
      const bool rows2 = sg.t.two;
      const int items = rows2 ? 2 * sg.nb : sg.nb;
      const int x0 = (w - g0) & 1;  // this stream's first step of the segment
      // what the row sees: keys before lim, and a tree's nodes; the first step
      // whose keys not every row sees
      bool live, busy;
      int lim, x_edge, low = 0, x_low;  // (windows: keys from `low` on, and steps before the first whose keys all see)
      uint32_t see = 0;
      {
        const int t0 = rows2 ? tt * x0 : 0, lt = P.rep_div(row);  // this thread's token, of its tile's
        live = lt < tt && t0 + lt < sg.t.toks;
        busy = P.rep_div(row - lane) < min(tt, sg.t.toks - t0);
        lim = sg.t.kend;
        if (live && sg.t.kind != 1) {
          if (tree) {
            const int2 node = P.plan.node[sg.t.tok0 + t0 + lt];
            see = (uint32_t)node.y;
            lim = sg.t.ctx - 1;
            if (kWindow) low = sg.t.ctx + node.x - window;
          } else {
            lim = min(lim, sg.t.ctx + t0 + lt);
            if (kWindow) low = sg.t.ctx + t0 + lt - window;
          }
        }
        const int first = sg.blk - (kWindow ? sink_blocks(sg.t) : 0);  // (of the blocks from kbeg on)
        const int before = sg.t.ctx - sg.t.kbeg - first * kKeyBlock;
        x_edge = (before > 0 ? before / kKeyBlock : 0) * (rows2 ? 2 : 1);
        x_low = kWindow && sg.t.low > 0 ? ((sg.t.low - sg.t.kbeg + kKeyBlock - 1) / kKeyBlock - first) * (rows2 ? 2 : 1) : 0;
      }
      // m in units of raw scores, and how far they may go before it moves; the
      // exponent's constant
      float m = -INFINITY, reach = -INFINITY, off = 0.f, l = 0.f;
      for (int x = x0; x < items; x += 2) {
        const bool edge = x >= x_edge || (kWindow && x < x_low);
        if (ok) ok = wait_for<!kEight>(&ctl->s_full[w], ((g0 + x) >> 1) & 1, ctl, P.wait_ns);
        ok = __all_sync(kFullMask, ok);
        tc_fence_after();
        if (ok && row == 0) {
          // the product is done with the block's keys, the last one with the
          // queries (arrivals here, since each commit of the products' warp
          // takes the matrix unit 57 clocks)
          const int t_k = 2 * (kb + (rows2 ? x >> 1 : x));
          if (!rows2 || (x & 1)) mbar_arrive(&ctl->empty[t_k % R::kStages]);
          if (x + 1 >= items - (int)rows2) mbar_arrive(&ctl->q_empty[(qt + (rows2 ? x & 1 : 0)) & 1]);
        }
        if (ok && busy) {
          uint32_t s[128];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32(mS + 32 * q, s + 32 * q);
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_wait_ld(s + 32 * q);
          if (edge) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int ks = block_key<kWindow>(sg.t, sg.blk + (rows2 ? x >> 1 : x)) + 32 * q;
              // bits of the 32 keys from ks on: those before lim, a window's and
              // those that stay visible, and a tree's
              uint32_t bits = first_bits(lim - ks);
              if (kWindow && x < x_low) bits &= ~first_bits(low - ks) | first_bits(sg.t.sinks - ks);
              if (see) {
                const int d = sg.t.ctx - 1 - ks;
                bits |= d >= 0 ? (d < 32 ? see << d : 0) : (d > -32 ? see >> -d : 0);
              }
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((bits >> e) & 1)) s[32 * q + e] = 0xff800000u;
            }
          }
          float mx[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = fmaxf(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
#pragma unroll
          for (int e = 4; e < 64; ++e)
            mx[e & 3] = max3(mx[e & 3], __uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
          const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
          if (__any_sync(kFullMask, live && top > reach)) {
            // the maximum moves (for the first block, or by more than 2^kLazy)
            float f = 1.f;
            if (top > reach) {
              if (m != -INFINITY) f = ex2_approx((m - top) * sc);
              m = top;
              off = H::kOffset - m * sc;
              reach = m + P.lazy;
              l *= f;
            }
            if (x >= 2) {
#pragma unroll 1
              for (int q = 0; q < D / 16; ++q) {
                uint32_t o[16];
                tmem_ld16(mO + 16 * q, o);
                tmem_wait_ld16(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st16(mO + 16 * q, o);
              }
            }
          }
          const uint64_t sc2 = pack2(sc, sc), off2 = pack2(off, off);
          uint64_t sum[2] = {0, 0};
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            uint32_t p[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 z = unpack2(fma2(
                  pack2(__uint_as_float(s[16 * q + 2 * e]), __uint_as_float(s[16 * q + 2 * e + 1])), sc2, off2));
              const float a = ex2_approx(z.x), d = ex2_approx(z.y);
              sum[e & 1] = add2(sum[e & 1], pack2(a, d));
              p[e] = H::pack(a, d);
            }
            tmem_st8(mS + 8 * q, p);
          }
          const float2 t2 = unpack2(add2(sum[0], sum[1]));
          l += t2.x + t2.y;
          tmem_wait_st();
        }
        if (edge) {
          const int b = rows2 ? x >> 1 : x, k0 = block_key<kWindow>(sg.t, sg.blk + b);
          const int t_v = 2 * (kb + b) + 1, st = t_v % R::kStages;
          if (ok) ok = wait_for<!kEight>(&ctl->full[st], (t_v / R::kStages) & 1, ctl, P.wait_ns);
          // (a unit of two row tiles: both streams use the values)
          if (ok)
            clean_values<T, D>(ring + st * R::kTile, kWindow && x < x_low ? 0 : max(sg.t.ctx - k0, 0),
                               min(block_end<kWindow>(sg.t, sg.blk + b) - k0, kKeyBlock), rows2 ? tid : row, rows2 ? 256 : 128,
                               ctl);
          if (rows2) named_sync(3, 256);
          else named_sync(1 + w, 128);
        }
        tc_fence_before();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&ctl->p_full[w]);
      }
      if (ok) ok = wait_for<!kEight>(&ctl->o_done, seg & 1, ctl, P.wait_ns);
      // (the streams' maxima and sums); all threads decide alike whether to go on
      const bool both = !rows2 && items > 1;
      ctl->ml[w][row] = {m, l};
      ok = !named_any(4, 256, !ok);
      if (!ok) break;
      tc_fence_after();
      const int wa = rows2 ? w : g0 & 1;  // the stream of the row's first step
      float f0 = 1.f, f1 = 0.f;
      if (!rows2) {
        const float2 a = ctl->ml[wa][row];
        m = a.x;
        l = a.y;
        if (both) {
          const float2 z = ctl->ml[wa ^ 1][row];
          m = fmaxf(a.x, z.x);
          const float mm = m == -INFINITY ? 0.f : m;
          f0 = ex2_approx((a.x - mm) * sc);
          f1 = ex2_approx((z.x - mm) * sc);
          l = a.y * f0 + z.y * f1;
        }
      }
      // a unit of two row tiles: a warpgroup its rows' sums; else each half of
      // them, both streams' added up
      const int nb = sg.nb, kind = sg.t.kind;
      const int lt = P.rep_div(row);
      const bool direct = nb == sg.t.blocks && kind == 0;
      const bool bad = ctl->bad && kind != 1;
      const int64_t q_row = ((int64_t)sg.t.tok0 + (rows2 ? tt * x0 : 0) + lt) * P.q_heads + sg.head * P.rep + row - lt * P.rep;
      int64_t slot = 0;
      if (!direct) {
        // a whole unit that is joined with others: the store of its kind; else
        // the first segment of a CTA's share, or its last
        slot = nb == sg.t.blocks ? (int64_t)2 * kKvCtas * P.plan.slot_rows + (kind == 1 ? P.plan.store : 0) + q_row
                                 : (int64_t)(2 * blockIdx.x + (seg > 0)) * P.plan.slot_rows + (rows2 ? kRows * x0 : 0) + row;
      }
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
      const int cols = rows2 ? D : D / 2, d0 = rows2 ? 0 : w * (D / 2);
      const uint32_t a0 = tO + lanes + 128 * wa + d0, a1 = tO + lanes + 128 * (wa ^ 1) + d0;
#pragma unroll 1
      for (int d = 0; d < cols; d += 16) {
        uint32_t u[16], v[16];
        if (busy) {
          tmem_ld16(a0 + d, u);
          if (both) tmem_ld16(a1 + d, v);
          tmem_wait_ld16(u);
          if (both) {
            tmem_wait_ld16(v);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              u[e] = __float_as_uint(__uint_as_float(u[e]) * f0 + __uint_as_float(v[e]) * f1);
          }
        }
        if (d + 16 >= cols) {  // O has been read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->o_free);
        }
        if (live) {
          if (direct) {
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              h[e] = H::pack(__uint_as_float(u[2 * e]) * inv, __uint_as_float(u[2 * e + 1]) * inv);
            store32(P.out + (q_row * D + d0 + d) * 2, h);
          } else {
            float* dst = P.plan.o + slot * D + d0 + d;
            store32(dst, u);
            store32(dst + 8, u + 8);
          }
        }
        __syncwarp();
      }
      if (bad && live) {
        auto add = [&](int from, int to, int first_seen) {
          add_unclean<T, kWindow, kEight>(P, sg.t.seq_row, sg.head, sg.t.ctx - 1, lim, first_seen, see, from, to, d0, cols,
                                  direct ? P.out + (q_row * D + d0) * 2 : nullptr, P.plan.o + slot * D + d0);
        };
        if (!kWindow) {
          add(max(sg.t.ctx, sg.t.kbeg + sg.blk * kKeyBlock), min(sg.t.kend, sg.t.kbeg + (sg.blk + nb) * kKeyBlock), 0);
        } else {
#pragma unroll 1
          for (int b = sg.blk; b < sg.blk + nb; ++b) {  // the parts of its blocks that were cleaned
            const int k0 = block_key<kWindow>(sg.t, b), end = min(block_end<kWindow>(sg.t, b), k0 + kKeyBlock);
            const int mid = min(max(k0, sg.t.sinks), end);  // (keys before it stay visible)
            if (k0 < sg.t.low) add(k0, mid, 0);
            add(k0 < sg.t.low ? mid : max(sg.t.ctx, k0), end, k0 < sg.t.low ? low : 0);
          }
        }
      }
      if (live && !direct && (rows2 || w == 0)) P.plan.ml[slot] = {m == -INFINITY ? m : m * sc, l};
      last = sg.last;
      g0 += items;
      kb += nb;
      qt += rows2 ? 2 : 1;
      if (!last) {
        ok = next_segment(qt);
        if (!ok) ++seg;
        if (bad) {  // (rare: the flag is cleared between two barriers)
          if (tid == 0) ctl->bad = 0;
          named_sync(4, 256);
        }
      }
      if (!ok) break;
    }
    if (!ok) {
      // the sequences of this and the following units have no result
      int k = 0;
      for (Walk wk(P, kWindow); wk.more(); wk.next(P), ++k)
        if (k >= seg) {
          const int end = (wk.t.tok0 + wk.t.toks - 1) / P.N;
          for (int j = wk.t.tok0 / P.N + tid; j <= end; j += 256) P.plan.status[j] = SAMSPEC_ST_TIMEOUT;
        }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (vload(&ctl->abort)) {
    // Given up, by whichever role: no role issues any more, and what is in flight
    // has to land before the CTA's shared and tensor memory go.  (A role cannot
    // see to that when it ends: it may have issued its last copy or product, and
    // met no wait that ran out, before another one gives up.)
    if (warp == 8) {
      const int kt = ctl->asked, qt = ctl->asked_q;
      for (int t = max(qt - 2, 0); t < qt; ++t) drain_wait(&ctl->q_full[t & 1], (t >> 1) & 1);
      if constexpr (kEight) {
        for (int t = max(kt - R::kStages8, 0); t < kt; ++t)
          drain_wait(&ctl->full8[t % R::kStages8], (t / R::kStages8) & 1);
      } else {
        for (int t = max(kt - R::kStages, 0); t < kt; ++t)
          drain_wait(&ctl->full[t % R::kStages], (t / R::kStages) & 1);
      }
    } else if (tid == 9 * 32) {  // (the thread that has issued them)
      mma_commit(&ctl->drain);
      drain_wait(&ctl->drain, 0);
    }
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 9) tmem_free(tmem, 512);
}

// ---- joining partial results ---------------------------------------------------
// Row `at` of a cut unit: where its part of CTA c0 lies (that one's first
// segment, or its last), and of CTA c0 + 1 (the first; the others follow 2 *
// slot_rows apart).
__device__ __forceinline__ int2 part_slots(const PlanView& p, int ti, int h, int c0, int at) {
  const int4 st = p.start[c0];
  const bool begins = st.x == ti && st.y == h && st.z == 0;
  return {(2 * c0 + !begins) * p.slot_rows + at, 2 * (c0 + 1) * p.slot_rows + at};
}

// 16 columns of a row (from d0 on) of its parts, added up by a thread, two in
// flight at once: `cnt` of them, the first at slot `first`, the others from
// `rest` on.
template <typename T, int D>
__device__ __forceinline__ void join_piece(const AttendParams& P, int64_t row, int d0, int cnt, int first, int rest) {
  using H = Type16<T>;
  constexpr int kDeep = 2;
  float m = -INFINITY, l = 0.f, o[16] = {};
#pragma unroll 1
  for (int q = 0; q < cnt; q += kDeep) {
    float2 z[kDeep];
    float4 a[kDeep][4];
#pragma unroll
    for (int e = 0; e < kDeep; ++e) {
      const int k = q + e;
      if (k < cnt) {
        const int64_t slot = k == 0 ? first : rest + (int64_t)(k - 1) * 2 * P.plan.slot_rows;
        z[e] = P.plan.ml[slot];
#pragma unroll
        for (int d = 0; d < 4; ++d) a[e][d] = reinterpret_cast<const float4*>(P.plan.o + slot * D + d0)[d];
      }
    }
#pragma unroll
    for (int e = 0; e < kDeep; ++e)
      if (q + e < cnt) {
        const float mn = fmaxf(m, z[e].x), mm = mn == -INFINITY ? 0.f : mn;
        const float f = exp2f(m - mm), g = exp2f(z[e].x - mm);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          o[4 * d] = o[4 * d] * f + a[e][d].x * g;
          o[4 * d + 1] = o[4 * d + 1] * f + a[e][d].y * g;
          o[4 * d + 2] = o[4 * d + 2] * f + a[e][d].z * g;
          o[4 * d + 3] = o[4 * d + 3] * f + a[e][d].w * g;
        }
        l = l * f + z[e].y * g;
        m = mn;
      }
  }
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
  uint32_t h[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] = H::pack(o[2 * e] * inv, o[2 * e + 1] * inv);
  store32(P.out + (row * D + d0) * 2, h);
}

// Without groups only units that were cut among CTAs are joined: `parts` CTAs
// for each, a thread 16 columns of a row.  Bound by latency (the plan holds
// where a unit's parts lie, since finding that here took 3 reads after one
// another) and, for units of 256 rows, by the parts' bytes: of prompt chunks'
// 114 us the join takes 13.  (Parts added up by the CTA that is done last, in
// the attention kernel: 27 us, on one SM what this spreads over eight.)
template <typename T, int D>
__global__ void __launch_bounds__(256) join_cut_kernel(AttendParams P, int parts) {
  wait_for_previous();
  let_next_start();
  const int joins = (kKvCtas - 1) * parts;
  if (blockIdx.x >= joins) {
    // four tokens a warp, neighbours to different ones: those that take no part
    // lie side by side
    const int warps = (gridDim.x - joins) * 8, lane = threadIdx.x & 31;
    const int t0 = (blockIdx.x - joins) * 8 + (threadIdx.x >> 5), tok = t0 + lane * warps;
    const bool dead = lane < 4 && tok < P.n * P.N && tok % P.N >= P.plan.seq[tok / P.N].ntok;
    for (uint32_t todo = __ballot_sync(kFullMask, dead); todo; todo &= todo - 1) {
      uint4* out = reinterpret_cast<uint4*>(P.out + (int64_t)(t0 + (__ffs(todo) - 1) * warps) * P.q_heads * D * 2);
      for (int x = lane; x < P.q_heads * (D / 8); x += 32) out[x] = uint4{0, 0, 0, 0};
    }
    return;
  }
  const KvJoin j = P.plan.join[blockIdx.x / parts + 1];
  const int tt = tile_tokens(P.rep);
  for (int x = blockIdx.x % parts * 256 + threadIdx.x; x < j.toks * P.rep * (D / 16); x += 256 * parts) {
    const int r = x / (D / 16), lt = P.rep_div(r);
    const int at = r + (lt >= tt ? kRows - tt * P.rep : 0);  // the second tile's rows from kRows on
    const int64_t row = ((int64_t)j.tok0 + lt) * P.q_heads + j.head * P.rep + r - lt * P.rep;
    join_piece<T, D>(P, row, x % (D / 16) * 16, j.parts, j.first + at, j.rest + at);
  }
}

// A row's parts added up by a warp, four in flight at once: `cnt` of them, the
// first n0 from f0, then s0 on, the others from f1, then s1 on.
template <typename T, int D>
__device__ __forceinline__ void join_row(const AttendParams& P, int64_t row, int cnt, int n0, int f0, int s0, int f1,
                                         int s1, int lane) {
  using H = Type16<T>;
  constexpr int kPer = D / 32;
  struct alignas(4 * kPer) Vec {
    float x[kPer];
  };
  float m = -INFINITY, l = 0.f, o[kPer] = {};
  for (int q = 0; q < cnt; q += 4) {
    float2 z[4];
    Vec a[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int k = q + e;
      z[e] = {-INFINITY, 0.f};
      if (k < cnt) {
        const int j = k < n0 ? k : k - n0;
        const int64_t slot = j == 0 ? (k < n0 ? f0 : f1) : (k < n0 ? s0 : s1) + (int64_t)(j - 1) * 2 * P.plan.slot_rows;
        z[e] = P.plan.ml[slot];
        a[e] = *reinterpret_cast<const Vec*>(P.plan.o + slot * D + lane * kPer);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (q + e < cnt) {
        const float mn = fmaxf(m, z[e].x), mm = mn == -INFINITY ? 0.f : mn;
        const float f = exp2f(m - mm), g = exp2f(z[e].x - mm);
#pragma unroll
        for (int d = 0; d < kPer; ++d) o[d] = o[d] * f + a[e].x[d] * g;
        l = l * f + z[e].y * g;
        m = mn;
      }
  }
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
  uint32_t* out = reinterpret_cast<uint32_t*>(P.out + row * D * 2) + lane * (kPer / 2);
#pragma unroll
  for (int e = 0; e < kPer / 2; ++e) out[e] = H::pack(o[2 * e] * inv, o[2 * e + 1] * inv);
}

// With groups: a warp takes 8 rows, a lane finds where one row's parts lie
// (none where it was written at once), then the warp adds up one after the
// other.
constexpr int kJoinRows = 8;
template <typename T, int D>
__global__ void __launch_bounds__(256) join_rows_kernel(AttendParams P) {
  const int lane = threadIdx.x & 31;
  const int64_t rows = (int64_t)P.n * P.N * P.q_heads;
  const int64_t r0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * kJoinRows;
  wait_for_previous();
  let_next_start();
  if (r0 >= rows) return;
  // of lane's row: parts (-1: none to join, 0: zeros), and for the shared and
  // the own keys where the first part lies and where the others begin
  int parts = -1, first[2] = {0, 0}, rest[2] = {0, 0}, cnt[2] = {0, 0};
  const int64_t mine = r0 + lane;
  if (lane < kJoinRows && mine < rows) {
    const int hq = (int)(mine % P.q_heads);
    const int64_t tok = mine / P.q_heads;
    const int i = (int)(tok / P.N), node = (int)(tok % P.N);
    const KvSeq s = P.plan.seq[i];
    if (node >= s.ntok) {
      parts = 0;
    } else {
      const int h = hq / P.rep, tt = tile_tokens(P.rep);
      const int ctas = P.plan.hdr[kHdrCtas], cost = P.plan.hdr[kHdrCost];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        if (p == 0 && s.shared == 0) continue;
        const int ft = p ? node : (i - s.leader) * P.N + node, lt = ft % (2 * tt);
        const int at = lt / tt * kRows + lt % tt * P.rep + hq % P.rep;  // its row of the unit
        const int ti = (p ? P.plan.suf0[i] : P.plan.pre0[s.leader]) + ft / (2 * tt);
        const int2 c = unit_ctas(P.plan.tile[ti], h, ctas, cost);
        cnt[p] = c.y - c.x + 1;
        if (c.x == c.y) {
          if (s.shared == 0) cnt[p] = 0;
          first[p] = (int)(2 * kKvCtas * P.plan.slot_rows + (p ? 0 : P.plan.store) + mine);
        } else {
          const int2 f = part_slots(P.plan, ti, h, c.x, at);
          first[p] = f.x;
          rest[p] = f.y;
        }
      }
      parts = cnt[0] + cnt[1];
      if (parts == 0) parts = -1;
    }
  }
  for (uint32_t todo = __ballot_sync(kFullMask, parts >= 0); todo; todo &= todo - 1) {
    const int w = __ffs(todo) - 1;
    const int n = __shfl_sync(kFullMask, parts, w), n0 = __shfl_sync(kFullMask, cnt[0], w);
    const int f0 = __shfl_sync(kFullMask, first[0], w), f1 = __shfl_sync(kFullMask, first[1], w);
    const int s0 = __shfl_sync(kFullMask, rest[0], w), s1 = __shfl_sync(kFullMask, rest[1], w);
    join_row<T, D>(P, r0 + w, n, n0, f0, s0, f1, s1, lane);
  }
}

// a pool as [layers * n_pages][kv_heads * page][head_dim], in boxes of one
// page and head, 64 elements wide
int pool_map(const KvView& c, int32_t dtype, void* pool, CUtensorMap* map) {
  const EncodeTiled enc = encode_tiled();
  if (!enc) return SAMSPEC_ECUDA;
  const cuuint64_t dims[3] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.kv_heads * c.page, (cuuint64_t)c.layers * c.n_pages};
  const cuuint64_t strides[2] = {(cuuint64_t)c.head_dim * 2, (cuuint64_t)c.kv_heads * c.page * c.head_dim * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)c.page, 1}, one[3] = {1, 1, 1};
  return enc(map, dtype == SAMSPEC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, pool,
             dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? SAMSPEC_OK
             : SAMSPEC_ECUDA;
}

// queries as [tokens][kv_heads][rep][head_dim], in boxes of one tile's tokens
// of one key head, 64 elements wide
int query_map(const AttendParams& P, int32_t dtype, CUtensorMap* map) {
  const EncodeTiled enc = encode_tiled();
  if (!enc) return SAMSPEC_ECUDA;
  const cuuint64_t D = P.c.head_dim, rep = P.rep;
  const cuuint64_t dims[4] = {D, rep, (cuuint64_t)P.c.kv_heads, (cuuint64_t)P.n * P.N};
  const cuuint64_t strides[3] = {D * 2, rep * D * 2, (cuuint64_t)P.q_stride * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)rep, 1, (cuuint32_t)tile_tokens(P.rep)}, one[4] = {1, 1, 1, 1};
  return enc(map, dtype == SAMSPEC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
             const_cast<unsigned char*>(P.q), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? SAMSPEC_OK
             : SAMSPEC_ECUDA;
}

template <typename T, int D>
int attend(AttendParams P, bool window, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mq,
           cudaStream_t s) {
  constexpr bool kBf16 = Type16<T>::kFormat == 1;
  if (few_rows(P.c, P.N, P.rep, P.plan.store != 0)) {
    if (attend_few(P, kBf16, window, s) != SAMSPEC_OK) return SAMSPEC_ECUDA;
  } else {
    const bool eight = P.c.elt == 1;
    const auto kernel = eight ? window ? attend_kernel<T, D, true, true> : attend_kernel<T, D, false, true>
                              : window ? attend_kernel<T, D, true, false> : attend_kernel<T, D, false, false>;
    const int bytes = eight ? Ring<D, true>::kBytes : Ring<D, false>::kBytes;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
      return SAMSPEC_ECUDA;
    P.lazy = Type16<T>::kLazy / P.scale_log2;
    if (launch_after(kernel, kKvCtas, eight ? Ring<D, true>::kThreads : Ring<D, false>::kThreads, bytes, s, P, mk, mv, mq) != cudaSuccess)
      return SAMSPEC_ECUDA;
  }
  const int64_t toks = (int64_t)P.n * P.N;
  const int parts = (P.plan.slot_rows * (D / 16) + 255) / 256;
  const cudaError_t e =
      P.plan.store ? launch_after(join_rows_kernel<T, D>, (unsigned)((toks * P.q_heads + 8 * kJoinRows - 1) / (8 * kJoinRows)),
                                  256, 0, s, P)
                   : launch_after(join_cut_kernel<T, D>, (unsigned)((kKvCtas - 1) * parts + (toks + 31) / 32), 256, 0, s, P,
                                  parts);
  return e == cudaSuccess ? launched() : SAMSPEC_ECUDA;
}

// the layout that plan_bytes bytes were asked for
bool plan_of(const KvView& c, int32_t n, int32_t N, int32_t q_heads, size_t bytes, PlanLayout* l) {
  *l = plan_layout(c, n, N, q_heads, true);
  if (l->bytes && bytes >= l->bytes) return true;
  *l = plan_layout(c, n, N, q_heads, false);
  return l->bytes && bytes >= l->bytes;
}

int plan_pass(const kv_cache* cache, const int32_t* d_rows, int32_t n, int32_t N, int32_t q_heads,
              const int32_t* d_n_tok, const int32_t* d_first_child, const int32_t* d_next_sibling,
              const int32_t* d_group, int32_t window, int32_t sinks, void* d_plan, size_t plan_bytes,
              samspec_stream_t stream) {
  PlanParams P;
  const int rc = kv_view(cache, &P.c);
  if (rc != SAMSPEC_OK) return rc;
  if (!d_plan || !d_first_child != !d_next_sibling) return SAMSPEC_EINVAL;
  PlanLayout l;
  if (!plan_of(P.c, n, N, q_heads, plan_bytes, &l) || (d_group && !l.store) ||
      (d_first_child && N > 32) || (!d_rows && n > P.c.seqs))
    return SAMSPEC_ESIZE;
  if (reinterpret_cast<uintptr_t>(d_plan) % 256 != 0) return SAMSPEC_EALIGN;
  P.plan = plan_view(d_plan, l);
  P.rows = d_rows;
  P.n_tok = d_n_tok;
  P.first_child = d_first_child;
  P.next_sibling = d_next_sibling;
  P.group = d_group;
  P.window = window;
  P.sinks = sinks;
  P.n = n;
  P.N = N;
  P.rep = q_heads / P.c.kv_heads;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // up to 32 sequences, a warp each, are judged by the units' CTA: one launch
  // less (at 64, two a warp, a step of 64 trees took 232 us instead of 224)
  const bool few = n <= 32;
  if ((!few && launch_after(plan_sequences_kernel, (n + 7) / 8, 256, 0, s, P) != cudaSuccess) ||
      launch_after(plan_units_kernel, 1, 1024, 0, s, P, few) != cudaSuccess)
    return SAMSPEC_ECUDA;
  return launched();
}

int attend_pass(const kv_cache* cache, int32_t layer, void* d_plan, size_t plan_bytes, int32_t n,
                int32_t N, int32_t q_heads, const void* d_q, int64_t q_stride, float scale,
                void* d_out, bool window, samspec_stream_t stream) {
  AttendParams P;
  const int rc = kv_view(cache, &P.c);
  if (rc != SAMSPEC_OK) return rc;
  if (!d_plan || !d_q || !d_out || layer < 0 || layer >= P.c.layers || !(scale > 0) ||
      !std::isfinite(scale * 1.4426950408889634f))
    return SAMSPEC_EINVAL;
  PlanLayout l;
  if (!plan_of(P.c, n, N, q_heads, plan_bytes, &l)) return SAMSPEC_ESIZE;
  if (q_stride < (int64_t)q_heads * P.c.head_dim) return SAMSPEC_EINVAL;
  if (reinterpret_cast<uintptr_t>(d_q) % 16 != 0 || reinterpret_cast<uintptr_t>(d_out) % 32 != 0 || q_stride % 8 != 0 ||
      reinterpret_cast<uintptr_t>(d_plan) % 256 != 0)
    return SAMSPEC_EALIGN;
  P.plan = plan_view(d_plan, l);
  P.layer = layer;
  P.n = n;
  P.N = N;
  P.q_heads = q_heads;
  P.rep = q_heads / P.c.kv_heads;
  P.rep_div = Divider((uint32_t)P.rep);
  P.q = static_cast<const unsigned char*>(d_q);
  P.q_stride = q_stride;
  P.scale_log2 = scale * 1.4426950408889634f;
  P.out = static_cast<unsigned char*>(d_out);
  const uint64_t limit = g_kv_wait_ns.load(), most = (uint64_t)1 << 41;  // (wait_for counts 32 bits of 1024 ns)
  P.wait_ns = limit < most ? limit : most;
  CUtensorMap mk = {}, mv = {}, mq;
  const int32_t io = io_dtype(cache);
  if (query_map(P, io, &mq) != SAMSPEC_OK) return SAMSPEC_ECUDA;
  if (P.c.elt == 2 && (pool_map(P.c, io, cache->k, &mk) != SAMSPEC_OK || pool_map(P.c, io, cache->v, &mv) != SAMSPEC_OK))
    return SAMSPEC_ECUDA;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (io == SAMSPEC_BF16)
    return cache->head_dim == 64 ? attend<__nv_bfloat16, 64>(P, window, mk, mv, mq, s)
                                 : attend<__nv_bfloat16, 128>(P, window, mk, mv, mq, s);
  return cache->head_dim == 64 ? attend<__half, 64>(P, window, mk, mv, mq, s)
                               : attend<__half, 128>(P, window, mk, mv, mq, s);
}

}  // namespace
}  // namespace samspec

using namespace samspec;

extern "C" {

size_t kv_plan_bytes(const kv_cache* cache, int32_t n, int32_t N, int32_t q_heads, int32_t grouped) {
  KvView c;
  if (kv_view(cache, &c) != SAMSPEC_OK) return 0;
  return plan_layout(c, n, N, q_heads, grouped != 0).bytes;
}

int kv_plan(const kv_cache* cache, const int32_t* d_rows, int32_t n, int32_t N, int32_t q_heads,
            const int32_t* d_n_tok, const int32_t* d_first_child, const int32_t* d_next_sibling,
            const int32_t* d_group, void* d_plan, size_t plan_bytes, samspec_stream_t stream) {
  return plan_pass(cache, d_rows, n, N, q_heads, d_n_tok, d_first_child, d_next_sibling, d_group, 0, 0, d_plan,
                   plan_bytes, stream);
}

int kv_plan_window(const kv_cache* cache, const int32_t* d_rows, int32_t n, int32_t N, int32_t q_heads,
                   const int32_t* d_n_tok, const int32_t* d_first_child, const int32_t* d_next_sibling,
                   int32_t window, int32_t sinks, void* d_plan, size_t plan_bytes, samspec_stream_t stream) {
  if (window < 1 || sinks < 0) return SAMSPEC_EINVAL;
  // (longer than any cache is as good as all of it, and its sums stay in 32 bits)
  const int32_t most = 1 << 30;
  return plan_pass(cache, d_rows, n, N, q_heads, d_n_tok, d_first_child, d_next_sibling, nullptr,
                   window < most ? window : most, sinks < most ? sinks : most, d_plan, plan_bytes, stream);
}

int kv_attend(const kv_cache* cache, int32_t layer, void* d_plan, size_t plan_bytes, int32_t n,
              int32_t N, int32_t q_heads, const void* d_q, int64_t q_stride, float scale,
              void* d_out, samspec_stream_t stream) {
  return attend_pass(cache, layer, d_plan, plan_bytes, n, N, q_heads, d_q, q_stride, scale, d_out, false, stream);
}

int kv_attend_window(const kv_cache* cache, int32_t layer, void* d_plan, size_t plan_bytes,
                     int32_t n, int32_t N, int32_t q_heads, const void* d_q, int64_t q_stride,
                     float scale, void* d_out, samspec_stream_t stream) {
  return attend_pass(cache, layer, d_plan, plan_bytes, n, N, q_heads, d_q, q_stride, scale, d_out, true, stream);
}

uint64_t kv_set_wait_limit_ns(uint64_t ns) {
  return g_kv_wait_ns.exchange(ns == 0 ? 2000000000ull : ns);
}

}  // extern "C"
