// attend.cu -- the plan of a verification pass and its attention over the
// paged cache.
#include "common.cuh"
#include "kv.cuh"

#include <atomic>
#include <cmath>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

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
  int n, N, q_heads, rep;
};

// One warp a sequence: its lengths and pages checked, the tree's depths and
// ancestors, the pages that it shares with the first sequence of its group.
__global__ void __launch_bounds__(256) plan_sequences_kernel(PlanParams P) {
  const KvView& c = P.c;
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (i >= P.n) return;
  int st = SAMSPEC_ST_OK;
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
    const int32_t* fc = P.first_child + (int64_t)i * P.N;
    const int32_t* ns = P.next_sibling + (int64_t)i * P.N;
    const int N = P.N;
    int first = -1, next = -1;
    if (lane < N) {
      first = fc[lane];
      next = ns[lane];
    }
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
    for (int k = lane; k < pages; k += 32) {
      const int p = t[k];
      const bool out = p < 0 || p >= c.n_pages;
      bad |= out;
      // a page that is written has to be the sequence's alone
      if (!out && k >= full && nt > 0) lent |= c.refs[p] > 1;
    }
    if (__any_sync(kFullMask, bad)) st = SAMSPEC_ST_PAGE;
    else if (__any_sync(kFullMask, lent)) st = SAMSPEC_ST_CAPACITY;
    if (st == SAMSPEC_ST_OK && P.group) {
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
      if (leader != i) {
        const int lrow = P.rows ? P.rows[leader] : leader;
        int lfull = 0;
        if (lrow >= 0 && lrow < c.seqs) {
          const int ll = c.lens[lrow];
          lfull = ll > 0 ? min(ll >> c.log_page, c.max_pages) : 0;
        }
        const int m = min(full, lfull);
        const int32_t* tl = c.table + (int64_t)(m ? lrow : 0) * c.max_pages;
        int same = m;
        for (int k = 0; k < m; k += 32) {
          const uint32_t differ = __ballot_sync(kFullMask, k + lane < m && t[k + lane] != tl[k + lane]);
          if (differ) {
            same = k + __ffs(differ) - 1;
            break;
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

// One CTA: what a group reads once, the units of work and their order, and
// each persistent CTA's equal share of the key blocks.
constexpr int kMinShared = 128;  // tokens: less is read by each sequence for itself

__global__ void __launch_bounds__(1024) plan_units_kernel(PlanParams P) {
  __shared__ int part[32];
  const KvView& c = P.c;
  const int tid = threadIdx.x, n = P.n;
  const int rows = P.N * P.rep;  // of one sequence and key head
  KvSeq* seq = P.plan.seq;
  if (P.group) {
    for (int i = tid; i < n; i += 1024)
      if (seq[i].ntok > 0 && seq[i].leader == i) {
        seq[i].shared = seq[i].lcp;
        seq[i].gsize = 1;
      }
    __syncthreads();
    for (int i = tid; i < n; i += 1024)
      if (seq[i].leader != i) {
        // the group's extent counts every member; those without new tokens
        // bring no rows and set no limit
        atomicMax(&seq[seq[i].leader].gsize, i - seq[i].leader + 1);
        if (seq[i].ntok > 0) atomicMin(&seq[seq[i].leader].shared, seq[i].lcp);
      }
    __syncthreads();
    for (int i = tid; i < n; i += 1024)
      if (seq[i].leader == i && (seq[i].gsize < 2 || seq[i].shared < kMinShared)) seq[i].shared = 0;
    __syncthreads();
    for (int i = tid; i < n; i += 1024)
      if (seq[i].leader != i) seq[i].shared = seq[i].ntok > 0 ? seq[seq[i].leader].shared : 0;
    __syncthreads();
  }
  // tiles of the groups' shared keys, then of each sequence's own
  int tiles = 0;
  for (int pass = P.group ? 0 : 1; pass < 2; ++pass)
    for (int i0 = 0; i0 < n; i0 += 1024) {
      const int i = i0 + tid;
      int cnt = 0;
      if (i < n) {
        if (pass == 0) {
          if (seq[i].leader == i && seq[i].shared > 0) cnt = (seq[i].gsize * rows + kTileRows - 1) / kTileRows;
        } else {
          cnt = (seq[i].ntok * P.rep + kTileRows - 1) / kTileRows;
        }
      }
      int sum;
      const int at = tiles + block_scan(cnt, part, &sum);
      if (i < n) (pass ? P.plan.suf0 : P.plan.pre0)[i] = at;
      for (int k = 0; k < cnt; ++k) {
        KvTile t;
        t.i0 = i;
        t.row0 = k * kTileRows;
        t.prefix = pass == 0;
        if (pass == 0) {
          t.rows = min(kTileRows, seq[i].gsize * rows - t.row0);
          t.kbeg = 0;
          t.kend = seq[i].shared;
        } else {
          t.rows = min(kTileRows, seq[i].ntok * P.rep - t.row0);
          t.kbeg = seq[i].shared;
          // a chain's tile sees no further than its last token
          t.kend = seq[i].base + (P.first_child ? seq[i].ntok : (t.row0 + t.rows - 1) / P.rep + 1);
        }
        t.blocks = (t.kend - t.kbeg + kKeyBlock - 1) / kKeyBlock;
        t.cost0 = 0;
        P.plan.tile[at + k] = t;
      }
      tiles += sum;
    }
  __syncthreads();
  int cost = 0;
  for (int t0 = 0; t0 < tiles; t0 += 1024) {
    const int t = t0 + tid;
    int sum;
    const int at = block_scan(t < tiles ? P.plan.tile[t].blocks * c.kv_heads : 0, part, &sum);
    if (t < tiles) P.plan.tile[t].cost0 = cost + at;
    cost += sum;
  }
  __syncthreads();
  const int ctas = min(kKvCtas, cost);
  for (int x = tid; x <= ctas; x += 1024) {
    const int b = ctas ? (int)((int64_t)x * cost / ctas) : 0;
    int lo = 0, hi = tiles - 1;  // the last tile that begins at or before b
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (P.plan.tile[mid].cost0 <= b) lo = mid;
      else hi = mid - 1;
    }
    int4 s = {0, 0, 0, b};
    if (x < ctas) {
      const KvTile t = P.plan.tile[lo];
      s.x = lo;
      s.y = (b - t.cost0) / t.blocks;
      s.z = (b - t.cost0) % t.blocks;
    }
    P.plan.start[x] = s;
  }
  if (tid == 0) {
    P.plan.hdr[kHdrTiles] = tiles;
    P.plan.hdr[kHdrCtas] = ctas;
    P.plan.hdr[kHdrCost] = cost;
    P.plan.hdr[kHdrTree] = P.first_child != nullptr;
    P.plan.hdr[kHdrTimeout] = 0;
  }
}

// ---- attention ---------------------------------------------------------------
struct AttendParams {
  KvView c;
  PlanView plan;
  int layer, n, N, q_heads, rep;
  const unsigned char* q;
  int64_t q_stride;
  float scale_log2;  // scale * log2(e)
  unsigned char* out;
};

template <typename T>
__device__ __forceinline__ float to_f(T x) { return (float)x; }

// One warp a query row, keys one after the other.
template <typename T>
__global__ void __launch_bounds__(256) attend_rows_kernel(AttendParams P) {
  const KvView& c = P.c;
  const int lane = threadIdx.x & 31, D = c.head_dim;
  const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= (int64_t)P.n * P.N * P.q_heads) return;
  const int h = (int)(r % P.q_heads);
  const int64_t tok = r / P.q_heads;
  const int i = (int)(tok / P.N), node = (int)(tok % P.N);
  const KvSeq s = P.plan.seq[i];
  T* out = reinterpret_cast<T*>(P.out) + r * D;
  if (node >= s.ntok) {
    for (int d = lane; d < D; d += 32) out[d] = (T)0.f;
    return;
  }
  const T* q = reinterpret_cast<const T*>(P.q) + tok * P.q_stride + h * D;
  const uint32_t see = P.plan.hdr[kHdrTree] ? (uint32_t)P.plan.node[tok].y : 0;
  const bool tree = P.plan.hdr[kHdrTree] != 0;
  float qv[4], o[4] = {0, 0, 0, 0}, m = -INFINITY, l = 0;
  for (int x = 0; x < D / 32; ++x) qv[x] = to_f(q[lane + 32 * x]);
  const int end = s.base + (tree ? s.ntok : node + 1);
  for (int key = 0; key < end; ++key) {
    if (tree && key >= s.base && !((see >> (key - s.base)) & 1)) continue;
    const int page = c.table[(int64_t)s.row * c.max_pages + (key >> c.log_page)];
    const int64_t at = kv_offset(c, P.layer, page, h / P.rep) + (int64_t)(key & (c.page - 1)) * D * 2;
    const T* k = reinterpret_cast<const T*>(c.k + at);
    const T* v = reinterpret_cast<const T*>(c.v + at);
    float a = 0;
    for (int x = 0; x < D / 32; ++x) a += qv[x] * to_f(k[lane + 32 * x]);
    a = warp_sum(a) * P.scale_log2;
    const float mn = fmaxf(m, a), f = mn == -INFINITY ? 1.f : exp2f(m - mn), p = exp2f(a - (mn == -INFINITY ? 0.f : mn));
    for (int x = 0; x < D / 32; ++x) o[x] = o[x] * f + p * to_f(v[lane + 32 * x]);
    l = l * f + p;
    m = mn;
  }
  for (int x = 0; x < D / 32; ++x) out[lane + 32 * x] = (T)(l > 0 || l != l ? o[x] / l : 0.f);
}

// the layout that plan_bytes bytes were asked for
bool plan_of(const KvView& c, int32_t n, int32_t N, int32_t q_heads, size_t bytes, PlanLayout* l) {
  *l = plan_layout(c, n, N, q_heads, true);
  if (l->bytes && bytes >= l->bytes) return true;
  *l = plan_layout(c, n, N, q_heads, false);
  return l->bytes && bytes >= l->bytes;
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
  P.n = n;
  P.N = N;
  P.q_heads = q_heads;
  P.rep = q_heads / P.c.kv_heads;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  plan_sequences_kernel<<<(n + 7) / 8, 256, 0, s>>>(P);
  plan_units_kernel<<<1, 1024, 0, s>>>(P);
  return launched();
}

int kv_attend(const kv_cache* cache, int32_t layer, void* d_plan, size_t plan_bytes, int32_t n,
              int32_t N, int32_t q_heads, const void* d_q, int64_t q_stride, float scale,
              void* d_out, samspec_stream_t stream) {
  AttendParams P;
  const int rc = kv_view(cache, &P.c);
  if (rc != SAMSPEC_OK) return rc;
  if (!d_plan || !d_q || !d_out || layer < 0 || layer >= P.c.layers || !std::isfinite(scale))
    return SAMSPEC_EINVAL;
  PlanLayout l;
  if (!plan_of(P.c, n, N, q_heads, plan_bytes, &l)) return SAMSPEC_ESIZE;
  if (q_stride < (int64_t)q_heads * P.c.head_dim) return SAMSPEC_EINVAL;
  if ((reinterpret_cast<uintptr_t>(d_q) | reinterpret_cast<uintptr_t>(d_out)) % 16 != 0 || q_stride % 8 != 0 ||
      reinterpret_cast<uintptr_t>(d_plan) % 256 != 0)
    return SAMSPEC_EALIGN;
  P.plan = plan_view(d_plan, l);
  P.layer = layer;
  P.n = n;
  P.N = N;
  P.q_heads = q_heads;
  P.rep = q_heads / P.c.kv_heads;
  P.q = static_cast<const unsigned char*>(d_q);
  P.q_stride = q_stride;
  P.scale_log2 = scale * 1.4426950408889634f;
  P.out = static_cast<unsigned char*>(d_out);
  const int64_t rows = (int64_t)n * N * q_heads;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cache->dtype == SAMSPEC_BF16)
    attend_rows_kernel<__nv_bfloat16><<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(P);
  else
    attend_rows_kernel<__half><<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(P);
  return launched();
}

uint64_t kv_set_wait_limit_ns(uint64_t ns) {
  return g_kv_wait_ns.exchange(ns == 0 ? 2000000000ull : ns);
}

}  // extern "C"
