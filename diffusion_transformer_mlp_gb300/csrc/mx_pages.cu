// The pages of the paged cache: reference counts, block table and lengths on the
// device, and copies of pages.
//
// The state is small (a few hundred KB of counts and table entries), so what
// counts is launches.  Growing and compacting need ranks of free or held pages
// over the whole pool: one cluster of eight blocks takes the pool in eight
// contiguous parts, a warp a contiguous piece of one, and the parts' counts meet
// behind a cluster barrier, where separate kernels would meet at a launch.  Free
// pages are taken in the order of their ids, so that the same state gives the
// same ids whatever the timing; counts are changed by atomics whose sums do not
// depend on their order.
//
// What bounds them: latency.  Growing 60 forked rows by a token takes 5 us (7.9 under a
// profiler: 2 to the growth of each row, 1 to their sums, 1 to the pool's counts, 1.5 to
// take the pages, 1.5 for the slots), 56 rows by 27,000 pages of a pool of 48,000 and
// 440,000 slots 11.6 + 4.9 us; selecting rows 2.5 to 3.5 us, making a pool of 9,000
// pages compact 5.4 + 2.4 us.  Code that runs once costs its fetching, so loops stay
// loops.  Copies are bound by HBM: 1,500 pages of 69 KB (208 MB moved) in 32.6 us, 94%
// of the copy rate.
//
// What one block writes and another reads inside a kernel is read from L2
// (__ldcg): the barrier orders it, and L1 may hold what was there before.
#include <algorithm>
#include <atomic>
#include <string>

#include "mx_common.cuh"

namespace nvfp4 {

nvfp4_status check_cache(const mxfp4_cache* cache, int* page_shift, const std::string& nm);

namespace {

constexpr int kCluster = 8;
constexpr int kThreads = 1024;  // of a block of the cluster
constexpr int kWarps = kThreads / 32;
constexpr int kGridThreads = 256;  // of the kernels over rows, tokens and bytes
constexpr int64_t kSmallTable = 1 << 16;  // table entries that one cluster works on

struct PagesParams {
  int32_t* refs;
  int32_t* table;
  int32_t* lens;
  int64_t pages, table_ld;
  int32_t rows, shift;
  // arguments
  const int32_t* in;  // sources or counts
  int64_t total;
  int64_t* slots;
  int32_t* pairs;   // copies [rows, 2] or moves [pages / 2, 2]
  int32_t* number;  // missing or used
  // workspace
  int64_t* need;     // [rows + 1] pages that the rows before need; of select: new lengths as int32
  int64_t* tokens;   // [rows + 1] new tokens of the rows before
  int64_t* part;     // of compact: held pages below their number
  int32_t* list;     // [pages] free ids in order; of compact: held ids in order
  int32_t* writers;  // [pages] rows that go on in a shared page; of compact: holes in order
  int32_t* lowest;   // [pages] the first of them; of compact: where a page goes
  int32_t* taken;    // [rows, table_ld] of select
};

// The aligned forms are for whole warps, and most of them stand behind loops that lanes
// leave at different times: the warp is brought together first.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// The same place in the shared memory of block `rank` of the cluster.
__device__ __forceinline__ void store_there(int64_t* mine, int rank, int64_t v) {
  asm volatile("{\n\t.reg .b32 there;\n\tmapa.shared::cluster.u32 there, %0, %1;\n\t"
               "st.shared::cluster.b64 [there], %2;\n\t}" ::"r"(smem_u32(mine)),
               "r"(rank), "l"(v)
               : "memory");
}

// Pages of a row of `len` tokens.
__device__ __forceinline__ int64_t held(const PagesParams& p, int64_t len) {
  const int64_t n = (max(len, int64_t(0)) + (int64_t(1) << p.shift) - 1) >> p.shift;
  return min(n, p.table_ld);
}
__device__ __forceinline__ bool is_page(const PagesParams& p, int32_t page) { return page >= 0 && page < p.pages; }

// How a row grows.
struct Growth {
  int64_t have, want;  // pages
  int32_t count;       // tokens
  int32_t last;        // the page that the next token goes into, if it holds some already; else -1
};
__device__ __forceinline__ Growth growth_of(const PagesParams& p, int32_t b) {
  Growth g;
  const int32_t len = max(p.lens[b], 0);
  g.count = max(p.in[b], 0);
  g.have = (int64_t(len) + (int64_t(1) << p.shift) - 1) >> p.shift;
  g.want = (int64_t(len) + g.count + (int64_t(1) << p.shift) - 1) >> p.shift;
  g.last = -1;
  if (g.count > 0 && (len & ((1 << p.shift) - 1)) != 0 && g.have <= p.table_ld)
    g.last = p.table[int64_t(b) * p.table_ld + g.have - 1];
  return g;
}

// This warp's piece of the pool: the ids [lo, hi).
struct Piece {
  int64_t lo, hi;
};
__device__ __forceinline__ Piece piece_of(int64_t pages, int rank, int warp) {
  const int64_t each = (pages + kCluster * kWarps - 1) / (kCluster * kWarps);
  const int64_t lo = min(pages, (int64_t(rank) * kWarps + warp) * each);
  return {lo, min(pages, lo + each)};
}
// Ids of the piece for which `held` is (or is not) so.
__device__ __forceinline__ int32_t count_piece(const PagesParams& p, const Piece& w, bool want_held) {
  const int lane = threadIdx.x & 31;
  int32_t n = 0;
#pragma unroll 8
  for (int64_t i = w.lo + lane; i < w.hi; i += 32) n += (p.refs[i] > 0) == want_held;
  return __reduce_add_sync(0xFFFFFFFFu, n);
}
// Ranks over the pool: `n` are in this warp's piece.  Returns those in the pieces
// before it; `all` gets the pool's.  The blocks push their sums into one another's
// shared memory (a round through L2 took 1.2 us instead of 0.4); they have arrived
// at the cluster's barrier once before, so that all are there.
struct Ranks {
  int64_t warp[kWarps], block[kCluster];
};
__device__ __forceinline__ int64_t rank_pieces(int32_t n, int rank, Ranks& r, int64_t& all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) r.warp[warp] = n;
  __syncthreads();
  cluster_wait();
  if (warp == 0) {
    const int64_t v = r.warp[lane];
    int64_t upto = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += u;
    }
    r.warp[lane] = upto - v;
    const int64_t sum = __shfl_sync(0xFFFFFFFFu, upto, 31);
    if (lane < kCluster) store_there(&r.block[rank], lane, sum);
    __syncwarp();
  }
  cluster_sync();
  int64_t before = r.warp[warp];
  all = 0;
#pragma unroll
  for (int i = 0; i < kCluster; ++i) {
    if (i < rank) before += r.block[i];
    all += r.block[i];
  }
  return before;
}

// The row of new token i: tokens[lo] <= i < tokens[lo + 1].
template <class F>
__device__ __forceinline__ int32_t row_of(int32_t rows, int64_t i, F tokens) {
  int32_t lo = 0, hi = rows;
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (tokens(mid) <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Up to so many new tokens get their slots from the cluster itself.
constexpr int64_t kInline = 4 * kCluster * kThreads;

// Sums over the rows of a block's threads: n and c become those up to this one.
__device__ __forceinline__ void scan_rows(int64_t& n, int64_t& c, int64_t (&sums)[2][kWarps]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t un = __shfl_up_sync(0xFFFFFFFFu, n, o), uc = __shfl_up_sync(0xFFFFFFFFu, c, o);
    if (lane >= o) n += un, c += uc;
  }
  if (lane == 31) sums[0][warp] = n, sums[1][warp] = c;
  __syncthreads();
  if (warp < 2) {
    int64_t upto = sums[warp][lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += u;
    }
    sums[warp][lane] = upto;
  }
  __syncthreads();
  if (warp > 0) n += sums[0][warp - 1], c += sums[1][warp - 1];
}

// The free pages that are needed: take(k, page) for the k-th of them.  `free_here`
// are in this warp's piece, `pages` are needed in all.  False, and none is taken,
// if there are too few (or `bad`).
template <class F>
__device__ __forceinline__ bool take_free(const PagesParams& p, int32_t free_here, int64_t pages, bool bad, int rank,
                                          Ranks& ranks, F take) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Piece mine = piece_of(p.pages, rank, warp);
  int64_t there, at = rank_pieces(free_here, rank, ranks, there);
  const bool ok = !bad && pages <= there;
  if (rank == 0 && threadIdx.x == 0) *p.number = bad ? -1 : int32_t(max(pages - there, int64_t(0)));
  if (!ok) return false;
  constexpr int kAtOnce = 8;  // loads under way: what is taken is stored between them
  for (int64_t i0 = mine.lo; i0 < mine.hi && at < pages; i0 += 32 * kAtOnce) {
    uint32_t of_lane = 0;  // lane u: which of the u-th 32 are free
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int64_t i = i0 + 32 * u + lane;
      const uint32_t all = __ballot_sync(0xFFFFFFFFu, i < mine.hi && p.refs[i] <= 0);
      if (lane == u) of_lane = all;
    }
#pragma unroll 1  // code that runs once costs its fetching (unrolled: 2.5 us more)
    for (int u = 0; u < kAtOnce; ++u) {
      const uint32_t all = __shfl_sync(0xFFFFFFFFu, of_lane, u);
      const int64_t k = at + __popc(all & ((1u << lane) - 1));
      if ((all >> lane & 1) && k < pages) take(k, int32_t(i0 + 32 * u + lane));
      at += __popc(all);
    }
  }
  return true;
}

// Row b takes its pages from place `first` of the list on, the copy (`own`) before
// the others; by a warp.
__device__ __forceinline__ void grow_row(const PagesParams& p, int32_t b, const Growth& g, int32_t len, int64_t first,
                                         int64_t own, bool ok) {
  const int lane = threadIdx.x & 31;
  int2 copy = make_int2(-1, -1);
  if (ok && g.count > 0) {
    int32_t* row = p.table + int64_t(b) * p.table_ld;
    const int64_t n = own + g.want - g.have;
    constexpr int kAtOnce = 8;
    for (int64_t i0 = lane; i0 < n; i0 += 32 * kAtOnce) {
      int32_t page[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
        if (i0 + 32 * u < n) page[u] = __ldcg(p.list + first + i0 + 32 * u);
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
        if (i0 + 32 * u < n) row[g.have - own + i0 + 32 * u] = page[u];
      if (i0 < own) {
        copy = make_int2(g.last, page[0]);
        atomicSub(p.refs + g.last, 1);
      }
    }
    if (lane == 0) p.lens[b] = len + g.count;
  }
  if (lane == 0) p.pairs[2 * int64_t(b)] = copy.x, p.pairs[2 * int64_t(b) + 1] = copy.y;
}

// Up to kThreads rows: every block has all of them, a thread a row, and what the
// rows need of one another stays in its shared memory.  The blocks meet to rank the
// free pages, and whoever finds one that is needed puts it into its row; they meet
// again only where the new tokens' slots are written here, too.
struct FewRows {
  static constexpr int kSlots = 2 * kThreads;  // of a hash table of shared pages
  int64_t need[kThreads + 1], tokens[kThreads + 1];
  int32_t len[kThreads], last[kThreads], have[kThreads], own[kThreads];
  int32_t page[kSlots], writers[kSlots], lowest[kSlots];
};
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1)
    k_pages_extend_few(const __grid_constant__ PagesParams p) {
  extern __shared__ __align__(16) uint8_t dynamic[];
  FewRows& f = *reinterpret_cast<FewRows*>(dynamic);
  __shared__ Ranks ranks;
  __shared__ int64_t sums[2][kWarps];
  const int rank = blockIdx.x, warp = threadIdx.x >> 5;
  const int32_t b = int32_t(threadIdx.x);
  cluster_arrive();
  for (int i = b; i < FewRows::kSlots; i += kThreads) f.page[i] = -1, f.writers[i] = 0, f.lowest[i] = kThreads;
  grid_wait();
  const int32_t free_here = count_piece(p, piece_of(p.pages, rank, warp), false);
  Growth g = {};
  g.last = -1;
  int32_t owners = 0;
  if (b < p.rows) {
    g = growth_of(p, b);
    f.len[b] = max(p.lens[b], 0), f.last[b] = g.last, f.have[b] = int32_t(min(g.have, p.table_ld));
    if (is_page(p, g.last)) owners = p.refs[g.last];
  }
  __syncthreads();
  // rows that go on in a page that others hold too: how many, and the first
  int at = -1;
  if (owners > 1) {
    at = int((uint32_t(g.last) * 2654435761u) >> 21) & (FewRows::kSlots - 1);
    for (;;) {  // at most half of the slots are taken
      const int32_t was = atomicCAS(&f.page[at], -1, g.last);
      if (was == -1 || was == g.last) break;
      at = (at + 1) & (FewRows::kSlots - 1);
    }
    atomicAdd(&f.writers[at], 1);
    atomicMin(&f.lowest[at], b);
  }
  __syncthreads();
  const bool copy = owners > 1 && !(f.writers[at] == owners && f.lowest[at] == b);
  const int64_t need = g.count > 0 ? g.want - g.have + copy : 0, count = g.count;
  int64_t n = need, c = count;
  scan_rows(n, c, sums);
  f.need[b] = n - need, f.tokens[b] = c - count, f.own[b] = copy;
  const int64_t pages = sums[0][kWarps - 1], tokens = sums[1][kWarps - 1];
  if (b == 0) f.need[kThreads] = pages, f.tokens[kThreads] = tokens;
  if (rank == 0) {  // for k_pages_slots
    if (b < p.rows) p.tokens[b] = c - count;
    if (b == 0) p.tokens[p.rows] = tokens;
  }
  const bool bad = __syncthreads_or((count > 0 && g.want > p.table_ld) || tokens > p.total);
  const bool listed = p.total <= kInline;  // else k_pages_slots finds the pages in the table
  const bool ok = take_free(p, free_here, pages, bad, rank, ranks, [&](int64_t k, int32_t page) {
    const int32_t r = row_of(p.rows, k, [&](int32_t x) { return f.need[x]; });
    const int64_t place = f.have[r] + k - f.need[r] - f.own[r];
    p.refs[page] = 1;
    p.table[r * p.table_ld + place] = page;
    if (listed) p.list[k] = page;
    if (place < f.have[r]) {
      p.pairs[2 * r] = f.last[r], p.pairs[2 * r + 1] = page;
      atomicSub(p.refs + f.last[r], 1);
    }
  });
  if (b < p.rows && b % kCluster == rank) {
    if (ok && g.count > 0) p.lens[b] = f.len[b] + g.count;
    if (!ok || !copy) p.pairs[2 * b] = -1, p.pairs[2 * b + 1] = -1;
  }
  if (!listed) return;
  cluster_sync();
  for (int64_t i = rank * kThreads + b; i < p.total; i += kCluster * kThreads) {
    int64_t slot = -1;
    if (ok && i < tokens) {
      const int32_t r = row_of(p.rows, i, [&](int32_t x) { return f.tokens[x]; });
      const int64_t t = f.len[r] + i - f.tokens[r], place = t >> p.shift, old = f.have[r] - f.own[r];
      const int32_t page = __ldcg(place >= old ? p.list + f.need[r] + place - old : p.table + r * p.table_ld + place);
      slot = (int64_t(page) << p.shift) + (t & ((1 << p.shift) - 1));
    }
    p.slots[i] = slot;
  }
}

// Any number of rows.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1)
    k_pages_extend(const __grid_constant__ PagesParams p) {
  __shared__ Ranks ranks;
  __shared__ int64_t sums[2][kWarps];
  const int rank = blockIdx.x, warp = threadIdx.x >> 5;
  const int32_t thread = rank * kThreads + int32_t(threadIdx.x);
  grid_wait();
  const int32_t free_here = count_piece(p, piece_of(p.pages, rank, warp), false);

  // Rows that go on in a page that others hold too: how many, and the first.
  for (int pass = 0; pass < 2; ++pass) {
    for (int32_t b = thread; b < p.rows; b += kCluster * kThreads) {
      const Growth g = growth_of(p, b);
      if (!is_page(p, g.last) || p.refs[g.last] <= 1) continue;
      if (pass == 0) {
        __stcg(p.writers + g.last, 0);
        __stcg(p.lowest + g.last, p.rows);
      } else {
        atomicAdd(p.writers + g.last, 1);
        atomicMin(p.lowest + g.last, b);
      }
    }
    cluster_sync();
  }

  cluster_arrive();

  // Pages and tokens of the rows before each row; every block for itself.
  int64_t pages = 0, tokens = 0;
  bool bad = false;
  for (int32_t b0 = 0; b0 < p.rows; b0 += kThreads) {
    const int32_t b = b0 + int32_t(threadIdx.x);
    int64_t need = 0, count = 0;
    if (b < p.rows) {
      const Growth g = growth_of(p, b);
      count = g.count;
      if (count > 0) {
        need = g.want - g.have;
        bad = bad || g.want > p.table_ld;
        if (is_page(p, g.last)) {
          const int32_t owners = p.refs[g.last];
          if (owners > 1 && !(__ldcg(p.writers + g.last) == owners && __ldcg(p.lowest + g.last) == b)) ++need;
        }
      }
    }
    int64_t n = need, c = count;
    scan_rows(n, c, sums);
    if (rank == 0 && b < p.rows) p.need[b] = pages + n - need, p.tokens[b] = tokens + c - count;
    pages += sums[0][kWarps - 1], tokens += sums[1][kWarps - 1];
    __syncthreads();
  }
  if (rank == 0 && threadIdx.x == 0) p.need[p.rows] = pages, p.tokens[p.rows] = tokens;
  bad = __syncthreads_or(bad || tokens > p.total);
  const bool ok = take_free(p, free_here, pages, bad, rank, ranks, [&](int64_t k, int32_t page) {
    p.list[k] = page;
    p.refs[page] = 1;
  });
  cluster_sync();
  for (int32_t b = rank * kWarps + warp; b < p.rows; b += kCluster * kWarps) {
    const Growth g = growth_of(p, b);
    const int32_t len = max(p.lens[b], 0);
    __syncwarp();  // all lanes have read the length
    const int64_t first = __ldcg(p.need + b), n = __ldcg(p.need + b + 1) - first;
    grow_row(p, b, g, len, first, n - (g.count > 0 ? g.want - g.have : 0), ok);
  }
}

// The slots of new tokens, once lengths and table have them: a warp takes 256
// neighbours, of which most lie in one row, and looks for that at 32 places at a time.
constexpr int kSlotsEach = 8;  // of a thread
__global__ void __launch_bounds__(kGridThreads) k_pages_slots(const __grid_constant__ PagesParams p) {
  grid_wait();
  const int lane = threadIdx.x & 31;
  const int64_t first = (int64_t(blockIdx.x) * (kGridThreads / 32) + (threadIdx.x >> 5)) * kSlotsEach * 32;
  const bool ok = *p.number == 0;
  const int64_t tokens = ok ? p.tokens[p.rows] : 0;
  int32_t row = 0, hi = p.rows;
  while (hi - row > 1) {
    const int32_t step = (hi - row + 31) / 32, x = row + lane * step;
    const uint32_t below = __ballot_sync(0xFFFFFFFFu, x < hi && p.tokens[min(x, hi)] <= first);
    row += max(__popc(below) - 1, 0) * step;
    hi = min(row + step, hi);
  }
  int64_t end = p.tokens[row + 1], len = p.lens[row];  // the row's last token, its length with them
#pragma unroll
  for (int k = 0; k < kSlotsEach; ++k) {
    const int64_t i = first + k * 32 + lane;
    if (i >= p.total) return;
    int64_t slot = -1;
    if (i < tokens) {
      if (i >= end) {
        row = row_of(p.rows, i, [&](int32_t x) { return p.tokens[x]; });
        end = p.tokens[row + 1], len = p.lens[row];
      }
      const int64_t t = len - (end - i);
      slot = (int64_t(p.table[row * p.table_ld + (t >> p.shift)]) << p.shift) + (t & ((1 << p.shift) - 1));
    }
    p.slots[i] = slot;
  }
}

// Rows that change: what they take, and the pages' counts.  (One row may be the
// source of another and change itself, so the table follows in a second launch.)
__device__ __forceinline__ int32_t* new_lens(const PagesParams& p) { return reinterpret_cast<int32_t*>(p.need); }


constexpr int kRowEach = 4;  // entries of a thread whose loads are under way

__device__ __forceinline__ void take_row(const PagesParams& p, int32_t b, int32_t first, int32_t step) {
  const int32_t src = p.in[b];
  if (src == b) return;
  const bool some = src >= 0 && src < p.rows;
  const int64_t had = held(p, p.lens[b]), has = some ? held(p, p.lens[src]) : 0;
  const int32_t* old = p.table + b * p.table_ld;
  const int32_t* from = p.table + (some ? src : 0) * p.table_ld;
  for (int64_t i0 = first; i0 < max(had, has); i0 += kRowEach * step) {
    int32_t leave[kRowEach], take[kRowEach];
#pragma unroll
    for (int u = 0; u < kRowEach; ++u) {
      const int64_t i = i0 + u * step;
      leave[u] = i < had ? old[i] : -1, take[u] = i < has ? from[i] : -1;
    }
#pragma unroll
    for (int u = 0; u < kRowEach; ++u) {
      const int64_t i = i0 + u * step;
      if (i < has) p.taken[b * p.table_ld + i] = take[u];
      if (leave[u] == take[u]) continue;
      if (is_page(p, leave[u])) atomicSub(p.refs + leave[u], 1);
      if (is_page(p, take[u])) atomicAdd(p.refs + take[u], 1);
    }
  }
  if (first == 0) new_lens(p)[b] = some ? max(p.lens[src], 0) : 0;
}
__device__ __forceinline__ void put_row(const PagesParams& p, int32_t b, int32_t first, int32_t step) {
  if (p.in[b] == b) return;
  const int32_t len = __ldcg(new_lens(p) + b);
  const int64_t has = held(p, len);
  for (int64_t i0 = first; i0 < has; i0 += kRowEach * step) {
    int32_t take[kRowEach];
#pragma unroll
    for (int u = 0; u < kRowEach; ++u)
      if (i0 + u * step < has) take[u] = __ldcg(p.taken + b * p.table_ld + i0 + u * step);
#pragma unroll
    for (int u = 0; u < kRowEach; ++u)
      if (i0 + u * step < has) p.table[b * p.table_ld + i0 + u * step] = take[u];
  }
  if (first == 0) p.lens[b] = len;
}
__global__ void __launch_bounds__(kGridThreads) k_pages_take(const __grid_constant__ PagesParams p) {
  grid_wait();
  take_row(p, blockIdx.x, threadIdx.x, kGridThreads);
}
__global__ void __launch_bounds__(kGridThreads) k_pages_put(const __grid_constant__ PagesParams p) {
  grid_wait();
  put_row(p, blockIdx.x, threadIdx.x, kGridThreads);
}
// Both, of a small table: a warp a row, and a cluster barrier for the launch between.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1)
    k_pages_select(const __grid_constant__ PagesParams p) {
  const int32_t w = int32_t(blockIdx.x) * kWarps + int32_t(threadIdx.x >> 5);
  grid_wait();
  for (int32_t b = w; b < p.rows; b += kCluster * kWarps) take_row(p, b, threadIdx.x & 31, 32);
  cluster_sync();
  for (int32_t b = w; b < p.rows; b += kCluster * kWarps) put_row(p, b, threadIdx.x & 31, 32);
}

// Held pages in order, and the free ids below their number, which those from
// there on go to.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1)
    k_pages_compact(const __grid_constant__ PagesParams p) {
  __shared__ Ranks ranks;
  const int rank = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t thread = rank * kThreads + int32_t(threadIdx.x);
  cluster_arrive();
  grid_wait();
  const Piece mine = piece_of(p.pages, rank, warp);
  int64_t used, at = rank_pieces(count_piece(p, mine, true), rank, ranks, used);
  if (thread == 0) {
    *p.number = int32_t(used);
    if (used == p.pages) *p.part = used;
  }
#pragma unroll 4
  for (int64_t i0 = mine.lo; i0 < mine.hi; i0 += 32) {
    const int64_t i = i0 + lane;
    const bool some = i < mine.hi && p.refs[i] > 0;
    const uint32_t all = __ballot_sync(0xFFFFFFFFu, some);
    const int64_t k = at + __popc(all & ((1u << lane) - 1));  // held pages below i
    if (some) p.list[k] = int32_t(i);
    else if (i < min(mine.hi, used)) p.writers[i - k] = int32_t(i);
    if (i < mine.hi && i == used) *p.part = k;
    at += __popc(all);
  }
  cluster_sync();
  const int64_t stay = __ldcg(p.part), moves = used - stay;
  for (int64_t j = thread; j < p.pages / 2; j += kCluster * kThreads) {
    int2 pair = make_int2(-1, -1);
    if (j < moves) {
      pair = make_int2(__ldcg(p.list + stay + j), __ldcg(p.writers + j));
      p.refs[pair.y] = p.refs[pair.x];
      p.refs[pair.x] = 0;
      p.lowest[pair.x] = pair.y;
    }
    p.pairs[2 * j] = pair.x, p.pairs[2 * j + 1] = pair.y;
  }
}
__global__ void __launch_bounds__(kGridThreads) k_pages_renumber(const __grid_constant__ PagesParams p) {
  grid_wait();
  const int32_t used = *p.number, b = blockIdx.x;
  int32_t* row = p.table + b * p.table_ld;
  for (int64_t i = threadIdx.x; i < held(p, p.lens[b]); i += kGridThreads) {
    const int32_t page = row[i];
    if (page >= used && page < p.pages) row[i] = p.lowest[page];
  }
}

// ------------------------------------------------------------------ copies --

// A page's four buffers in a row, in chunks of 16 bytes; a block copies kUnit of
// them at a time, four a thread.
constexpr int kUnitEach = 4;
constexpr int kUnit = kUnitEach * kGridThreads;

struct CopyParams {
  const uint4* src[4];
  uint4* dst[4];
  int32_t chunks[4];  // of a page's buffer
  int32_t units;      // of a page
  int64_t src_pages, dst_pages, count;
  const int32_t* pairs;
};

// Lists of pairs are mostly empty behind their first entries, or here and there:
// a warp looks up its block's next 32 units at once and passes over the empty ones.
__global__ void __launch_bounds__(kGridThreads) k_cache_copy(const __grid_constant__ CopyParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t all = p.count * p.units;
  grid_wait();
  for (int64_t u0 = blockIdx.x; u0 < all; u0 += int64_t(gridDim.x) * 32) {
    const int64_t u = u0 + int64_t(gridDim.x) * lane, pair = u / p.units;
    int32_t from = -1, to = -1;
    if (u < all) from = p.pairs[2 * pair], to = p.pairs[2 * pair + 1];
    uint32_t live =
        __ballot_sync(0xFFFFFFFFu, from >= 0 && from < p.src_pages && to >= 0 && to < p.dst_pages);
    const int32_t part = int32_t(u - pair * p.units);
    while (live != 0) {
      const int k = __ffs(live) - 1;
      live &= live - 1;
      const int64_t from_k = __shfl_sync(0xFFFFFFFFu, from, k), to_k = __shfl_sync(0xFFFFFFFFu, to, k);
      const int32_t first = __shfl_sync(0xFFFFFFFFu, part, k) * kUnit + int32_t(threadIdx.x);
      uint4 v[kUnitEach];
      uint4* dst[kUnitEach];
#pragma unroll
      for (int i = 0; i < kUnitEach; ++i) {
        int32_t c = first + i * kGridThreads, t = 0;
        dst[i] = nullptr;
#pragma unroll
        for (int x = 0; x < 3; ++x)
          if (t == x && c >= p.chunks[x]) c -= p.chunks[x], t = x + 1;
        if (c >= p.chunks[t]) continue;
        v[i] = __ldcs(p.src[t] + from_k * p.chunks[t] + c);
        dst[i] = p.dst[t] + to_k * p.chunks[t] + c;
      }
#pragma unroll
      for (int i = 0; i < kUnitEach; ++i)
        if (dst[i] != nullptr) *dst[i] = v[i];
    }
  }
}

// ------------------------------------------------------------------ checks --

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }

nvfp4_status check_pages(const mxfp4_pages* g, const void* workspace, int64_t workspace_bytes, const std::string& nm,
                         PagesParams& p) {
  if (!g || !g->refs || !g->table || !g->lens || !workspace) return fail(NVFP4_EINVAL, nm + ": null pointer");
  if (g->pages < 1 || g->rows < 1 || g->table_ld < 1 || g->page_size < 1)
    return fail(NVFP4_EINVAL, nm + ": pages, rows, table_ld and page_size must be positive");
  int sh = 0;
  while ((1 << sh) < g->page_size) ++sh;
  if ((1 << sh) != g->page_size || g->page_size < 16 || g->page_size > 256)
    return fail(NVFP4_EUNSUPPORTED, nm + ": page_size must be 16, 32, 64, 128 or 256");
  if (g->pages > (int64_t(1) << 30) || g->rows > (1 << 20) ||
      g->table_ld > ((int64_t(1) << 31) - (int64_t(1) << 25)) / g->page_size ||
      g->table_ld > (int64_t(1) << 31) / g->rows)
    return fail(NVFP4_EUNSUPPORTED, nm + ": too many pages, rows or table entries");
  if (!aligned16(workspace) || reinterpret_cast<uintptr_t>(g->refs) % 4 != 0 ||
      reinterpret_cast<uintptr_t>(g->table) % 4 != 0 || reinterpret_cast<uintptr_t>(g->lens) % 4 != 0)
    return fail(NVFP4_EALIGN, nm + ": workspace must be 16-byte aligned, the others aligned to their elements");
  const int64_t need = mxfp4_pages_workspace_bytes(g);
  if (workspace_bytes < need)
    return fail(NVFP4_EINVAL, nm + ": workspace too small, " + std::to_string(need) + " bytes are needed");
  p = {};
  p.refs = g->refs, p.table = g->table, p.lens = g->lens;
  p.pages = g->pages, p.table_ld = g->table_ld, p.rows = g->rows, p.shift = sh;
  uint8_t* ws = static_cast<uint8_t*>(const_cast<void*>(workspace));
  auto take = [&](int64_t bytes) {
    uint8_t* at = ws;
    ws += align256(bytes);
    return at;
  };
  p.need = reinterpret_cast<int64_t*>(take((int64_t(g->rows) + 1) * 8));
  p.tokens = reinterpret_cast<int64_t*>(take((int64_t(g->rows) + 1) * 8));
  p.part = reinterpret_cast<int64_t*>(take(8));
  p.taken = p.list = reinterpret_cast<int32_t*>(ws);
  p.writers = p.list + g->pages;
  p.lowest = p.writers + g->pages;
  return NVFP4_OK;
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" int64_t mxfp4_pages_workspace_bytes(const mxfp4_pages* g) {
  if (!g || g->pages < 1 || g->rows < 1 || g->table_ld < 1) return 0;
  return 2 * align256((int64_t(g->rows) + 1) * 8) + align256(8) +
         align256(4 * std::max(3 * g->pages, g->rows * g->table_ld));
}

extern "C" nvfp4_status mxfp4_pages_select(const mxfp4_pages* pages, const int32_t* sources, void* workspace,
                                           int64_t workspace_bytes, nvfp4_stream_t stream) {
  const std::string nm("mxfp4_pages_select");
  PagesParams p;
  nvfp4_status st = check_pages(pages, workspace, workspace_bytes, nm, p);
  if (st != NVFP4_OK) return st;
  if (!sources) return fail(NVFP4_EINVAL, nm + ": null pointer");
  if (reinterpret_cast<uintptr_t>(sources) % 4 != 0)
    return fail(NVFP4_EALIGN, nm + ": sources must be aligned to its elements");
  p.in = sources;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (p.rows * p.table_ld <= kSmallTable)
    return launch("launch k_pages_select", k_pages_select, dim3(kCluster), dim3(kThreads), 0, 0, s, p);
  st = launch("launch k_pages_take", k_pages_take, dim3(unsigned(p.rows)), dim3(kGridThreads), 0, 0, s, p);
  if (st != NVFP4_OK) return st;
  return launch("launch k_pages_put", k_pages_put, dim3(unsigned(p.rows)), dim3(kGridThreads), 0, 0, s, p);
}

extern "C" nvfp4_status mxfp4_pages_extend(const mxfp4_pages* pages, const int32_t* counts, int64_t total,
                                           int64_t* slots, int32_t* copies, int32_t* missing, void* workspace,
                                           int64_t workspace_bytes, nvfp4_stream_t stream) {
  const std::string nm("mxfp4_pages_extend");
  PagesParams p;
  nvfp4_status st = check_pages(pages, workspace, workspace_bytes, nm, p);
  if (st != NVFP4_OK) return st;
  if (total < 0) return fail(NVFP4_EINVAL, nm + ": total must not be negative");
  if (total > 0x7FFFFFFF) return fail(NVFP4_EUNSUPPORTED, nm + ": too many tokens");
  if (!counts || (total > 0 && !slots) || !copies || !missing) return fail(NVFP4_EINVAL, nm + ": null pointer");
  if (reinterpret_cast<uintptr_t>(counts) % 4 != 0 || reinterpret_cast<uintptr_t>(slots) % 8 != 0 ||
      reinterpret_cast<uintptr_t>(copies) % 4 != 0 || reinterpret_cast<uintptr_t>(missing) % 4 != 0)
    return fail(NVFP4_EALIGN, nm + ": counts, slots, copies and missing must be aligned to their elements");
  p.in = counts, p.total = total, p.slots = slots, p.pairs = copies, p.number = missing;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (p.rows <= kThreads) {
    static std::atomic<uint64_t> ready{0};
    st = allow_smem(reinterpret_cast<const void*>(k_pages_extend_few), int(sizeof(FewRows)), ready);
    if (st == NVFP4_OK)
      st = launch("launch k_pages_extend_few", k_pages_extend_few, dim3(kCluster), dim3(kThreads), sizeof(FewRows), 0, s, p);
    if (total <= kInline) return st;
  } else {
    st = launch("launch k_pages_extend", k_pages_extend, dim3(kCluster), dim3(kThreads), 0, 0, s, p);
  }
  if (st != NVFP4_OK || total == 0) return st;
  const int64_t each = kGridThreads * kSlotsEach, blocks = (total + each - 1) / each;
  return launch("launch k_pages_slots", k_pages_slots, dim3(unsigned(blocks)), dim3(kGridThreads), 0, 0, s, p);
}

extern "C" nvfp4_status mxfp4_pages_compact(const mxfp4_pages* pages, int32_t* moves, int32_t* used, void* workspace,
                                            int64_t workspace_bytes, nvfp4_stream_t stream) {
  const std::string nm("mxfp4_pages_compact");
  PagesParams p;
  nvfp4_status st = check_pages(pages, workspace, workspace_bytes, nm, p);
  if (st != NVFP4_OK) return st;
  if ((pages->pages > 1 && !moves) || !used) return fail(NVFP4_EINVAL, nm + ": null pointer");
  if (reinterpret_cast<uintptr_t>(moves) % 4 != 0 || reinterpret_cast<uintptr_t>(used) % 4 != 0)
    return fail(NVFP4_EALIGN, nm + ": moves and used must be aligned to their elements");
  p.pairs = moves, p.number = used;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  st = launch("launch k_pages_compact", k_pages_compact, dim3(kCluster), dim3(kThreads), 0, 0, s, p);
  if (st != NVFP4_OK) return st;
  return launch("launch k_pages_renumber", k_pages_renumber, dim3(unsigned(p.rows)), dim3(kGridThreads), 0, 0, s, p);
}

extern "C" nvfp4_status mxfp4_cache_copy(const mxfp4_cache* cache, const mxfp4_cache* source, const int32_t* pairs,
                                         int64_t count, nvfp4_stream_t stream) {
  const std::string nm("mxfp4_cache_copy");
  int sh = 0, src_sh = 0;
  nvfp4_status st = check_cache(cache, &sh, nm);
  if (st == NVFP4_OK) st = check_cache(source, &src_sh, nm);
  if (st != NVFP4_OK) return st;
  if (sh != src_sh || cache->kv_heads != source->kv_heads || cache->dim != source->dim)
    return fail(NVFP4_EINVAL, nm + ": both caches must have one page_size, kv_heads and dim");
  if (count < 0) return fail(NVFP4_EINVAL, nm + ": count must not be negative");
  if (count == 0) return NVFP4_OK;
  if (!pairs) return fail(NVFP4_EINVAL, nm + ": null pointer");
  if (count > 0x7FFFFFFF) return fail(NVFP4_EUNSUPPORTED, nm + ": too many pairs");
  if (reinterpret_cast<uintptr_t>(pairs) % 4 != 0)
    return fail(NVFP4_EALIGN, nm + ": pairs must be aligned to its elements");
  CopyParams p = {};
  const void* src[4] = {source->k_codes, source->v_codes, source->k_scales, source->v_scales};
  void* dst[4] = {cache->k_codes, cache->v_codes, cache->k_scales, cache->v_scales};
  int32_t chunks = 0;
  for (int i = 0; i < 4; ++i) {
    p.src[i] = static_cast<const uint4*>(src[i]), p.dst[i] = static_cast<uint4*>(dst[i]);
    p.chunks[i] = int32_t(int64_t(cache->kv_heads) * cache->page_size * (cache->dim / (i < 2 ? 2 : 32)) / 16);
    chunks += p.chunks[i];
  }
  p.units = (chunks + kUnit - 1) / kUnit;
  p.src_pages = source->pages, p.dst_pages = cache->pages, p.count = count, p.pairs = pairs;
  const int64_t most = int64_t(sm_count()) * 8;
  return launch("launch k_cache_copy", k_cache_copy, dim3(unsigned(std::min(count * p.units, most))), dim3(kGridThreads),
                0, 0, reinterpret_cast<cudaStream_t>(stream), p);
}
