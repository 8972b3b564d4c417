// Page operations of a paged entry cache: reserve, fork, free, compact.
//
// The free list is the refcounts themselves: a page with refcount <= 0 is free,
// and new pages are the free ones of the lowest ids, so the outcome does not
// depend on scheduling.  Everything lives on the device and nothing is read
// back.  A metadata kernel (one CTA, whose scans order the free pages) checks the lists
// first and changes nothing if any check fails; it leaves a list of page copies in
// the workspace for the kernel behind it, which makes them and brings the
// tables up to date, a CTA a page or row.
//
// The copies are bound by HBM (each page read and written once); the metadata
// by the latency of the scans over N refcounts and of the launches (N = 4096: reserving
// for 64 rows 5 us; freeing, forking and reserving 64 rows 16.6 us in four launches, 20.4
// with a fork's ids and counts written by the one CTA; compacting 2048 pages in use 14.0
// us, 15.0 with the tables in a launch of their own).
#include <climits>

#include "common.cuh"

namespace csa {

constexpr int kMetaThreads = 1024;
constexpr int kMaxPages = 1 << 20;   // page counts of 1024 list items add up within 31 bits

// Exclusive prefix sum over the CTA; *total gets the sum.  Two syncs.
__device__ __forceinline__ int block_excl_scan(int v, int* total, int* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int incl = warp_incl_scan(v);
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const int w = warp_sums[lane];
    const int wi = warp_incl_scan(w);
    warp_sums[lane] = wi - w;
    if (lane == 31) warp_sums[32] = wi;
  }
  __syncthreads();
  *total = warp_sums[32];
  return warp_sums[warp] + incl - v;
}

// list[k] = the k-th free page, for k < need (ascending ids); returns how many
// were found.  All threads call it.
__device__ int find_free(const int32_t* refcount, int N, int need, int32_t* list, int* warp_sums) {
  int found = 0;
  for (int base = 0; base < N && found < need; base += kMetaThreads) {
    const int id = base + threadIdx.x;
    const int fr = id < N && refcount[id] <= 0;
    int total;
    const int k = found + block_excl_scan(fr, &total, warp_sums);
    if (fr && k < need) list[k] = id;
    found += total;
    __syncthreads();
  }
  return found;
}

// A row of the list is taken by this call: held -> -1 - held.  False if it is
// taken already (the row is listed twice).
__device__ __forceinline__ bool claim(int32_t* held, int h) { return h >= 0 && atomicCAS(held, h, -1 - h) == h; }

struct MetaArgs {
  const int32_t* src;        // fork
  const int32_t* dst;        // fork's new rows, reserve's rows
  const int32_t* n_entries;
  int n, P, R, max_pages, N;
  int32_t* table;
  int32_t* held;
  int32_t* refcount;
  int32_t* copies;           // workspace [1 + 3 n]: fork's copies: count, then (from, to, rows)
  int32_t* off;              // workspace [n]: first new page of list item i, or -1 while unclaimed
  int32_t* cnt;              // workspace [n]: its number of new pages
  int32_t* list;             // workspace [N]: free pages
  int* status;
};

// Reserve and fork: check and claim every item, count the new pages, find them,
// then write tables and refcounts (of a fork only the new pages', and the copy list).
template <bool kFork>
__global__ void __launch_bounds__(kMetaThreads) grow_kernel(const MetaArgs a) {
  __shared__ int warp_sums[33];
  __shared__ int bad, few;
  const int tid = threadIdx.x;
  if (tid == 0) bad = few = 0;
  __syncthreads();
  int need = 0;
  for (int base = 0; base < a.n; base += kMetaThreads) {
    const int i = base + tid;
    int c = 0;
    if (i < a.n) {
      const int r = a.dst[i], ne = a.n_entries[i];
      const long long pages = ne < 0 ? -1 : (static_cast<long long>(ne) + a.P - 1) / a.P;
      bool ok = r >= 0 && r < a.R && pages >= 0 && pages <= a.max_pages;
      if (kFork && ok) {
        const int s = a.src[i];
        // (a row that this call claims reads as negative: it holds nothing)
        ok = s >= 0 && s < a.R && pages <= max(__ldcg(a.held + s), 0);
      }
      bool mine = false;
      if (ok) {
        const int h = __ldcg(a.held + r);
        ok = (!kFork || h == 0) && claim(a.held + r, h);
        mine = ok;
        if (ok) c = kFork ? (ne % a.P != 0) : max(0, static_cast<int>(pages) - h);
        if (c > a.N) { c = 0; few = 1; }
      }
      a.cnt[i] = mine ? c : -1;
      if (!ok) bad = 1;
    }
    int total;
    const int ex = block_excl_scan(c, &total, warp_sums);
    if (i < a.n) a.off[i] = need + ex;
    need = need > INT_MAX - total ? INT_MAX : need + total;
    __syncthreads();
  }
  int why = bad ? (CSA_ERR_INVALID_ARG | ((kFork ? 2 : 1) << 8)) : 0;
  if (!why && (few || need > 0) && (few || need > a.N || find_free(a.refcount, a.N, need, a.list, warp_sums) < need))
    why = CSA_ERR_NO_SPACE | ((kFork ? 2 : 1) << 8);
  __syncthreads();
  if (why) {
    // give the claimed rows back; nothing else has changed
    for (int i = tid; i < a.n; i += kMetaThreads)
      if (a.cnt[i] >= 0) { const int r = a.dst[i]; a.held[r] = -1 - a.held[r]; }
    if (kFork && tid == 0) a.copies[0] = 0;
    if (tid == 0) atomicCAS(a.status, 0, why);
    return;
  }
  if (kFork && tid == 0) a.copies[0] = a.n;
  if (kFork) {
    for (int i = tid; i < a.n; i += kMetaThreads) {
      const int ne = a.n_entries[i], whole = ne / a.P, tail = ne % a.P;
      int32_t* cp = a.copies + 1 + 3 * static_cast<size_t>(i);
      cp[0] = -1;
      if (tail) {
        const int id = a.list[a.off[i]];
        const int old = a.table[static_cast<size_t>(a.src[i]) * a.max_pages + whole];
        a.table[static_cast<size_t>(a.dst[i]) * a.max_pages + whole] = id;
        a.refcount[id] = 1;
        if (old >= 0 && old < a.N) { cp[0] = old; cp[1] = id; cp[2] = tail; }
      }
    }
    return;
  }
  const int lane = tid & 31;
  for (int i = tid >> 5; i < a.n; i += kMetaThreads / 32) {
    const int r = a.dst[i];
    int32_t* row = a.table + static_cast<size_t>(r) * a.max_pages;
    const int h = -1 - a.held[r], c = a.cnt[i];
    __syncwarp();
    for (int k = lane; k < c; k += 32) {
      const int id = a.list[a.off[i] + k];
      row[h + k] = id;
      a.refcount[id] = 1;
    }
    if (lane == 0) a.held[r] = h + c;
  }
}

struct PoolArgs {
  uint8_t* pool;
  long long page_bytes, layer_bytes;
  int entry_bytes;           // fork
  int L;
};
// The first `bytes` of page `from` to page `to` in one layer, by the CTAs of a grid row.
__device__ __forceinline__ void copy_page(const PoolArgs& p, int layer, int from, int to, long long bytes) {
  const uint4* s = reinterpret_cast<const uint4*>(p.pool + layer * p.layer_bytes + from * p.page_bytes);
  uint4* d = reinterpret_cast<uint4*>(p.pool + layer * p.layer_bytes + to * p.page_bytes);
  for (long long k = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; k < bytes / 16;
       k += static_cast<long long>(gridDim.x) * blockDim.x)
    d[k] = s[k];
}

// Fork, step 2: the shared pages' ids and refcounts, and the copies of partial last pages.
// CTA = (chunk of the page, fork, layer).
__global__ void __launch_bounds__(256) fork_apply_kernel(const MetaArgs a, const PoolArgs p) {
  const int n = a.copies[0];           // 0: the call was refused
  for (int i = blockIdx.y; i < n; i += gridDim.y) {
    if (blockIdx.x == 0 && blockIdx.z == 0) {
      const int r = a.dst[i], ne = a.n_entries[i], whole = ne / a.P;
      const int32_t* from = a.table + static_cast<size_t>(a.src[i]) * a.max_pages;
      int32_t* row = a.table + static_cast<size_t>(r) * a.max_pages;
      for (int k = threadIdx.x; k < whole; k += blockDim.x) {
        const int id = from[k];
        row[k] = id;
        if (id >= 0 && id < a.N) atomicAdd(a.refcount + id, 1);
      }
      if (threadIdx.x == 0) a.held[r] = whole + (ne % a.P ? 1 : 0);
    }
    const int32_t* cp = a.copies + 1 + 3 * static_cast<size_t>(i);
    if (cp[0] >= 0) copy_page(p, blockIdx.z, cp[0], cp[1], static_cast<long long>(cp[2]) * p.entry_bytes);
  }
}

// One warp per listed row.  The exchange on held makes a row listed twice free once.
__global__ void __launch_bounds__(256) free_kernel(const int32_t* __restrict__ rows, int n, int32_t* table,
                                                   int32_t* held, int R, int max_pages, int32_t* refcount, int N,
                                                   int* status) {
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (i >= n) return;
  const int r = rows[i];
  if (r < 0 || r >= R) {
    if (lane == 0) atomicCAS(status, 0, CSA_ERR_INVALID_ARG | (3 << 8));
    return;
  }
  int h = 0;
  if (lane == 0) h = atomicExch(held + r, 0);
  h = min(__shfl_sync(0xffffffffu, h, 0), max_pages);
  int32_t* row = table + static_cast<size_t>(r) * max_pages;
  for (int k = lane; k < h; k += 32) {
    const int id = row[k];
    row[k] = -1;
    if (id >= 0 && id < N) atomicSub(refcount + id, 1);
  }
}

// Compaction, step 1: n_live, the pages that move, where to, and the new
// refcounts.  moves = (from, to) pairs behind their count; map[id] = new id.
__global__ void __launch_bounds__(kMetaThreads) compact_meta_kernel(const int32_t* refcount, int N,
                                                                    int32_t* refcount_out, int32_t* n_live_out,
                                                                    int32_t* count, int32_t* moves, int32_t* map) {
  __shared__ int warp_sums[33];
  const int tid = threadIdx.x;
  int mine = 0, n_live;
  for (int id = tid; id < N; id += kMetaThreads) mine += refcount[id] > 0;
  block_excl_scan(mine, &n_live, warp_sums);
  __syncthreads();
  int nm = 0, nh = 0;
  for (int base = 0; base < N; base += kMetaThreads) {
    const int id = base + tid;
    const int rc = id < N ? refcount[id] : 0;
    const int mv = id < N && rc > 0 && id >= n_live, ho = id < N && rc <= 0 && id < n_live;
    int total;
    // movers and holes never lie on both sides of n_live: one scan counts both
    const int ex = block_excl_scan(mv | (ho << 16), &total, warp_sums);
    if (mv) moves[2 * (nm + (ex & 0xffff))] = id;
    if (ho) moves[2 * (nh + (ex >> 16)) + 1] = id;
    nm += total & 0xffff;
    nh += total >> 16;
    if (id < N) {
      map[id] = id;
      if (refcount_out != refcount) refcount_out[id] = rc;
    }
    __syncthreads();
  }
  for (int k = tid; k < nm; k += kMetaThreads) {
    const int from = moves[2 * k], to = moves[2 * k + 1];
    map[from] = to;
    refcount_out[to] = refcount[from];
    refcount_out[from] = 0;
  }
  if (tid == 0) { *count = nm; *n_live_out = n_live; }
}

// Compaction, step 2: the pages that move, CTA = (chunk of the page, move, layer); and, in
// the grid's last layer, the tables in the new numbering.
__global__ void __launch_bounds__(256) compact_apply_kernel(const int32_t* __restrict__ count,
                                                            const int32_t* __restrict__ moves, const PoolArgs p,
                                                            const int32_t* table, const int32_t* __restrict__ held,
                                                            int max_pages, long long total, int N,
                                                            const int32_t* __restrict__ map, int32_t* table_out) {
  if (blockIdx.z < p.L) {
    for (int i = blockIdx.y; i < *count; i += gridDim.y)
      copy_page(p, blockIdx.z, moves[2 * static_cast<size_t>(i)], moves[2 * static_cast<size_t>(i) + 1], p.page_bytes);
    return;
  }
  const long long cta = static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x;
  for (long long i = cta * blockDim.x + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * gridDim.y * blockDim.x) {
    const int id = table[i];
    const bool use = i % max_pages < held[i / max_pages];
    table_out[i] = use && id >= 0 && id < N ? map[id] : id;
  }
}

namespace {
int check_pool(const void* pool, int L, int64_t page_bytes) {
  CSA_REQUIRE(pool && L >= 1 && page_bytes > 0, CSA_ERR_INVALID_ARG);
  CSA_REQUIRE(aligned16(pool), CSA_ERR_ALIGNMENT);
  return CSA_OK;
}
int check_cache(const void* table, const void* held, const void* refcount, int R, int max_pages, int N) {
  CSA_REQUIRE(table && held && refcount, CSA_ERR_INVALID_ARG);
  CSA_REQUIRE(R >= 0 && max_pages >= 1 && N >= 0, CSA_ERR_INVALID_ARG);
  CSA_REQUIRE(N <= kMaxPages, CSA_ERR_UNSUPPORTED);
  return CSA_OK;
}
// Grid of the copies of up to n pages in `layers` layers.
dim3 copy_grid(int64_t page_bytes, int n, int layers) {
  return dim3(static_cast<unsigned>((page_bytes + 256 * 16 * 4 - 1) / (256 * 16 * 4)), n < 16384 ? n : 16384, layers);
}
}  // namespace

}  // namespace csa

using namespace csa;

extern "C" size_t kv_pages_workspace_size(int N, int n) {
  if (N < 0 || n < 0) return 0;
  // grow: copies [1 + 3 n], off, cnt [n], list [N]; compact: count, moves [2 N], map [N]
  return 4 * (3 * static_cast<size_t>(N) + 5 * static_cast<size_t>(n) + 4);
}

static int grow(bool fork, const int32_t* src, const int32_t* dst, const int32_t* n_entries, int n, int P,
                int32_t* table, int32_t* held, int R, int max_pages, int32_t* refcount, int N, void* pool, int L,
                int64_t page_bytes, void* workspace, size_t ws_bytes, int32_t* status, csa_stream_t stream) {
  int st = check_cache(table, held, refcount, R, max_pages, N);
  if (st != CSA_OK) return st;
  CSA_REQUIRE(n >= 0 && P >= 1, CSA_ERR_INVALID_ARG);
  if (n == 0) return CSA_OK;
  CSA_REQUIRE(dst && n_entries && workspace && ws_bytes >= kv_pages_workspace_size(N, n), CSA_ERR_INVALID_ARG);
  CSA_REQUIRE((reinterpret_cast<uintptr_t>(workspace) & 3) == 0, CSA_ERR_ALIGNMENT);
  MetaArgs a;
  a.src = src; a.dst = dst; a.n_entries = n_entries; a.n = n; a.P = P; a.R = R; a.max_pages = max_pages; a.N = N;
  a.table = table; a.held = held; a.refcount = refcount;
  a.copies = static_cast<int32_t*>(workspace);      // (first: callers may read the count)
  a.off = a.copies + 1 + 3 * static_cast<size_t>(n);
  a.cnt = a.off + n;
  a.list = a.cnt + n;
  a.status = status_word(status);
  CSA_REQUIRE(a.status != nullptr, CSA_ERR_CUDA);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!fork) {
    grow_kernel<false><<<1, kMetaThreads, 0, s>>>(a);
    return check_launch();
  }
  grow_kernel<true><<<1, kMetaThreads, 0, s>>>(a);
  st = check_launch();
  if (st != CSA_OK) return st;
  const PoolArgs p{static_cast<uint8_t*>(pool), page_bytes, page_bytes * N, static_cast<int>(page_bytes / P), L};
  fork_apply_kernel<<<copy_grid(page_bytes, n, L), 256, 0, s>>>(a, p);
  return check_launch();
}

extern "C" int kv_pages_reserve(const int32_t* rows, const int32_t* n_entries, int n, int P, int32_t* table,
                                int32_t* held, int R, int max_pages, int32_t* refcount, int N, void* workspace,
                                size_t ws_bytes, int32_t* status, csa_stream_t stream) {
  return grow(false, nullptr, rows, n_entries, n, P, table, held, R, max_pages, refcount, N, nullptr, 0, 0, workspace,
              ws_bytes, status, stream);
}

extern "C" int kv_pages_fork(const int32_t* src, const int32_t* dst, const int32_t* n_entries, int n, int P,
                             int32_t* table, int32_t* held, int R, int max_pages, int32_t* refcount, int N,
                             void* pool, int L, int64_t page_bytes, void* workspace, size_t ws_bytes,
                             int32_t* status, csa_stream_t stream) {
  const int st = check_pool(pool, L, page_bytes);
  if (st != CSA_OK) return st;
  CSA_REQUIRE(P >= 1 && (n == 0 || src), CSA_ERR_INVALID_ARG);
  CSA_REQUIRE(page_bytes % P == 0 && page_bytes / P % 16 == 0 && page_bytes / P < (1ll << 31), CSA_ERR_UNSUPPORTED);
  CSA_REQUIRE(L <= 65535, CSA_ERR_UNSUPPORTED);
  return grow(true, src, dst, n_entries, n, P, table, held, R, max_pages, refcount, N, pool, L, page_bytes, workspace,
              ws_bytes, status, stream);
}

extern "C" int kv_pages_free(const int32_t* rows, int n, int32_t* table, int32_t* held, int R, int max_pages,
                             int32_t* refcount, int N, int32_t* status, csa_stream_t stream) {
  int st = check_cache(table, held, refcount, R, max_pages, N);
  if (st != CSA_OK) return st;
  CSA_REQUIRE(n >= 0, CSA_ERR_INVALID_ARG);
  if (n == 0) return CSA_OK;
  CSA_REQUIRE(rows != nullptr, CSA_ERR_INVALID_ARG);
  int* sw = status_word(status);
  CSA_REQUIRE(sw != nullptr, CSA_ERR_CUDA);
  free_kernel<<<(n + 7) / 8, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(rows, n, table, held, R, max_pages,
                                                                             refcount, N, sw);
  return check_launch();
}

extern "C" int kv_pages_compact(const int32_t* table, const int32_t* held, int R, int max_pages,
                                const int32_t* refcount, int N, void* pool, int L, int64_t page_bytes,
                                int32_t* table_out, int32_t* refcount_out, int32_t* n_live, void* workspace,
                                size_t ws_bytes, csa_stream_t stream) {
  int st = check_cache(table, held, refcount, R, max_pages, N);
  if (st == CSA_OK) st = check_pool(pool, L, page_bytes);
  if (st != CSA_OK) return st;
  CSA_REQUIRE(table_out && refcount_out && n_live && workspace, CSA_ERR_INVALID_ARG);
  CSA_REQUIRE(ws_bytes >= kv_pages_workspace_size(N, 0), CSA_ERR_INVALID_ARG);
  CSA_REQUIRE(page_bytes % 16 == 0 && page_bytes < (1ll << 31) && L < 65535, CSA_ERR_UNSUPPORTED);
  CSA_REQUIRE((reinterpret_cast<uintptr_t>(workspace) & 3) == 0, CSA_ERR_ALIGNMENT);
  int32_t* count = static_cast<int32_t*>(workspace);
  int32_t* moves = count + 2;
  int32_t* map = moves + 2 * static_cast<size_t>(N);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  compact_meta_kernel<<<1, kMetaThreads, 0, s>>>(refcount, N, refcount_out, n_live, count, moves, map);
  st = check_launch();
  if (st != CSA_OK) return st;
  const PoolArgs p{static_cast<uint8_t*>(pool), page_bytes, page_bytes * N, 0, L};
  // (at most N / 2 pages move)
  compact_apply_kernel<<<copy_grid(page_bytes, N < 2 ? 1 : N / 2, L + 1), 256, 0, s>>>(
      count, moves, p, table, held, max_pages, static_cast<long long>(R) * max_pages, N, map, table_out);
  return check_launch();
}
