// hca_prefix_attn_fwd in bf16 on tcgen05: attention of a batch over paged entries
// that groups of sequences share, the raw window and the sink.
//
//   l_j = tau <q, k_j>;  out = sum_j e^{l_j} k_j / (e^sigma + sum_j e^{l_j})
//
// A job is up to 128 query rows, whole (sequence, token) pairs of H heads of one
// group, as the M side of the MMAs; thread = row in the softmax:
//   S [128 rows x 128 keys] = Q K^T   (Q and the key tile in shared memory)
//   O [128 rows x 128 dims] += P K    (P in tensor memory beside S; the same tile
//                                      read with its dims as N)
// Key tiles come in three kinds:
//   shared  128 entries that every row of the job sees, loaded once for all;
//   own     128 entries of one sequence (its pairs that see equally many share a tile);
//   runs    8 runs of 16 keys, each of one pair: entries behind its last whole tile,
//           then raw tokens of its window.
// Own tiles and runs concern some rows only.  The PV MMA of such a tile writes
// those rows' lanes alone (its lane mask; a lone pair, whose lane 0 .. H - 1 count, needs
// none: a masked MMA took 150 cycles more), so a row's sum holds its own keys
// and nothing else: an infinity or NaN in one sequence's keys cannot reach
// another's row as 0 * inf.  Keys a row must not see inside its own tiles are
// zero-filled in shared memory and get P = 0.
//
// Split.  A cluster of c CTAs shares each job: whole entry tile i goes to rank i % c, the
// 16-key runs behind the last whole tile and those of the window in turn to all
// ranks (a last tile as a whole would fall to one rank for all of a job's sequences).
// The ranks' (O, M, l) meet in distributed shared memory, in rank order, each rank
// finishing 128 / c rows.  c depends on the cache's capacity and H alone, tiles
// sit at multiples of 128 entries, and a row's stabiliser is its own: its bits do
// not depend on batch or grouping.
//
// Softmax.  A row's stabiliser M is the maximum of its first tile in the rank, and
// stays: weights 2^(l - M) and their sums keep fp32's (and, in P, bf16's) relative
// precision at any scale, so M only has to keep them in range.  A row in which
// a later weight passes 2^100 is flagged and computed again, exactly, on CUDA
// cores with a running maximum; a weight below 2^-126 of the first tile's
// largest is lost against it anyway.  (Such a row costs 0.5 us a key, a warp's rows
// one after the other: with one of 16 rows over 1024 entries 0.56 ms for 15 us, over
// 8192 4.1 ms for 20 us, all 16 of them 8.6 ms.  Logits that differ by 69 within a
// row; with normalised q and k they are bounded by tau D times the norms' weights.)  So once M is there a tile needs no maximum and no
// word from the tiles before (a running one took a third of a tile's time).
// P is rounded to bf16 for the MMA (a half step of 2^-8 a weight, of the size
// of the output's own rounding).  A row has two sums of its weights, by tile parity
// (i / c) % 2: as rounded, the output's denominator, so that what all of a row's
// weights have in common cancels; and in fp32 before it, for lse.
//
// Tile order: the runs, the shared tiles, the own ones.
//
// Roles (12 warps).  Softmax warpgroups 0 and 1 (warps 0 - 3, 4 - 7) take the even
// and the odd tiles, a thread a row; S and P are double buffered, O is one.  Before
// that they load Q and the first run tiles, a warp a run, by 16-byte asynchronous
// copies (one warp took 4700 cycles for a tile); warps 8 and 9 load the further ones.  Warp 8
// loads entries: by TMA boxes of a page (or the largest power of two of its rows),
// row by row where a page is missing.  Warp 10 issues QK (a warpgroup's next as soon
// as it has read the last S), warp 11 PV.
//
// All waits are bounded in time and every thread reaches the cluster barriers.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "prefix_attn.cuh"

namespace csa {
namespace pa {

constexpr int kTile = 128, kDim = 128;
constexpr int kStages = 5;                    // a tile lives ~6700 cycles: load, QK, softmax, PV
constexpr int kTileBytes = kTile * kDim * 2;
constexpr int kRegion = kTile * 128;          // the 64-dim half of a tile
constexpr int kPairs = 16;                    // most pairs of a job
constexpr int kSoftWarps = 8, kEntryWarp = 8, kRunWarp = 9, kQkWarp = 10, kPvWarp = 11;
constexpr int kThreads = 384;
constexpr int kFull = 8 * 33;                 // arrivals that fill a stage: 8 warps' lanes and words
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColP = 256, kColO = 384;   // S, P of tile parity w at 128 w, 256 + 64 w
constexpr float kMost = 1.2676506e30f;        // 2^100: a row's weights beyond it are done again

enum : int { kShared = 0, kOwn = 1, kRuns = 2, kEnd = 3 };

struct Pair {
  int b, t, n, nw;        // sequence, token; visible entries; window rows (0 .. W)
  int p, slot;            // position, its ring slot
};
// A tile: its kind; own: the pairs u .. u + m - 1; at: an own tile's parity, the first
// run's number.  One 16-byte word.
struct __align__(16) Desc {
  int kind, u, m, at;
};

struct __align__(1024) Smem {
  uint8_t q[kTileBytes];
  uint8_t kv[kStages][kTileBytes];     // reused at the end: the CTA's O (64 KB), then the ranks' parts of its rows (64 KB)
  uint64_t kv_full[kStages], kv_empty[kStages], q_full, s_full[2], s_free[2], p_full[2], pv_done[2];
  uint64_t drain[2], joined;
  // (tile, value) on its way between the warpgroups: a row's M (by the tile parity it
  // comes from) and sums (by the parity they belong to)
  unsigned long long m_next[2][kTile];
  ulonglong2 l_sum[3][kTile];          // rounded and exact (the third: the runs')
  uint8_t redo[kTile];
  // M, the sums and whether to do the row again: the CTA's rows, the ranks' of the rows it finishes
  float4 ml[kTile], ml_in[kTile];
  uint4 valid[kStages];                // which rows are keys
  int rows[32];                        // page chunks on their way to the boxes
  Desc desc[kStages];
  float sink_l2[kTile];                // by head
  Pair pair[kPairs];
  int npair;
  int group, tile, shared, leader;
  uint32_t tmem;
  int tiles;                           // of this CTA, once the last S is on its way
  int abort_flag;
};

struct Args : PrefixAttnArgs {
  float scale_log2;     // |tau| log2(e)
  int negate;           // tau < 0: Q is negated on load
  int box;              // rows of a page chunk that a TMA box brings (0: pages too odd)
  uint32_t p_mul, p_shift;   // key / P = (key p_mul) >> (32 + p_shift), P > 1
  int log_c;
  uint32_t h_inv;       // ceil(2^16 / H): r / H = r h_inv >> 16 for r < 128
  int c;                // cluster size
  int ppt;              // pairs a job
  int tail_runs, win_runs;   // 16-key runs that a rank takes of each pair: entries, window
  int pair_runs, log_room;   // the room they have in the run tiles: a pair lies in one or fills several
  uint4 off[kPairs];         // lanes that are not pair u's (here, a constant's address: an MMA takes them uniform)
  unsigned long long wait_ns;
  unsigned hint_ns;
};

// ------------------------------------------------------------------- waits
__device__ __forceinline__ bool try_wait(uint64_t* bar, uint32_t parity, uint32_t hint) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(hint)
      : "memory");
  return ok != 0;
}
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, const Args& a, volatile int* abort_flag,
                                       int site) {
  const uint64_t t0 = global_ns();
  while (true) {
    if (try_wait(bar, parity, a.hint_ns)) return true;
    if (*abort_flag) return false;
    if (global_ns() - t0 > a.wait_ns) break;
  }
  atomicCAS(a.status, 0, CSA_ERR_TIMEOUT | (site << 8));
  *abort_flag = 1;
  return false;
}
// Bounded wait of one thread.
__device__ __forceinline__ bool wait1(uint64_t* bar, uint32_t parity, const Args& a, volatile int* abort_flag,
                                      int site) {
  return try_wait(bar, parity, a.hint_ns) || wait_slow(bar, parity, a, abort_flag, site);
}
// Bounded wait with the same answer in every lane of the warp.
__device__ __forceinline__ bool waitw(uint64_t* bar, uint32_t parity, const Args& a, volatile int* abort_flag,
                                      int site) {
  const bool ok = try_wait(bar, parity, a.hint_ns) || wait_slow(bar, parity, a, abort_flag, site);
  return __all_sync(0xffffffffu, ok);
}
// A value handed from one thread to one other, tagged with its tile (one 64-bit
// word, so both arrive together): a satisfied read costs a shared-memory load where
// an mbarrier wait took 200 to 300 cycles.
__device__ __forceinline__ void hand_over(unsigned long long* slot, int tile, float x) {
  const unsigned long long v =
      (static_cast<unsigned long long>(static_cast<uint32_t>(tile)) << 32) | __float_as_uint(x);
  asm volatile("st.volatile.shared.b64 [%0], %1;" ::"r"(smem_u32(slot)), "l"(v) : "memory");
}
__device__ __forceinline__ float handed(const unsigned long long* slot, int* tile) {
  unsigned long long v;
  asm volatile("ld.volatile.shared.b64 %0, [%1];" : "=l"(v) : "r"(smem_u32(slot)) : "memory");
  *tile = static_cast<int>(v >> 32);
  return __uint_as_float(static_cast<uint32_t>(v));
}
// Two values, each with its tag (*tile: -2 while the tags differ).
__device__ __forceinline__ void hand_over(ulonglong2* slot, int tile, float2 x) {
  const unsigned long long tag = static_cast<unsigned long long>(static_cast<uint32_t>(tile)) << 32;
  asm volatile("st.volatile.shared.v2.b64 [%0], {%1, %2};" ::"r"(smem_u32(slot)), "l"(tag | __float_as_uint(x.x)),
               "l"(tag | __float_as_uint(x.y))
               : "memory");
}
__device__ __forceinline__ float2 handed(const ulonglong2* slot, int* tile) {
  unsigned long long v, w;
  asm volatile("ld.volatile.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v), "=l"(w) : "r"(smem_u32(slot)) : "memory");
  *tile = (v >> 32) == (w >> 32) ? static_cast<int>(v >> 32) : -2;
  return make_float2(__uint_as_float(static_cast<uint32_t>(v)), __uint_as_float(static_cast<uint32_t>(w)));
}
// Bounded wait of a warp for its rows' values of `tile`.
template <typename Slot, typename Value>
__device__ __forceinline__ bool take(const Slot* slot, int tile, Value* x, const Args& a, volatile int* abort_flag,
                                     int site) {
  int t;
  *x = handed(slot, &t);
  if (__all_sync(0xffffffffu, t == tile)) return true;
  const uint64_t t0 = global_ns();
  while (true) {
    *x = handed(slot, &t);
    if (__all_sync(0xffffffffu, t == tile)) return true;
    const bool late = global_ns() - t0 > a.wait_ns;
    if (late && !*abort_flag) {
      atomicCAS(a.status, 0, CSA_ERR_TIMEOUT | (site << 8));
      *abort_flag = 1;
    }
    if (__any_sync(0xffffffffu, late || *abort_flag)) return false;
  }
}
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = global_ns();
  while (!try_wait(bar, parity, 1000u))
    if (global_ns() - t0 > 1000000ull) break;
}

// ------------------------------------------------------------ PTX helpers
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// (x0, x1) += (y0, y1) on the packed fp32 pipe
__device__ __forceinline__ void add2(float2& x, float y0, float y1) {
  asm("{\n\t.reg .b64 rx, ry;\n\t"
      "mov.b64 rx, {%0, %1};\n\tmov.b64 ry, {%2, %3};\n\t"
      "add.rn.f32x2 rx, rx, ry;\n\tmov.b64 {%0, %1}, rx;\n\t}"
      : "+f"(x.x), "+f"(x.y)
      : "f"(y0), "f"(y1));
}
// (x0, x1) += the two bf16 of p
__device__ __forceinline__ void add_bf16(float2& x, uint32_t p) {
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "add.rn.f32.bf16 %0, lo, %0;\n\tadd.rn.f32.bf16 %1, hi, %1;\n\t}"
      : "+f"(x.x), "+f"(x.y)
      : "r"(p));
}
__device__ __forceinline__ float2 operator+(float2 a, float2 b) { return make_float2(a.x + b.x, a.y + b.y); }
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
#define PA_TMEM_LD_X32(taddr, r)                                                                          \
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "                                                 \
               "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"                                  \
               "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"                 \
               : "=r"((r)[0]), "=r"((r)[1]), "=r"((r)[2]), "=r"((r)[3]), "=r"((r)[4]), "=r"((r)[5]),      \
                 "=r"((r)[6]), "=r"((r)[7]), "=r"((r)[8]), "=r"((r)[9]), "=r"((r)[10]), "=r"((r)[11]),    \
                 "=r"((r)[12]), "=r"((r)[13]), "=r"((r)[14]), "=r"((r)[15]), "=r"((r)[16]),               \
                 "=r"((r)[17]), "=r"((r)[18]), "=r"((r)[19]), "=r"((r)[20]), "=r"((r)[21]),               \
                 "=r"((r)[22]), "=r"((r)[23]), "=r"((r)[24]), "=r"((r)[25]), "=r"((r)[26]),               \
                 "=r"((r)[27]), "=r"((r)[28]), "=r"((r)[29]), "=r"((r)[30]), "=r"((r)[31])                \
               : "r"(taddr))

// If `on`, D[tmem] += A[tmem] * B[smem]; lanes whose bit is set in `off` are not written.
__device__ __forceinline__ void mma_ts_lanes(uint32_t on, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                             uint32_t idesc, const uint4& off) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, 1, 0;\n\tsetp.ne.b32 q, %8, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%4, %5, %6, %7}, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(off.x), "r"(off.y), "r"(off.z), "r"(off.w), "r"(on)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, 1, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc)
      : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(smem_u32(bar)), "r"(n)
               : "memory");
}
// K-major operand, 16-element step j; the same tile with its rows as K.
__device__ __forceinline__ uint64_t desc_kmajor(uint32_t base, int j) {
  return make_sdesc(base + (j >> 2) * kRegion + (j & 3) * 32, 16, 1024, kLayoutSw128);
}
__device__ __forceinline__ uint64_t desc_mnmajor(uint32_t base, int j) {
  return make_sdesc(base + j * 2048, kRegion, 1024, kLayoutSw128);
}
// One lane of the (converged) warp.  The compiler knows that a branch on this runs
// one thread and keeps the MMA operands in uniform registers; under `lane == 0` it
// wraps every MMA in a loop over threads (measured 3000 cycles for 8 of them).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// Bits of lanes outside [lo, hi), 32 at a time.
__host__ __device__ __forceinline__ void lanes_off(uint32_t off[4], int lo, int hi) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int a = lo - 32 * i, b = hi - 32 * i;
    const uint32_t below_a = a >= 32 ? 0xffffffffu : a <= 0 ? 0u : (1u << a) - 1u;
    const uint32_t below_b = b >= 32 ? 0xffffffffu : b <= 0 ? 0u : (1u << b) - 1u;
    off[i] = ~(below_b & ~below_a);
  }
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
// Copy shared memory to a peer's; its mbarrier counts the bytes.
__device__ __forceinline__ void push_to_peer(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "r"(smem_u32(src)), "r"(bytes), "r"(bar)
               : "memory");
}

// ----------------------------------------------------------------- set-up
// Where group g's members start (kept within the list).
__device__ __forceinline__ int group_start(const Args& a, int g) {
  return min(max(a.group_off[g], 0), a.n_seq);
}

// A warp: the job's group and tile of pairs (jobs are numbered group by group); false
// when there is no such job.  Four groups a lane (1024 groups of a sequence each, 64 heads:
// 117 us with one, 85).
__device__ bool find_job(const Args& a, int job, Smem* sm, int* start, int* count) {
  const int lane = threadIdx.x & 31;
  if (a.G == 1) {
    if (sm != nullptr && lane == 0) {
      sm->group = 0;
      sm->tile = job;
    }
    __syncwarp();
    *start = 0;
    *count = a.n_seq;
    return static_cast<long long>(job) * a.ppt < static_cast<long long>(a.n_seq) * a.T;
  }
  int before = 0;
  for (int g0 = 0; g0 < a.G; g0 += 128) {
    const int g = g0 + 4 * lane;
    int o[5], jobs[4], all = 0;
#pragma unroll
    for (int k = 0; k < 5; ++k) o[k] = group_start(a, min(g + k, a.G));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      jobs[k] = static_cast<int>((static_cast<uint32_t>(max(o[k + 1] - o[k], 0)) * a.T + a.ppt - 1) /
                                 static_cast<uint32_t>(a.ppt));
      all += jobs[k];
    }
    const int incl = warp_incl_scan(all);
    const uint32_t hit = __ballot_sync(0xffffffffu, before + incl > job);
    if (hit) {
      const int src = __ffs(hit) - 1;
      int at = before + incl - all, k = 0, first = o[0], n = max(o[1] - o[0], 0);
#pragma unroll
      for (int x = 0; x < 3; ++x) {
        if (k == x && at + jobs[x] <= job) {
          at += jobs[x];
          k = x + 1;
          first = o[x + 1];
          n = max(o[x + 2] - o[x + 1], 0);
        }
      }
      if (sm != nullptr && lane == src) {
        sm->group = g + k;
        sm->tile = job - at;
      }
      *start = __shfl_sync(0xffffffffu, first, src);
      *count = __shfl_sync(0xffffffffu, n, src);
      __syncwarp();
      return true;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

// Warp 0: the job's pairs, and the entries that all of them share (whole tiles): a lone
// pair's all.
__device__ void load_pairs(const Args& a, Smem& sm, int o0, int members) {
  const int lane = threadIdx.x & 31;
  const int first = sm.tile * a.ppt;
  const int np = min(members * a.T - first, a.ppt);
  const int lead = a.group_seq[o0];
  int n = max(a.group_shared[sm.group], 0);
  if (lane < np) {
    Pair pr{-1, 0, 0, 0, -1, 0};
    const int i = first + lane;
    const int b = a.group_seq[o0 + i / a.T];
    if (b >= 0 && b < a.B) {
      pr.b = b;
      pr.t = i % a.T;
      const long long p = static_cast<long long>(a.q_pos0[b]) + pr.t;
      pr.p = static_cast<int>(min(p, static_cast<long long>(INT32_MAX)));
      pr.n = visible_entries(a, b, p);
      pr.slot = p < 0 || a.W == 0 ? 0 : static_cast<int>(static_cast<uint32_t>(pr.p) % static_cast<uint32_t>(a.raw_cap));
      pr.nw = p < 0 ? 0 : static_cast<int>(min(static_cast<long long>(a.W), p + 1));
    } else {
      atomicCAS(a.status, 0, CSA_ERR_INVALID_ARG | (4 << 8));
    }
    sm.pair[lane] = pr;
    n = np == 1 ? pr.n : min(n, pr.n);
  } else if (np == 1) {
    n = INT_MAX;
  } else if (lane == 31) {       // (a job has 16 pairs at most)
    n = lead < 0 || lead >= a.B
            ? 0
            : static_cast<int>(min(static_cast<long long>(n),
                                   static_cast<long long>(max(min(a.held[lead], a.max_pages), 0)) * a.P));
  }
  n = __reduce_min_sync(0xffffffffu, n);
  if (lane == 0) {
    sm.npair = np;
    sm.shared = n / kTile;
    sm.leader = np == 1 ? a.group_seq[o0 + first / a.T] : lead;
  }
}

// One row again on CUDA cores (a warp; a lane 4 dims): the online softmax in fp32 over
// the row's entries and window, as the definition states.
__device__ __noinline__ void row_exact(const Args& a, const Pair& pr, int h, float sink_l2) {
  const int lane = threadIdx.x & 31;
  const size_t row = (static_cast<size_t>(pr.b) * a.T + pr.t) * a.H + h;
  const float sl2 = a.negate ? -a.scale_log2 : a.scale_log2;
  float q[4], acc[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
  auto load4 = [&](const __nv_bfloat16* p, float x[4]) {
    const uint2 v = *reinterpret_cast<const uint2*>(p + 4 * lane);
    x[0] = __uint_as_float(v.x << 16);
    x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16);
    x[3] = __uint_as_float(v.y & 0xffff0000u);
  };
  load4(static_cast<const __nv_bfloat16*>(a.q) + row * kDim, q);
  auto visit = [&](const __nv_bfloat16* key) {
    float k[4];
    load4(key, k);
    float x = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    x *= sl2;
    const float mn = x > m ? x : m;
    const float f = mn > -INFINITY ? exp2f(m - mn) : 1.f, w = exp2f(x - (mn > -INFINITY ? mn : 0.f));
    l = fmaf(l, f, w);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = fmaf(acc[e], f, w * k[e]);
    m = mn;
  };
  const int32_t* tab = a.table + static_cast<size_t>(pr.b) * a.max_pages;
  for (int s = 0; s < pr.n; ++s) {
    const int id = tab[s / a.P];
    if (id >= 0 && id < a.N)
      visit(static_cast<const __nv_bfloat16*>(a.pool) + (static_cast<size_t>(id) * a.P + s % a.P) * kDim);
  }
  for (int j = 0; j < pr.nw; ++j)
    visit(static_cast<const __nv_bfloat16*>(a.kv_raw) +
          (static_cast<size_t>(pr.b) * a.raw_cap + (pr.p - j) % a.raw_cap) * kDim);
  float sc = 0.f, lse = -INFINITY;
  if (l != 0.f) {
    const float X = fmaxf(m, sink_l2), f = exp2f(m - X);
    sc = __fdiv_rn(f, fmaf(l, f, exp2f(sink_l2 - X)));
    lse = (m + log2f(l)) * 0.6931471805599453f;
  }
  uint2 o2;
  o2.x = pack_bf16(acc[0] * sc, acc[1] * sc);
  o2.y = pack_bf16(acc[2] * sc, acc[3] * sc);
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row * kDim + lane * 4) = o2;
  if (a.lse && lane == 0) a.lse[row] = lse;
}

// The factor of O and the lse of a row with stabiliser M and sums L, rounded and exact
// (log2 domain).
__device__ __forceinline__ void finish_row(float M, float2 L, float sink_l2, float* sc, float* lse) {
  *sc = 0.f;
  *lse = -INFINITY;
  if (L.x != 0.f) {
    const float X = fmaxf(M, sink_l2), fm = ex2(M - X);
    *sc = __fdiv_rn(fm, fmaf(L.x, fm, ex2(sink_l2 - X)));
    *lse = (M + log2f(L.y)) * 0.6931471805599453f;
  }
}

// Entry `key` of sequence b as a row of the pool, or -1.
__device__ __forceinline__ int entry_row(const Args& a, int b, int key) {
  const int pg = a.P > 1 ? static_cast<int>(__umulhi(key, a.p_mul) >> a.p_shift) : key;
  const int id = a.table[static_cast<size_t>(b) * a.max_pages + pg];
  return id >= 0 && id < a.N ? id * a.P + (key - pg * a.P) : -1;
}

// How many of this rank's entry tiles lie in [i0, ceil(n / 128)).
__device__ __forceinline__ int tiles_of(int i0, int n, int log_c) {
  const int end = static_cast<int>((static_cast<uint32_t>(n) + kTile - 1) / kTile);
  return end > i0 ? (end - i0 + (1 << log_c) - 1) >> log_c : 0;
}
// Pair u continues the tiles of pair u - 1: the same sequence, as many entries.
__device__ __forceinline__ bool joined(const Smem& sm, int u) {
  return u > 0 && sm.pair[u].b == sm.pair[u - 1].b && sm.pair[u].n == sm.pair[u - 1].n;
}

// (Without lse a tile's exact sums are left out: 32 x 128 queries over 8192 entries take
// 29.2 us for 29.9.)
template <bool kLse>
__global__ void __launch_bounds__(kThreads, 1) prefix_attn_kernel(const __grid_constant__ Args a,
                                                                  const __grid_constant__ CUtensorMap pool_map) {
  extern __shared__ __align__(1024) uint8_t pa_smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(pa_smem_raw) + 1023) &
                                      ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &sm.abort_flag;
  const int rank = static_cast<int>(cluster_rank());
  const int job = blockIdx.x >> a.log_c;

  // What the entry warp looks up ahead, while warp 0 still loads the job's pairs: the
  // page chunks of this rank's first tiles of the group's first member.
  int pre_b = -1, pre_row = -1;
  const int chunks = a.box ? kTile / a.box : 32, ahead = a.box ? 32 / chunks : 1;
  if (warp == kEntryWarp) {
    int start, members, b = -1;
    if (a.box && find_job(a, job, nullptr, &start, &members)) b = a.group_seq[start];
    if (b >= 0 && b < a.B) {
      const long long key = (rank + static_cast<long long>(lane / chunks) * a.c) * kTile + (lane % chunks) * a.box;
      pre_b = b;
      if (key < static_cast<long long>(a.max_pages) * a.P) pre_row = entry_row(a, b, static_cast<int>(key));
    }
  } else if (warp == 0) {
    int start, members;
    const bool some = find_job(a, job, &sm, &start, &members);
    if (some) load_pairs(a, sm, start, members);
    else if (lane == 0) sm.group = -1;
  } else if (warp == 1 && lane == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.kv_full[s], kFull);
      mbar_init(&sm.kv_empty[s], 1);
    }
    mbar_init(&sm.q_full, 32 * kSoftWarps);
    for (int w = 0; w < 2; ++w) {
      mbar_init(&sm.s_full[w], 2);
      mbar_init(&sm.s_free[w], 128);
      mbar_init(&sm.p_full[w], 128);
      mbar_init(&sm.pv_done[w], 1);
      mbar_init(&sm.drain[w], 1);
    }
    mbar_init(&sm.joined, 1);
    sm.abort_flag = 0;
    sm.tiles = INT32_MAX;
    fence_mbar_init();
  } else if (warp >= 2 && warp < 6) {
    const int h = threadIdx.x - 64;
    sm.sink_l2[h] = a.sink && h < a.H ? a.sink[h] * 1.4426950408889634f : -INFINITY;
  } else if (warp == kQkWarp) {
    tmem_alloc(&sm.tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const bool idle = sm.group < 0;      // the same in every CTA of the cluster
  const int room = a.pair_runs, run_tiles = idle ? 0 : (sm.npair * room + 7) / 8;
  // Where row x (0 .. 15) of run `run` lies, or null.
  auto run_row = [&](int run, int x) -> const __nv_bfloat16* {
    // (a pair has a power of two of runs in a tile, or whole tiles)
    const int u = room <= 8 ? run >> a.log_room : run / room, i = run - u * room;
    if (u >= sm.npair) return nullptr;
    const Pair pr = sm.pair[u];
    if (i < a.tail_runs) {
      const int key = (pr.n & ~(kTile - 1)) + (rank + i * a.c) * 16 + x;
      const int y = key < pr.n ? entry_row(a, pr.b, key) : -1;
      return y >= 0 ? static_cast<const __nv_bfloat16*>(a.pool) + static_cast<size_t>(y) * kDim : nullptr;
    }
    // how many tokens before the query's own
    const int back = (rank + (i - a.tail_runs) * a.c) * 16 + x;
    if (i >= a.tail_runs + a.win_runs || back >= pr.nw) return nullptr;
    const int slot = pr.slot - back + (back > pr.slot ? a.raw_cap : 0);
    return static_cast<const __nv_bfloat16*>(a.kv_raw) + (static_cast<size_t>(pr.b) * a.raw_cap + slot) * kDim;
  };
  // the first entry tile of this rank behind the shared ones
  const int own0 = idle ? 0 : sm.shared + ((rank - sm.shared) & (a.c - 1));

  if (!idle && (warp == kEntryWarp || warp == kRunWarp)) {
    // ================================================================= producers
    const int half = lane >> 4, c = lane & 15;
    bool ok = true;
    // The first kStages run tiles are the softmax warps'.  Both warps here see every
    // stage through its uses (an mbarrier tells a phase from the next alone, so a
    // waiter must not skip one).
    int g = kStages;
    auto stage_free = [&]() {
      const int use = g / kStages;
      return use < 1 || waitw(&sm.kv_empty[g % kStages], (use - 1) & 1, a, abort_flag, 20);
    };
    // One tile row by row: src(r) gives where tile row r's key lies, or null.  Runs of 16
    // rows without a key are left out (and by the PV).
    auto put = [&](const Desc& d, int rows, auto&& src) {
      const int stage = g % kStages;
      if (!stage_free()) { ok = false; return; }
      const char* none = static_cast<const char*>(a.pool);
      uint32_t dst = smem_u32(sm.kv[stage]) + (c >> 3) * kRegion + half * 128;
      const uint32_t cx = static_cast<uint32_t>((c & 7) ^ half);
      uint4 bits = make_uint4(0u, 0u, 0u, 0u);
      // (rolled: code that runs once or twice is paid for in instruction fetches)
#pragma unroll 1
      for (int i = 0; 32 * i < rows; ++i, dst += 32 * 128) {
        const unsigned long long x = reinterpret_cast<unsigned long long>(src(32 * i + lane));
        const uint32_t word = __ballot_sync(0xffffffffu, x != 0ull);
        if (i == 0) bits.x = word;
        else if (i == 1) bits.y = word;
        else if (i == 2) bits.z = word;
        else bits.w = word;
#pragma unroll 1
        for (int run = 0; run < 2; ++run) {
          if (!((word >> (16 * run)) & 0xffffu)) continue;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const unsigned long long y = __shfl_sync(0xffffffffu, x, 16 * run + 2 * j + half);
            cp_async16(dst + (8 * run + j) * 256 + ((cx ^ static_cast<uint32_t>((2 * j) & 7)) << 4),
                       (y ? reinterpret_cast<const char*>(y) : none) + c * 16, y ? 16u : 0u);
          }
        }
      }
      cp_async_mbar_arrive(&sm.kv_full[stage]);
      if (lane == 0) {
        sm.valid[stage] = bits;
        sm.desc[stage] = d;
        mbar_arrive_n(&sm.kv_full[stage], kFull - 32);
      }
      ++g;
    };
    auto pool_row = [&](int b, int key) -> const void* {
      const int x = entry_row(a, b, key);
      return x >= 0 ? static_cast<const __nv_bfloat16*>(a.pool) + static_cast<size_t>(x) * kDim : nullptr;
    };
    // The further run tiles: the odd or the even ones.
    auto put_runs = [&](int odd) {
      while (ok && g < run_tiles) {
        if ((g & 1) != odd) {
          ok = stage_free();
          ++g;
          continue;
        }
        const int at = 8 * g, runs = min(8, sm.npair * room - at);
        put(Desc{kRuns, 0, 0, at}, runs * 16, [&](int r) -> const void* { return run_row(at + (r >> 4), r & 15); });
      }
    };
    if (warp == kEntryWarp) {
      // This rank's entry tiles i, i + c, .. of sequence b below tile `end`.  The page chunks of
      // the next 32 / chunks tiles are looked up at once, a lane each; then one
      // thread walks those tiles (per tile, a warp's lookups, votes and branches paced
      // the loop at 2000 cycles; these take a few dozen instructions).
      auto put_tiles = [&](int kind, int u, int m, int b, int i, int end) {
        while (ok && i < end) {
          const int batch = min(ahead, (end - i + a.c - 1) >> a.log_c);
          int good = 0;                  // tiles before the first with a missing page
          if (a.box) {
            const int t = lane / chunks;
            int row = -1;
            if (t < batch)
              row = b == pre_b && i == rank ? pre_row : entry_row(a, b, (i + t * a.c) * kTile + (lane % chunks) * a.box);
            const uint32_t bad = __ballot_sync(0xffffffffu, t < batch && row < 0);
            good = bad ? (__ffs(bad) - 1) / chunks : batch;
            sm.rows[lane] = row;
            __syncwarp();
            bool fine = true;
            if (elect_one()) {
              int stage = g % kStages, use = g / kStages, tile = i;
              for (int k = 0; k < good; ++k, tile += a.c) {
                if (use >= 1 && !wait1(&sm.kv_empty[stage], (use - 1) & 1, a, abort_flag, 20)) { fine = false; break; }
                sm.valid[stage] = make_uint4(0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu);
                sm.desc[stage] = Desc{kind, u, m, (tile >> a.log_c) & 1};
                mbar_expect_tx(&sm.kv_full[stage], kTileBytes);
                uint32_t dst = smem_u32(sm.kv[stage]);
                for (int x = 0; x < chunks; ++x, dst += a.box * 128) {
                  const int y = sm.rows[k * chunks + x];
                  tma_load_2d(dst, reinterpret_cast<uint64_t>(&pool_map), 0, y, &sm.kv_full[stage]);
                  tma_load_2d(dst + kRegion, reinterpret_cast<uint64_t>(&pool_map), 64, y, &sm.kv_full[stage]);
                }
                mbar_arrive_n(&sm.kv_full[stage], kFull);
                if (++stage == kStages) { stage = 0; ++use; }
              }
            }
            ok = __all_sync(0xffffffffu, fine);
            g += good;
            i += good * a.c;
          }
          if (ok && good < batch) {
            const int key0 = i * kTile;
            put(Desc{kind, u, m, (i >> a.log_c) & 1}, kTile, [&](int r) { return pool_row(b, key0 + r); });
            i += a.c;
          }
        }
      };
      put_runs(1);
      g = run_tiles;
      put_tiles(kShared, 0, 0, sm.leader, rank, sm.shared);
      for (int u = 0; u < sm.npair && ok;) {
        int m = 1;
        while (u + m < sm.npair && joined(sm, u + m)) ++m;
        put_tiles(kOwn, u, m, sm.pair[u].b, own0, sm.pair[u].n / kTile);
        u += m;
      }
      if (ok) put(Desc{kEnd, 0, 0, 0}, 0, [](int) -> const void* { return nullptr; });
      cp_async_wait<0>();
    } else {
      put_runs(0);
      cp_async_wait<0>();
    }
  } else if (!idle && warp == kQkWarp) {
    // ================================================================= S = Q K^T
    constexpr uint32_t idesc_qk = idesc_bf16(128, 128, 0, 0);
    if (elect_one()) {
      const uint64_t qd = desc_kmajor(smem_u32(sm.q), 0);
      bool ok = wait1(&sm.q_full, 0, a, abort_flag, 21);
      int stage = 0, round = 0;
      for (int g = 0, ends = 0; ok; ++g) {
        const int w = g & 1;
        if (!ends) {
          ok = wait1(&sm.kv_full[stage], round & 1, a, abort_flag, 25);
          if (!ok) break;
          ends = sm.desc[stage].kind == kEnd;
        }
        ok = g < 2 || wait1(&sm.s_free[w], ((g >> 1) - 1) & 1, a, abort_flag, 27);
        if (!ok) break;
        if (ends) {                 // the end, told to both warpgroups
          if (ends == 1) *const_cast<volatile int*>(&sm.tiles) = g;
          mbar_arrive_n(&sm.s_full[w], 2);
          if (++ends == 3) break;
          continue;
        }
        fence_proxy_async();
        tc_fence_after();
        const uint64_t kd = desc_kmajor(smem_u32(sm.kv[stage]), 0);
        const uint32_t scol = tmem + kColS + 128 * w;
#pragma unroll
        for (int j = 0; j < kDim / 16; ++j) {
          // (16 elements on: 32 bytes, or the other 64-dim half)
          const uint64_t step = ((j >> 2) * kRegion + (j & 3) * 32) >> 4;
          mma_bf16(scol, qd + step, kd + step, idesc_qk, j > 0);
        }
        tc_commit(&sm.s_full[w]);
        mbar_arrive(&sm.s_full[w]);
        if (++stage == kStages) { stage = 0; ++round; }
      }
      tc_commit(&sm.drain[0]);
      drain_wait(&sm.drain[0], 0);
    }
    __syncwarp();
  } else if (!idle && warp == kPvWarp) {
    // ================================================================= O += P K
    constexpr uint32_t idesc_pv = idesc_bf16(128, 128, 0, 1);
    const uint32_t ocol = tmem + kColO;
    if (elect_one()) {
      int stage = 0, round = 0;
      for (int g = 0;; ++g) {
        const int w = g & 1;
        if (!wait1(&sm.kv_full[stage], round & 1, a, abort_flag, 28)) break;
        const Desc d = sm.desc[stage];
        if (d.kind == kEnd) break;
        const uint64_t kd = desc_mnmajor(smem_u32(sm.kv[stage]), 0);
        const uint32_t pcol = tmem + kColP + 64 * w;
        // (steps without a key are left out: nothing was loaded for them)
        const uint4 bits = sm.valid[stage];
        const uint32_t words[4] = {bits.x, bits.y, bits.z, bits.w};
        const bool whole = (bits.x & bits.y & bits.z & bits.w) == 0xffffffffu;
        const bool all_rows = d.kind == kShared || sm.npair == 1;      // else the rows' lanes alone
        if (!wait1(&sm.p_full[w], (g >> 1) & 1, a, abort_flag, 26)) break;
        fence_proxy_async();
        tc_fence_after();
        if (all_rows && whole) {
#pragma unroll
          for (int j = 0; j < kTile / 16; ++j) mma_ts(ocol, pcol + 8 * j, kd + j * (2048 >> 4), idesc_pv);
        } else {
          if (all_rows) {
#pragma unroll
            for (int j = 0; j < kTile / 16; ++j)
              if (words[j >> 1] & (0xffffu << (16 * (j & 1)))) mma_ts(ocol, pcol + 8 * j, kd + j * (2048 >> 4), idesc_pv);
          } else if (g < run_tiles) {
#pragma unroll
            for (int j = 0; j < kTile / 16; ++j)
              mma_ts_lanes(words[j >> 1] & (0xffffu << (16 * (j & 1))), ocol, pcol + 8 * j, kd + j * (2048 >> 4), idesc_pv,
                           a.off[room <= 8 ? (8 * g + j) >> a.log_room : 8 * g / room]);
          } else {
            uint4 off = a.off[d.u];
            for (int u = d.u + 1; u < d.u + d.m; ++u) {
              const uint4 more = a.off[u];
              off = make_uint4(off.x & more.x, off.y & more.y, off.z & more.z, off.w & more.w);
            }
#pragma unroll
            for (int j = 0; j < kTile / 16; ++j)
              mma_ts_lanes(words[j >> 1] & (0xffffu << (16 * (j & 1))), ocol, pcol + 8 * j, kd + j * (2048 >> 4), idesc_pv,
                           off);
          }
        }
        tc_commit(&sm.kv_empty[stage]);
        tc_commit(&sm.pv_done[w]);
        if (++stage == kStages) { stage = 0; ++round; }
      }
      // whatever was issued has finished before O is read and tensor memory released
      tc_commit(&sm.drain[1]);
      drain_wait(&sm.drain[1], 0);
    }
    __syncwarp();
  } else if (!idle && warp < kSoftWarps) {
    // ================================================================= softmax
    // tiles g % 2 == w
    const int w = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t scol = tmem + lane_addr + kColS + 128 * w, pcol = tmem + lane_addr + kColP + 64 * w;
    const uint32_t ocol = tmem + lane_addr + kColO + 64 * w;      // (to be cleared)
    const int rows = sm.npair * a.H;
    {
      // Q: 16 lanes a row; rows beyond the job's are zero
      const int c = threadIdx.x & 15;
      const uint32_t dst = smem_u32(sm.q) + (c >> 3) * kRegion;
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + c * 8;
#pragma unroll
      for (int i = 0; i < kTile / kSoftWarps / 2; ++i) {
        const int y = (threadIdx.x >> 4) + 2 * kSoftWarps * i;
        const int uy = static_cast<int>((static_cast<uint32_t>(y) * a.h_inv) >> 16);
        size_t row = 0;
        bool some = y < rows;
        if (some) {
          const int b = sm.pair[uy].b;
          some = b >= 0;
          row = (static_cast<size_t>(max(b, 0)) * a.T + sm.pair[uy].t) * a.H + (y - uy * a.H);
        }
        cp_async16(dst + y * 128 + (((c & 7) ^ (y & 7)) << 4), q + row * kDim, some ? 16u : 0u);
      }
      cp_async_commit();
      // The first run tiles: run `warp` of each, 16 lanes a row.
#pragma unroll 1
      for (int t = 0; t < min(run_tiles, kStages); ++t) {
        const unsigned long long x = reinterpret_cast<unsigned long long>(run_row(8 * t + warp, lane & 15));
        const uint32_t word = __ballot_sync(0xffffffffu, x != 0ull) & 0xffffu;
        if (word) {
          const int half = lane >> 4;
          const uint32_t to = smem_u32(sm.kv[t]) + (c >> 3) * kRegion + (16 * warp + half) * 128;
          const uint32_t cx = static_cast<uint32_t>((c & 7) ^ half);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const unsigned long long y = __shfl_sync(0xffffffffu, x, 2 * j + half);
            cp_async16(to + j * 256 + ((cx ^ static_cast<uint32_t>((2 * j) & 7)) << 4),
                       (y ? reinterpret_cast<const char*>(y) : static_cast<const char*>(a.pool)) + c * 16, y ? 16u : 0u);
          }
        }
        cp_async_mbar_arrive(&sm.kv_full[t]);
        if (lane == 0) {
          reinterpret_cast<uint16_t*>(&sm.valid[t])[warp] = static_cast<uint16_t>(word);
          if (warp == 0) sm.desc[t] = Desc{kRuns, 0, 0, 8 * t};
          mbar_arrive(&sm.kv_full[t]);
        }
      }
      cp_async_commit();
      uint32_t z[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) z[e] = 0u;
#pragma unroll
      for (int cc = 0; cc < 64; cc += 16) tmem_st16(ocol + cc, z);
      tmem_st_wait();
      tc_fence_before();
      hand_over(&sm.m_next[w][r], -1, -INFINITY);
      hand_over(&sm.l_sum[w][r], -1, make_float2(0.f, 0.f));
      if (w == 0) {
        hand_over(&sm.l_sum[2][r], -1, make_float2(0.f, 0.f));
        sm.redo[r] = 0;
      }
      cp_async_wait<1>();
      if (a.negate) {
        for (int i = 0; i < kTile / kSoftWarps / 2; ++i) {
          const int y = (threadIdx.x >> 4) + 2 * kSoftWarps * i;
          uint4* v = reinterpret_cast<uint4*>(sm.q + (c >> 3) * kRegion + y * 128 + (((c & 7) ^ (y & 7)) << 4));
          *v = make_uint4(v->x ^ 0x80008000u, v->y ^ 0x80008000u, v->z ^ 0x80008000u, v->w ^ 0x80008000u);
        }
      }
      fence_proxy_async();
      mbar_arrive(&sm.q_full);
    }
    const int u = r < rows ? static_cast<int>((static_cast<uint32_t>(r) * a.h_inv) >> 16) : -1;
    const float sl2 = a.scale_log2;
    const int own_at = run_tiles + tiles_of(rank, sm.shared * kTile, a.log_c);      // the first own tile
    const int p_of = (run_tiles + w) & 1;      // the parity of this warpgroup's shared tiles
    float M = -INFINITY;                 // -inf: not set yet
    float2 l = make_float2(0.f, 0.f);
    bool first_known = false;
    int stage = w;                       // g % kStages
    for (int g = w;; g += 2, stage = stage + 2 >= kStages ? stage + 2 - kStages : stage + 2) {
      const int k = g >> 1;
      if (!waitw(&sm.s_full[w], k & 1, a, abort_flag, 22)) break;
      tc_fence_after();
      // S is on its way to registers while the tile's kind is looked up
      uint32_t v[128];
      PA_TMEM_LD_X32(scol, v);
      PA_TMEM_LD_X32(scol + 32, v + 32);
      PA_TMEM_LD_X32(scol + 64, v + 64);
      PA_TMEM_LD_X32(scol + 96, v + 96);
      const bool end = g >= *const_cast<volatile int*>(&sm.tiles);
      const Desc d = sm.desc[stage];
      const uint4 bits = sm.valid[stage];
      bool mine = d.kind == kShared;       // the tile's MMA writes this row's lane
      int lo = 0, hi = kTile;
      if (d.kind == kOwn) {
        mine = u >= d.u && u < d.u + d.m;
      } else if (d.kind == kRuns) {
        lo = min(max(u * room - d.at, 0), 8) * 16;
        hi = min(max((u + 1) * room - d.at, 0), 8) * 16;
        mine = u >= 0 && hi > lo;
      }
      // every row that counts sees every column
      const bool full = d.kind != kRuns && (bits.x & bits.y & bits.z & bits.w) == 0xffffffffu;
      const bool any = __any_sync(0xffffffffu, mine);
      tmem_ld_wait();
      if (end) break;
      tc_fence_before();
      mbar_arrive(&sm.s_free[w]);
      if (any && !full) {
        uint32_t off[4];
        lanes_off(off, lo, hi);
        const uint32_t see[4] = {mine ? bits.x & ~off[0] : 0u, mine ? bits.y & ~off[1] : 0u,
                                 mine ? bits.z & ~off[2] : 0u, mine ? bits.w & ~off[3] : 0u};
#pragma unroll
        for (int e = 0; e < 128; ++e)
          if (!((see[e >> 5] >> (e & 31)) & 1u)) v[e] = 0xff800000u;   // -inf: weight 0
      }
      // A row's M comes with the first tile in which it sees a key; what is set goes along
      // from tile to tile until all of the warp's rows have theirs.
      if (!first_known) {
        if (g > 0 && !take(&sm.m_next[w ^ 1][r], g - 1, &M, a, abort_flag, 23)) break;
        if (u < 0) M = 0.f;
        const bool sets = mine && M == -INFINITY;
        if (__any_sync(0xffffffffu, sets)) {
          float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 128; e += 2)
            mx4[(e >> 1) & 3] = max3(mx4[(e >> 1) & 3], __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
          // (NaN stays; -inf, where it sees nothing here, sets nothing)
          if (sets) M = max3(max3(mx4[0], mx4[1], mx4[2]), mx4[3], -INFINITY) * sl2;
        }
        hand_over(&sm.m_next[w][r], g, M);
        first_known = __all_sync(0xffffffffu, M != -INFINITY);
      }
      // P's buffer is free once the PV two tiles back has read it
      if (g >= 2 && !waitw(&sm.pv_done[w], (k - 1) & 1, a, abort_flag, 29)) break;
      tc_fence_after();
      float2 sum = make_float2(0.f, 0.f);
      if (any) {
        const float negM = M == -INFINITY ? 0.f : -M;
        float2 s0 = make_float2(0.f, 0.f), s1 = s0, e0 = s0, e1 = s0;
#pragma unroll
        for (int cc = 0; cc < 128; cc += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float x0 = ex2(fmaf(__uint_as_float(v[cc + e]), sl2, negM));
            const float x1 = ex2(fmaf(__uint_as_float(v[cc + e + 1]), sl2, negM));
            const float x2 = ex2(fmaf(__uint_as_float(v[cc + e + 2]), sl2, negM));
            const float x3 = ex2(fmaf(__uint_as_float(v[cc + e + 3]), sl2, negM));
            const uint32_t p0 = pack_bf16(x0, x1), p1 = pack_bf16(x2, x3);
            if (kLse) {
              add2(e0, x0, x1);
              add2(e1, x2, x3);
            }
            // (the weights that PV multiplies)
            add_bf16(s0, p0);
            add_bf16(s1, p1);
            pk[e >> 1] = p0;
            pk[(e >> 1) + 1] = p1;
          }
          tmem_st16(pcol + (cc >> 1), pk);
        }
        if (mine) sum = make_float2((s0.x + s0.y) + (s1.x + s1.y), (e0.x + e0.y) + (e1.x + e1.y));
        tmem_st_wait();
      }
      tc_fence_before();
      mbar_arrive(&sm.p_full[w]);
      if (sum.x > kMost) sm.redo[r] = 1;
      // Row sums: the runs' in their order, the entries' by parity (i / c) % 2.  Shared
      // tiles alternate between the warpgroups, so each has a parity of its own;
      // behind them a tile may come to either, and both go along.
      if (d.kind == kRuns) {
        float2 run = make_float2(0.f, 0.f);
        if (g > 0 && !take(&sm.l_sum[2][r], g - 1, &run, a, abort_flag, 35)) break;
        hand_over(&sm.l_sum[2][r], g, run + sum);
      } else if (d.kind == kShared) {
        l = l + sum;
        hand_over(&sm.l_sum[p_of][r], g, l);
      } else {
        float2 own = l, other = make_float2(0.f, 0.f);
        if (g > run_tiles) {
          if (!take(&sm.l_sum[p_of ^ 1][r], g - 1, &other, a, abort_flag, 30)) break;
          if (g > own_at && !take(&sm.l_sum[p_of][r], g - 1, &own, a, abort_flag, 33)) break;
        }
        if (d.at == p_of) own = own + sum; else other = other + sum;
        hand_over(&sm.l_sum[p_of ^ 1][r], g, other);
        hand_over(&sm.l_sum[p_of][r], g, own);
      }
    }
    cp_async_wait<0>();
  }
  __syncthreads();
  if (*abort_flag) {
    // boxes still in flight land within microseconds
    for (const uint64_t t0 = global_ns(); global_ns() - t0 < 200000ull;) {}
  } else if (!idle && warp < kSoftWarps) {
    // A thread has a row and, in warpgroup w, its dims [64 w, 64 w + 64) of O.
    const int w = warp >> 2, r = (warp & 3) * 32 + lane;
    int t;
    // (a row's M is set once: whichever parity has it, the other has it or nothing)
    const float m0 = handed(&sm.m_next[0][r], &t), m1 = handed(&sm.m_next[1][r], &t);
    const float M = m0 == -INFINITY ? m1 : m0;
    const float2 l = (handed(&sm.l_sum[0][r], &t) + handed(&sm.l_sum[1][r], &t)) + handed(&sm.l_sum[2][r], &t);
    tc_fence_after();
    uint32_t x[64];
    const uint32_t ocol = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + kColO + 64 * w;
    PA_TMEM_LD_X32(ocol, x);
    PA_TMEM_LD_X32(ocol + 32, x + 32);
    tmem_ld_wait();
    if (a.c > 1) {
      // to where the key tiles were, for the ranks to join
      if (w == 0) sm.ml[r] = make_float4(M, l.x, l.y, sm.redo[r] ? 1.f : 0.f);
      uint8_t* dst = &sm.kv[0][0] + r * (kDim * 4);
#pragma unroll
      for (int e = 0; e < 64; e += 4)
        *reinterpret_cast<uint4*>(dst + ((((64 * w + e) >> 2) ^ lane) << 4)) = make_uint4(x[e], x[e + 1], x[e + 2], x[e + 3]);
    } else {
      // nothing to join
      const int u = static_cast<int>((static_cast<uint32_t>(r) * a.h_inv) >> 16);
      const bool real = r < sm.npair * a.H && sm.pair[min(u, kPairs - 1)].b >= 0;
      const bool again = real && sm.redo[r];
      const int h = r - u * a.H;
      if (real && !again) {
        const Pair& pr = sm.pair[u];
        const size_t row = (static_cast<size_t>(pr.b) * a.T + pr.t) * a.H + h;
        float sc, lse;
        finish_row(M, l, sm.sink_l2[h], &sc, &lse);
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + row * kDim + 64 * w;
#pragma unroll
        for (int e = 0; e < 64; e += 8) {
          uint4 o;
          o.x = pack_bf16(__uint_as_float(x[e]) * sc, __uint_as_float(x[e + 1]) * sc);
          o.y = pack_bf16(__uint_as_float(x[e + 2]) * sc, __uint_as_float(x[e + 3]) * sc);
          o.z = pack_bf16(__uint_as_float(x[e + 4]) * sc, __uint_as_float(x[e + 5]) * sc);
          o.w = pack_bf16(__uint_as_float(x[e + 6]) * sc, __uint_as_float(x[e + 7]) * sc);
          *reinterpret_cast<uint4*>(out + e) = o;
        }
        if (kLse && w == 0) a.lse[row] = lse;
      }
      for (uint32_t todo = w == 0 ? __ballot_sync(0xffffffffu, again) : 0u; todo; todo &= todo - 1) {
        const int rr = (warp & 3) * 32 + __ffs(todo) - 1;
        const int uu = static_cast<int>((static_cast<uint32_t>(rr) * a.h_inv) >> 16);
        row_exact(a, sm.pair[uu], rr - uu * a.H, sm.sink_l2[rr - uu * a.H]);
      }
    }
  }
  if (a.c == 1) {
    tc_fence_before();
    __syncthreads();
    if (warp == kQkWarp) {
      tc_fence_after();
      tmem_dealloc(tmem, kTmemCols);
    }
    return;
  }
  // The ranks' parts of a row meet at the rank that owns it (128 / c rows each): every
  // rank pushes 16-byte-aligned row blocks to the others (pulling them with loads
  // from distributed shared memory took three times as long).
  const int per = kTile >> a.log_c, row0 = rank * per;
  uint8_t* const parts = &sm.kv[2][0];
  if (threadIdx.x == 0) mbar_arrive_expect_tx(&sm.joined, (a.c - 1) * per * (kDim * 4 + 16));
  tc_fence_before();
  fence_proxy_async();
  cluster_arrive();
  cluster_wait();
  const bool finish = !idle && !*abort_flag;
  const int rows_all = idle ? 0 : sm.npair * a.H;
  if (finish && warp == 0 && elect_one()) {
    for (int k = 1; k < a.c; ++k) {
      const int to = (rank + k) & (a.c - 1);
      push_to_peer(peer_addr(parts + rank * (per * kDim * 4), to), &sm.kv[0][0] + to * (per * kDim * 4), per * kDim * 4,
                   peer_addr(&sm.joined, to));
      push_to_peer(peer_addr(&sm.ml_in[rank * per], to), &sm.ml[to * per], per * 16, peer_addr(&sm.joined, to));
    }
  }
  __syncwarp();
  const bool there = finish && waitw(&sm.joined, 0, a, abort_flag, 34);
  // 2 c threads a row, 4 dims of 8 c at a time; each works out for itself what its row needs
  // of the ranks' (M, l).  (A warp a row, the ranks' (M, l) by loads from their shared
  // memory and shuffles: 32 x 128 queries over 8192 entries 29.5 us for 28.7.)
  const int i_of = threadIdx.x >> (a.log_c + 1), sub = threadIdx.x & (2 * a.c - 1), r_of = row0 + i_of;
  const int u_of = static_cast<int>((static_cast<uint32_t>(min(r_of, kTile - 1)) * a.h_inv) >> 16);
  const bool real = there && warp < kSoftWarps && r_of < rows_all && sm.pair[u_of].b >= 0;
  bool again = false;
  if (real) {
    float f[8], M = -INFINITY;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (k >= a.c) break;
      f[k] = (k == rank ? sm.ml[r_of] : sm.ml_in[k * per + i_of]).x;
      M = fmaxf(M, f[k]);
    }
    float2 L = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (k >= a.c) break;
      const float4 v = k == rank ? sm.ml[r_of] : sm.ml_in[k * per + i_of];
      f[k] = f[k] == -INFINITY ? 0.f : ex2(f[k] - M);
      L.x = fmaf(f[k], v.y, L.x);
      L.y = fmaf(f[k], v.z, L.y);
      again = again || v.w != 0.f;
    }
    const int h = r_of - u_of * a.H;
    const size_t row = (static_cast<size_t>(sm.pair[u_of].b) * a.T + sm.pair[u_of].t) * a.H + h;
    float sc, lse;
    finish_row(M, L, sm.sink_l2[h], &sc, &lse);
    if (!again) {                        // (else done again below)
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + row * kDim;
      for (int x = sub; x < kDim / 4; x += 2 * a.c) {
        const uint32_t at = (x ^ (r_of & 31)) << 4;
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (k >= a.c) break;
          const uint8_t* part = k == rank ? &sm.kv[0][0] + r_of * (kDim * 4) : parts + (k * per + i_of) * (kDim * 4);
          const float4 o = *reinterpret_cast<const float4*>(part + at);
          acc[0] = fmaf(f[k], o.x, acc[0]);
          acc[1] = fmaf(f[k], o.y, acc[1]);
          acc[2] = fmaf(f[k], o.z, acc[2]);
          acc[3] = fmaf(f[k], o.w, acc[3]);
        }
        uint2 o2;
        o2.x = pack_bf16(acc[0] * sc, acc[1] * sc);
        o2.y = pack_bf16(acc[2] * sc, acc[3] * sc);
        *reinterpret_cast<uint2*>(out + x * 4) = o2;
      }
      if (kLse && sub == 0) a.lse[row] = lse;
    }
  }
  const uint32_t redo_lanes = __ballot_sync(0xffffffffu, real && again && sub == 0);
  // (a push that a peer gave up waiting for must not outlive the peer)
  if (finish && !there)
    for (const uint64_t t0 = global_ns(); global_ns() - t0 < 200000ull;) {}
  __syncwarp();
  cluster_arrive();        // peers may not leave before their parts are read
  if (warp == kQkWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  cluster_wait();
  // Rows whose weights left the range, one after the other.
  for (uint32_t todo = redo_lanes; todo; todo &= todo - 1) {
    const int r = row0 + ((warp * 32 + __ffs(todo) - 1) >> (a.log_c + 1));
    const int u = static_cast<int>((static_cast<uint32_t>(r) * a.h_inv) >> 16);
    row_exact(a, sm.pair[u], r - u * a.H, sm.sink_l2[r - u * a.H]);
  }
}

// The pool as rows of 128 bf16, in boxes of 64 dims with a 128-byte swizzle.
bool make_pool_map(CUtensorMap* m, const void* base, uint64_t rows, int box_rows) {
  static PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
  if (enc == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return false;
    enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  cuuint64_t dims[2] = {kDim, rows};
  cuuint64_t strides[1] = {kDim * 2};
  cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace pa

int launch_prefix_attn_tc(const PrefixAttnArgs& base, cudaStream_t st) {
  using namespace pa;
  Args a;
  static_cast<PrefixAttnArgs&>(a) = base;
  // (never 0, which would turn a masked -inf into NaN; 2^-126 times a logit adds nothing)
  a.scale_log2 = fmaxf(fabsf(base.tau) * 1.4426950408889634f, 1.17549435e-38f);
  a.negate = base.tau < 0.f;
  a.h_inv = (65536u + a.H - 1) / a.H;
  // TMA boxes: the largest power of two of rows (8, a swizzle atom, to a tile's 128) in a page
  a.box = a.P & -a.P;
  a.box = a.box > kTile ? kTile : a.box < 8 ? 0 : a.box;
  CUtensorMap map = {};
  if (a.N == 0) a.box = 0;
  if (a.box && !make_pool_map(&map, a.pool, static_cast<uint64_t>(a.N) * a.P, a.box)) return CSA_ERR_CUDA;
  CSA_REQUIRE(static_cast<long long>(a.N) * a.P < (1ll << 31), CSA_ERR_UNSUPPORTED);
  CSA_REQUIRE(a.W == 0 || static_cast<long long>(a.B) * a.raw_cap < (1ll << 31) - 2, CSA_ERR_UNSUPPORTED);
  // Ranks for the longest sequence that the cache can hold, three entry tiles each at
  // least: a tile takes a microsecond, a CTA's set-up and join ten.  (8 tiles of 64 heads: a
  // sequence alone 14.1 us with 4 ranks, 15.6 with 2; 100 of them, which then run at
  // once, 31.7 and 19.1.  4 tiles of 128 heads, 1 and 100: 14.5 and 30.0 us with 2,
  // 13.9 and 15.2 with one.)
  // Few heads make few jobs, so up to eight ranks; many heads make a job
  // a sequence, and four.  (32 of 16 heads, 66 tiles: 28.3 us with 4 ranks, 21.6 with 8; 32
  // of 64 heads, 18 tiles: 18.2 us with 4, 31.5 with 8, whose clusters do not all run at
  // once; 4 of 64 heads, 34 tiles: 20.0 and 17.0.)  From 128 tiles on a sequence that
  // fills them is what takes long, and many heads have eight ranks too: 1, 4 and 12
  // sequences of 128 heads over 16384 entries 26.9, 27.4 and 28.8 us (with four 40.1,
  // 40.8, 41.2), over 32768 40.5, 41.3, 45.4 (67.7, 68.3, 73.0).  Batches whose clusters
  // do not all run at once pay for it: 32 of them 85.5 us for 47.6, and 41.8 for 16.6
  // if each has but 1000 entries in use.
  const long long tiles = (static_cast<long long>(a.max_pages) * a.P + kTile - 1) / kTile;
  const int most_c = a.H > 32 && tiles < 128 ? 4 : 8;
  a.c = 1;
  while (a.c < most_c && 6 * a.c <= tiles) a.c *= 2;
  a.log_c = 31 - __builtin_clz(static_cast<unsigned>(a.c));
  // The round-up reciprocal of P for 31-bit numerators: with 2^s the power of two at or
  // above P, ceil(2^(31 + s) / P) fits 32 bits and errs by less than 2^s.
  a.p_shift = a.P > 1 ? 31 - __builtin_clz(static_cast<unsigned>(a.P - 1)) : 0;      // s - 1
  a.p_mul = a.P > 1 ? static_cast<uint32_t>(((1ull << (32 + a.p_shift)) + a.P - 1) / a.P) : 0;
  // (of a cache that cannot fill a tile only the runs that it can)
  a.tail_runs = static_cast<int>(min(8ll / a.c, (static_cast<long long>(a.max_pages) * a.P + 15) / 16));
  a.win_runs = ((a.W + 15) / 16 + a.c - 1) / a.c;
  // room for them: a power of two below 8 or a multiple of it, so that a pair's runs do
  // not straddle a tile's end (its first tile sets its rows' stabiliser)
  a.pair_runs = 1;
  while (a.pair_runs < 8 && a.pair_runs < a.tail_runs + a.win_runs) a.pair_runs *= 2;
  a.log_room = 31 - __builtin_clz(static_cast<unsigned>(a.pair_runs));
  if (a.pair_runs < a.tail_runs + a.win_runs) a.pair_runs = (a.tail_runs + a.win_runs + 7) / 8 * 8;
  int dev = 0;
  cudaGetDevice(&dev);
  const long long pairs = static_cast<long long>(a.n_seq) * a.T;
  CSA_REQUIRE(pairs < (1ll << 30), CSA_ERR_UNSUPPORTED);
  for (int u = 0; u < kPairs; ++u) {
    uint32_t off[4];
    lanes_off(off, u * a.H, u * a.H + a.H);
    a.off[u] = make_uint4(off[0], off[1], off[2], off[3]);
  }
  a.wait_ns = wait_limit_ns();
  a.hint_ns = static_cast<unsigned>(a.wait_ns < 200000ull ? a.wait_ns : 200000ull);
  const size_t smem = sizeof(Smem) + 1024;
  const auto kernel = a.lse ? prefix_attn_kernel<true> : prefix_attn_kernel<false>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.c));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // Set once per device: the kernel's shared memory; how many clusters run at once.
  static bool attr_set[2][64] = {};
  static int at_once[64][4] = {};
  const bool known = dev >= 0 && dev < 64;
  cudaError_t e;
  if (!known || !attr_set[a.lse != nullptr][dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return set_cuda_error(e);
    if (known) attr_set[a.lse != nullptr][dev] = true;
  }
  int slots = known ? at_once[dev][a.log_c] : 0;
  if (slots == 0) {
    e = cudaOccupancyMaxActiveClusters(&slots, kernel, &cfg);
    if (e != cudaSuccess) return set_cuda_error(e);
    slots = slots > 1 ? slots : 1;
    if (known) at_once[dev][a.log_c] = slots;
  }
  // Pairs a job: few, so that the jobs fill the SMs, but no more jobs than run at once, up to
  // what its rows and the set-up allow.  (A row's bits are the same in any job.  With the
  // most at all times 12 x 4 queries of 8 heads over 46 entries took 75 us for 9.2, 64
  // of 16 heads 37 for 11.0; with jobs for 148 SMs in clusters of eight, of which 15 run
  // at once, 47 x 2 queries of 16 heads in three groups 31.5 us for 20.4.)
  const int most = 128 / a.H < kPairs ? 128 / a.H : kPairs;
  a.ppt = 1;
  if (pairs > slots) {
    const long long full = slots - a.G;         // (each group may leave one job part full)
    a.ppt = full > 0 && (pairs + full - 1) / full < most ? static_cast<int>((pairs + full - 1) / full) : most;
  }
  const long long jobs = min(pairs, pairs / a.ppt + a.G);
  CSA_REQUIRE(jobs * a.c < (1ll << 31), CSA_ERR_UNSUPPORTED);
  cfg.gridDim = dim3(static_cast<unsigned>(jobs * a.c));
  e = cudaLaunchKernelEx(&cfg, kernel, a, map);
  if (e != cudaSuccess) return set_cuda_error(e);
  return check_launch();
}

}  // namespace csa
