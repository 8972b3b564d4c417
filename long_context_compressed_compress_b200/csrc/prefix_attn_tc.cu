// hca_prefix_attn_fwd in bf16 on tcgen05: attention of a batch over paged entries
// that groups of sequences share, the raw window and the sink.
//
//   l_j = tau <q, k_j>;  out = sum_j e^{l_j} k_j / (e^sigma + sum_j e^{l_j})
//
// A job is up to 128 query rows, whole (sequence, token) pairs of H heads of one
// group, as the M side of the MMAs; thread = row in the softmax:
//   S [128 rows x 128 keys] = Q K^T   (Q and the key tile in shared memory)
//   O [128 rows x 128 dims] += P K    (P in tensor memory over S; the same tile
//                                      read with its dims as N)
// Key tiles come in three kinds:
//   shared  128 entries that every row of the job sees, loaded once for all;
//   own     128 entries of one pair's sequence;
//   window  8 runs of 16 raw tokens, each of one pair.
// Own and window tiles concern some rows only.  The PV MMA of such a tile writes
// those rows' lanes alone (its lane mask), so a row's sum holds its own keys
// and nothing else: an infinity or NaN in one sequence's keys cannot reach
// another's row as 0 * inf.  Keys a row must not see inside its own tiles are
// zero-filled in shared memory and get P = 0.
//
// Split.  A cluster of c CTAs shares each job: entry tile i goes to rank i % c, each
// window in equal runs of 16 tokens to all ranks.  The ranks' (O, M, l) meet in
// distributed shared memory, in rank order, each rank finishing every c-th row.
// c depends on the cache's capacity alone, tiles sit at multiples of 128 entries,
// and a row's rescaling depends on the row: its bits do not depend on batch or
// grouping.
//
// Softmax.  Exact online form with a lazy stabiliser: a row's M starts as its
// first maximum and moves (rescaling O in tensor memory) only when a later one
// exceeds it by more than 2^8, so weights stay below 2^8 and sums in fp32.
// P is rounded to bf16 for the MMA (a half step of 2^-9 a weight, of the size
// of the output's own rounding); the row sum adds the unrounded weights.
//
// Roles (12 warps).  Softmax warpgroups 0 and 1 (warps 0 - 3, 4 - 7) take the even
// and the odd tiles, with S and P buffers of their own and one O; they hand each
// row's M from tile to tile.  Producer warps 8, 9 (64 tile rows each): whole
// tiles by TMA boxes of a page (or its largest power of two of rows), the others
// by 16-byte asynchronous copies.  Warp 10 issues QK (a warpgroup's next as soon
// as it has read the last S), warp 11 PV.
//
// All waits are bounded in time and every thread reaches the cluster barriers.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstdlib>
#include "common.cuh"
#include "prefix_attn.cuh"

namespace csa {
namespace pa {

constexpr int kTile = 128, kDim = 128;
constexpr int kStages = 5;                    // a tile lives ~6700 cycles: load, QK, softmax, PV
constexpr int kTileBytes = kTile * kDim * 2;
constexpr int kRegion = kTile * 128;          // the 64-dim half of a tile
constexpr int kMaxCluster = 8;
constexpr int kPairs = 16;                    // most pairs of a job
constexpr int kProdWarps = 2, kProd0 = 8, kQkWarp = 10, kPvWarp = 11;
constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColP = 256, kColO = 384;   // S, P of warpgroup w at 128 w, 256 + 64 w
constexpr float kLazy = 8.f;                  // log2 of the growth a stabiliser lets pass

enum : int { kShared = 0, kOwn = 1, kWindow = 2, kEnd = 3 };

struct Pair {
  int b, t, n, nw;        // sequence, token; visible entries; window rows (0 .. W)
  int p;                  // position
};
struct Desc {
  int kind, u, nk, seg0;  // nk: 16-key steps of the PV
};

struct __align__(1024) Smem {
  uint8_t q[kTileBytes];
  uint8_t kv[kStages][kTileBytes];     // the first half is reused for the CTA's O (64 KB) at the end
  uint64_t kv_full[kStages], kv_empty[kStages], q_full, s_full[2], s_free[2], p_full[2], pv_done[2];
  uint64_t drain[2];
  unsigned long long m_next[2][kTile], l_next[2][kTile];   // (tile, value) on its way between the warpgroups
  float m[kTile], l[kTile];            // the CTA's, at the end
  uint32_t valid[kStages][4];
  Desc desc[kStages];
  int s_stage[2];
  float sink_l2[kTile];                // by head
  Pair pair[kPairs];
  int npair;
  int group, tile, shared, leader;
  uint32_t tmem;
  int abort_flag;
};

struct Args : PrefixAttnArgs {
  float scale_log2;     // |tau| log2(e)
  int negate;           // tau < 0: Q is negated on load
  int box;              // rows of a page chunk that a TMA box brings (0: pages too odd)
  uint32_t h_inv;       // ceil(2^16 / H): r / H = r h_inv >> 16 for r < 128
  int c;                // cluster size
  int ppt;              // pairs a job
  int win_run;          // window tokens a rank takes of each pair (a multiple of 16)
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
// Bounded wait of a warp for its rows' values of `tile`.
__device__ __forceinline__ bool take(const unsigned long long* slot, int tile, float* x, const Args& a,
                                     volatile int* abort_flag, int site) {
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
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// (a0, a1) * b + c on the packed fp32 pipe
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b, float c) {
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %4};\n\tmov.b64 rc, {%5, %5};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b), "f"(c));
}
__device__ __forceinline__ void add2(float& x0, float& x1, float y0, float y1) {
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%0, %1};\n\tmov.b64 rb, {%2, %3};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(y0), "f"(y1));
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

#define PA_TMEM_LD_X8(taddr, r)                                                                           \
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"                   \
               : "=r"((r)[0]), "=r"((r)[1]), "=r"((r)[2]), "=r"((r)[3]), "=r"((r)[4]), "=r"((r)[5]),      \
                 "=r"((r)[6]), "=r"((r)[7])                                                               \
               : "r"(taddr))
#define PA_TMEM_ST_X8(taddr, r)                                                                           \
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),      \
               "r"((r)[0]), "r"((r)[1]), "r"((r)[2]), "r"((r)[3]), "r"((r)[4]), "r"((r)[5]), "r"((r)[6]), \
               "r"((r)[7])                                                                                \
               : "memory")

// D[tmem] += A[tmem] * B[smem]; lanes whose bit is set in `off` are not written.
__device__ __forceinline__ void mma_ts_lanes(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             const uint32_t off[4]) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, 1, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%4, %5, %6, %7}, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3])
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
__device__ __forceinline__ void lanes_off(uint32_t off[4], int lo, int hi) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int a = min(max(lo - 32 * i, 0), 32), b = min(max(hi - 32 * i, 0), 32);
    const uint32_t below_b = b >= 32 ? 0xffffffffu : (1u << b) - 1u;
    const uint32_t below_a = a >= 32 ? 0xffffffffu : (1u << a) - 1u;
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
__device__ __forceinline__ float ld_peer(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_peer4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// ----------------------------------------------------------------- set-up
// Where group g's members start (kept within the list).
__device__ __forceinline__ int group_start(const Args& a, int g) {
  if (a.G == 1) return g * a.n_seq;
  return min(max(a.group_off[g], 0), a.n_seq);
}

// Warp 0: the job's group and tile of pairs (jobs are numbered group by group); false
// when there is no such job.
__device__ bool find_job(const Args& a, int job, Smem& sm, int* start, int* count) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int g0 = 0; g0 < a.G; g0 += 32) {
    const int g = g0 + lane;
    int jobs = 0, o0 = 0, n = 0;
    if (g < a.G) {
      o0 = group_start(a, g);
      n = max(group_start(a, g + 1) - o0, 0);
      jobs = static_cast<int>((static_cast<long long>(n) * a.T + a.ppt - 1) / a.ppt);
    }
    const int incl = warp_incl_scan(jobs);
    const uint32_t hit = __ballot_sync(0xffffffffu, before + incl > job);
    if (hit) {
      const int src = __ffs(hit) - 1;
      if (lane == src) {
        sm.group = g;
        sm.tile = job - (before + incl - jobs);
      }
      *start = __shfl_sync(0xffffffffu, o0, src);
      *count = __shfl_sync(0xffffffffu, n, src);
      __syncwarp();
      return true;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

// Warp 0: the job's pairs, and the entries that all of them share (whole tiles).
__device__ void load_pairs(const Args& a, Smem& sm, int o0, int members) {
  const int lane = threadIdx.x & 31;
  const int first = sm.tile * a.ppt;
  const int np = min(members * a.T - first, a.ppt);
  const int lead = a.group_seq[o0];
  int n = max(a.group_shared[sm.group], 0);
  if (lane < np) {
    Pair pr{-1, 0, 0, 0, -1};
    const int i = first + lane;
    const int b = a.group_seq[o0 + i / a.T];
    if (b >= 0 && b < a.B) {
      pr.b = b;
      pr.t = i % a.T;
      const long long p = static_cast<long long>(a.q_pos0[b]) + pr.t;
      pr.p = static_cast<int>(min(p, static_cast<long long>(INT32_MAX)));
      pr.n = visible_entries(a, b, p);
      pr.nw = p < 0 ? 0 : static_cast<int>(min(static_cast<long long>(a.W), p + 1));
    } else {
      atomicCAS(a.status, 0, CSA_ERR_INVALID_ARG | (4 << 8));
    }
    sm.pair[lane] = pr;
    n = min(n, pr.n);
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
    sm.leader = lead;
  }
}

__global__ void __launch_bounds__(kThreads, 1) prefix_attn_kernel(const __grid_constant__ Args a,
                                                                  const __grid_constant__ CUtensorMap pool_map) {
  extern __shared__ __align__(1024) uint8_t pa_smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(pa_smem_raw) + 1023) &
                                      ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &sm.abort_flag;
  const int rank = static_cast<int>(cluster_rank());
  const int job = blockIdx.x / a.c;

  if (warp == 0) {
    int start, members;
    const bool some = find_job(a, job, sm, &start, &members);
    if (some) load_pairs(a, sm, start, members);
    else if (lane == 0) sm.group = -1;
  } else if (warp == 1 && lane == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.kv_full[s], 32 * kProdWarps + kProdWarps);
      mbar_init(&sm.kv_empty[s], 1);
    }
    mbar_init(&sm.q_full, 256);
    for (int w = 0; w < 2; ++w) {
      mbar_init(&sm.s_full[w], 2);
      mbar_init(&sm.s_free[w], 128);
      mbar_init(&sm.p_full[w], 128);
      mbar_init(&sm.pv_done[w], 1);
      mbar_init(&sm.drain[w], 1);
    }
    sm.abort_flag = 0;
    fence_mbar_init();
  } else if (warp < 6) {
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

  if (!idle && warp >= kProd0 && warp < kProd0 + kProdWarps) {
    // ================================================================= producers
    const int pw = warp - kProd0, half = lane >> 4, c = lane & 15;
    const __nv_bfloat16* pool = static_cast<const __nv_bfloat16*>(a.pool) + c * 8;
    const __nv_bfloat16* ring = static_cast<const __nv_bfloat16*>(a.kv_raw) + c * 8;
    int g = 0;
    bool ok = true;
    int armed[kStages];                // last use of each stage by TMA
#pragma unroll
    for (int s = 0; s < kStages; ++s) armed[s] = -1;
    // Entry `key` of sequence b as a row of the pool, or -1.
    auto entry = [&](int b, int key, int n) {
      if (key >= n) return -1;
      const int id = a.table[static_cast<size_t>(b) * a.max_pages + key / a.P];
      return id >= 0 && id < a.N ? id * a.P + key % a.P : -1;
    };
    auto announce = [&](int stage, const Desc& d, uint32_t v0, uint32_t v1) {
      sm.valid[stage][2 * pw] = v0;
      sm.valid[stage][2 * pw + 1] = v1;
      if (pw == 0) sm.desc[stage] = d;
    };
    // One tile, row by row: src(r) gives the row of the pool (or ring) for tile row r, or -1.
    auto put = [&](const Desc& d, auto&& src) {
      const int stage = g % kStages, use = g / kStages;
      const bool data = d.kind != kEnd;
      const int r0 = 64 * pw + lane;
      const int x0 = data ? src(r0) : -1, x1 = data ? src(r0 + 32) : -1;
      const uint32_t v0 = __ballot_sync(0xffffffffu, x0 >= 0), v1 = __ballot_sync(0xffffffffu, x1 >= 0);
      if (use >= 1 && !waitw(&sm.kv_empty[stage], (use - 1) & 1, a, abort_flag, 20)) return false;
      if (data) {
        const __nv_bfloat16* base = d.kind == kWindow ? ring : pool;
        const uint32_t dbase = smem_u32(sm.kv[stage]) + (c >> 3) * kRegion + (64 * pw + half) * 128;
        const uint32_t cx = static_cast<uint32_t>((c & 7) ^ half);
#pragma unroll 8
        for (int j = 0; j < 32; ++j) {
          const int x = __shfl_sync(0xffffffffu, j < 16 ? x0 : x1, (2 * j + half) & 31);
          const uint32_t dst = dbase + j * 256 + ((cx ^ static_cast<uint32_t>((2 * j) & 7)) << 4);
          cp_async16(dst, base + static_cast<size_t>(max(x, 0)) * kDim, x >= 0 ? 16u : 0u);
        }
      }
      cp_async_mbar_arrive(&sm.kv_full[stage]);
      if (lane == 0) {
        announce(stage, d, v0, v1);
        mbar_arrive(&sm.kv_full[stage]);
      }
      ++g;
      return true;
    };
    // This rank's entry tiles i, i + c, .. of sequence b below n: by TMA where all
    // 128 entries are there, else row by row.  The page chunks of the next 32 /
    // boxes tiles are looked up at once, a lane each (one tile at a time, the
    // lookup's latency alone would pace the loop at 2000 cycles a tile).
    const int boxes = a.box ? 64 / a.box : 32;         // of this warp's 64 rows
    const int ahead = 32 / boxes;
    auto put_tiles = [&](int kind, int u, int b, int i, int n) {
      int rows = -1;
      for (int k = 0; ok && static_cast<long long>(i) * kTile < n; i += a.c, k = k + 1 == ahead ? 0 : k + 1) {
        const int key0 = i * kTile;
        const Desc d{kind, u, (min(kTile, n - key0) + 15) / 16, 0};
        if (a.box && k == 0) {
          const long long key = (i + static_cast<long long>(lane / boxes) * a.c) * kTile + 64 * pw + (lane % boxes) * a.box;
          rows = key < n ? entry(b, static_cast<int>(key), n) : -1;
        }
        const int y = __shfl_sync(0xffffffffu, rows, k * boxes + lane % boxes);
        if (!a.box || key0 + kTile > n || __any_sync(0xffffffffu, y < 0)) {
          ok = put(d, [&](int r) { return entry(b, key0 + r, n); });
          continue;
        }
        const int stage = g % kStages, use = g / kStages;
        if (use >= 1 && !waitw(&sm.kv_empty[stage], (use - 1) & 1, a, abort_flag, 20)) { ok = false; break; }
        if (lane == 0) {
          announce(stage, d, 0xffffffffu, 0xffffffffu);
          mbar_arrive_expect_tx(&sm.kv_full[stage], 64 * kDim * 2);
        }
        __syncwarp();
        if (lane < 2 * boxes) {                        // lanes [0, boxes): dims 0 .. 63, the next: 64 .. 127
          const int h = lane >= boxes ? 1 : 0;
          tma_load_2d(smem_u32(sm.kv[stage]) + h * kRegion + (64 * pw + (lane - h * boxes) * a.box) * 128,
                      reinterpret_cast<uint64_t>(&pool_map), 64 * h, y, &sm.kv_full[stage]);
        }
        mbar_arrive(&sm.kv_full[stage]);
#pragma unroll
        for (int s = 0; s < kStages; ++s)
          if (s == stage) armed[s] = use;
        ++g;
      }
    };
    put_tiles(kShared, 0, sm.leader, rank, sm.shared * kTile);
    // the first tile of this rank behind the shared ones
    const int own0 = sm.shared + (rank - sm.shared % a.c + a.c) % a.c;
    for (int u = 0; u < sm.npair && ok; ++u) put_tiles(kOwn, u, sm.pair[u].b, own0, sm.pair[u].n);
    const int segs = a.win_run / 16;
    if (rank * a.win_run < a.W) {
      for (int k0 = 0; ok && k0 < sm.npair * segs; k0 += 8)
        ok = put(Desc{kWindow, 0, min(8, sm.npair * segs - k0), k0}, [&](int r) {
          const int sg = k0 + (r >> 4), u = sg / segs;
          if (u >= sm.npair) return -1;
          const Pair pr = sm.pair[u];
          // how many tokens before the query's own
          const int back = rank * a.win_run + (sg - u * segs) * 16 + (r & 15);
          return back < pr.nw ? pr.b * a.raw_cap + (pr.p - back) % a.raw_cap : -1;
        });
    }
    if (ok) put(Desc{kEnd, 0, 0, 0}, [](int) { return -1; });
    cp_async_wait<0>();
    if (*abort_flag) {
      // boxes still in flight land within microseconds
#pragma unroll
      for (int s = 0; s < kStages; ++s)
        if (armed[s] >= 0) drain_wait(&sm.kv_full[s], armed[s] & 1);
    }
  } else if (!idle && warp == kQkWarp) {
    // ================================================================= S = Q K^T
    constexpr uint32_t idesc_qk = idesc_bf16(128, 128, 0, 0);
    const uint32_t qb = smem_u32(sm.q);
    bool ok = waitw(&sm.q_full, 0, a, abort_flag, 21), more = true;
    int ends = 0;
    for (int g = 0; ok; ++g) {
      const int stage = g % kStages, w = g & 1;
      if (more) {
        ok = waitw(&sm.kv_full[stage], (g / kStages) & 1, a, abort_flag, 25);
        if (!ok) break;
        more = sm.desc[stage].kind != kEnd;
      }
      ok = g < 2 || waitw(&sm.s_free[w], ((g >> 1) - 1) & 1, a, abort_flag, 27);
      if (!ok) break;
      if (!more) {                 // the end, told to both warpgroups
        if (elect_one()) {
          sm.s_stage[w] = -1;
          mbar_arrive(&sm.s_full[w]);
          mbar_arrive(&sm.s_full[w]);
        }
        __syncwarp();
        if (++ends == 2) break;
        continue;
      }
      fence_proxy_async();
      tc_fence_after();
      const uint32_t kb = smem_u32(sm.kv[stage]), scol = tmem + kColS + 128 * w;
      if (elect_one()) {
#pragma unroll
        for (int j = 0; j < kDim / 16; ++j)
          mma_bf16(scol, desc_kmajor(qb, j), desc_kmajor(kb, j), idesc_qk, j > 0);
        tc_commit(&sm.s_full[w]);
        sm.s_stage[w] = stage;
        mbar_arrive(&sm.s_full[w]);
      }
      __syncwarp();
    }
    if (elect_one()) {
      tc_commit(&sm.drain[0]);
      drain_wait(&sm.drain[0], 0);
    }
    __syncwarp();
  } else if (!idle && warp == kPvWarp) {
    // ================================================================= O += P K
    constexpr uint32_t idesc_pv = idesc_bf16(128, 128, 0, 1);
    const int segs = max(a.win_run / 16, 1);
    const uint32_t ocol = tmem + kColO;
    for (int g = 0;; ++g) {
      const int stage = g % kStages, w = g & 1;
      if (!waitw(&sm.kv_full[stage], (g / kStages) & 1, a, abort_flag, 28)) break;
      const Desc d = sm.desc[stage];
      if (d.kind == kEnd) break;
      if (!waitw(&sm.p_full[w], (g >> 1) & 1, a, abort_flag, 26)) break;
      fence_proxy_async();
      tc_fence_after();
      const uint32_t kb = smem_u32(sm.kv[stage]), pcol = tmem + kColP + 64 * w;
      if (d.kind == kShared) {
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < kTile / 16; ++j) mma_ts(ocol, pcol + 8 * j, desc_mnmajor(kb, j), idesc_pv);
          tc_commit(&sm.kv_empty[stage]);
          tc_commit(&sm.pv_done[w]);
        }
      } else if (elect_one()) {
        int u = d.kind == kWindow ? d.seg0 / segs : d.u;
        int left = d.kind == kWindow ? segs - d.seg0 % segs : kTile;
        uint32_t off[4];
        lanes_off(off, u * a.H, u * a.H + a.H);
        for (int j = 0; j < d.nk; ++j) {
          mma_ts_lanes(ocol, pcol + 8 * j, desc_mnmajor(kb, j), idesc_pv, off);
          if (--left == 0) {        // the next run is the next pair's
            ++u;
            left = segs;
            lanes_off(off, u * a.H, u * a.H + a.H);
          }
        }
        tc_commit(&sm.kv_empty[stage]);
        tc_commit(&sm.pv_done[w]);
      }
      __syncwarp();
    }
    // whatever was issued has finished before O is read and tensor memory released
    if (elect_one()) {
      tc_commit(&sm.drain[1]);
      drain_wait(&sm.drain[1], 0);
    }
    __syncwarp();
  } else if (!idle && warp < kProd0) {
    // ================================================================= softmax, tiles g % 2 == w
    const int w = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t scol = tmem + lane_addr + kColS + 128 * w, pcol = tmem + lane_addr + kColP + 64 * w;
    const uint32_t ocol = tmem + lane_addr + kColO;
    const int rows = sm.npair * a.H;
    {
      // Q: 16 lanes a row; rows beyond the job's are zero
      const int c = threadIdx.x & 15;
      const uint32_t dst = smem_u32(sm.q) + (c >> 3) * kRegion;
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + c * 8;
#pragma unroll
      for (int i = 0; i < kTile / 16; ++i) {
        const int x = (threadIdx.x >> 4) + 16 * i;
        const int ux = static_cast<int>((static_cast<uint32_t>(x) * a.h_inv) >> 16);
        size_t row = 0;
        bool some = x < rows;
        if (some) {
          const int b = sm.pair[ux].b;
          some = b >= 0;
          row = (static_cast<size_t>(max(b, 0)) * a.T + sm.pair[ux].t) * a.H + (x - ux * a.H);
        }
        cp_async16(dst + x * 128 + (((c & 7) ^ (x & 7)) << 4), q + row * kDim, some ? 16u : 0u);
      }
      cp_async_commit();
      uint32_t z[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) z[e] = 0u;
#pragma unroll
      for (int cc = 0; cc < 64; cc += 16) tmem_st16(ocol + 64 * w + cc, z);
      tmem_st_wait();
      tc_fence_before();
      cp_async_wait<0>();
      if (a.negate) {
        for (int i = 0; i < kTile / 16; ++i) {
          const int x = (threadIdx.x >> 4) + 16 * i;
          uint4* v = reinterpret_cast<uint4*>(sm.q + (c >> 3) * kRegion + x * 128 + (((c & 7) ^ (x & 7)) << 4));
          *v = make_uint4(v->x ^ 0x80008000u, v->y ^ 0x80008000u, v->z ^ 0x80008000u, v->w ^ 0x80008000u);
        }
      }
      hand_over(&sm.m_next[w][r], -1, -INFINITY);
      hand_over(&sm.l_next[w][r], -1, 0.f);
      fence_proxy_async();
      mbar_arrive(&sm.q_full);
    }
    const int u = r < rows ? static_cast<int>((static_cast<uint32_t>(r) * a.h_inv) >> 16) : -1;
    const int segs = max(a.win_run / 16, 1);
    const float sl2 = a.scale_log2;
    for (int g = w;; g += 2) {
      const int k = g >> 1;
      if (!waitw(&sm.s_full[w], k & 1, a, abort_flag, 22)) break;
      tc_fence_after();
      // S is on its way to registers while the tile's kind is looked up
      uint32_t v[128];
      PA_TMEM_LD_X32(scol, v);
      PA_TMEM_LD_X32(scol + 32, v + 32);
      PA_TMEM_LD_X32(scol + 64, v + 64);
      PA_TMEM_LD_X32(scol + 96, v + 96);
      const int stage = sm.s_stage[w];
      const Desc d = sm.desc[max(stage, 0)];
      uint32_t see[4];
      bool mine = d.kind == kShared;       // the tile's MMA writes this row's lane
      int lo = 0, hi = kTile;
      if (d.kind == kOwn) {
        mine = u == d.u;
      } else if (d.kind == kWindow) {
        lo = min(max(u * segs - d.seg0, 0), 8) * 16;
        hi = min(max((u + 1) * segs - d.seg0, 0), 8) * 16;
        mine = u >= 0 && hi > lo;
      }
      bool full = d.kind != kWindow;       // every row that counts sees every column
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        see[i] = sm.valid[max(stage, 0)][i];
        full = full && see[i] == 0xffffffffu;
      }
      const bool any = __any_sync(0xffffffffu, mine);
      tmem_ld_wait();
      if (stage < 0) break;
      tc_fence_before();
      mbar_arrive(&sm.s_free[w]);
      float mx = -INFINITY;
      if (any) {
        if (!full) {
          uint32_t off[4];
          lanes_off(off, lo, hi);
#pragma unroll
          for (int i = 0; i < 4; ++i) see[i] = mine ? see[i] & ~off[i] : 0u;
#pragma unroll
          for (int e = 0; e < 128; ++e)
            if (!((see[e >> 5] >> (e & 31)) & 1u)) v[e] = 0xff800000u;   // -inf: weight 0
        }
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 128; e += 2) mx4[(e >> 1) & 3] = max3(mx4[(e >> 1) & 3], __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
        mx = max3(max3(mx4[0], mx4[1], mx4[2]), mx4[3], -INFINITY) * sl2;   // NaN if there is one
        if (!mine) mx = -INFINITY;
      }
      // M as the tile before left it, then as this one does
      float Mp = -INFINITY;
      if (g > 0 && !take(&sm.m_next[w ^ 1][r], g - 1, &Mp, a, abort_flag, 23)) break;
      const bool move = Mp > -INFINITY && mx > Mp + kLazy;
      const float Mn = Mp == -INFINITY || move ? fmaxf(mx, Mp) : Mp;
      hand_over(&sm.m_next[w][r], g, Mn);
      if (__any_sync(0xffffffffu, move)) {
        // O moves to the new M: behind the PV of the tile before, ahead of this one's
        if (!waitw(&sm.pv_done[w ^ 1], ((g - 1) >> 1) & 1, a, abort_flag, 24)) break;
        tc_fence_after();
        const float f = move ? ex2(Mp - Mn) : 1.f;
#pragma unroll 1
        for (int cc = 0; cc < kDim; cc += 8) {
          uint32_t o[8];
          PA_TMEM_LD_X8(ocol + cc, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
          PA_TMEM_ST_X8(ocol + cc, o);
        }
        tmem_st_wait();
      }
      // P's buffer is free once the PV two tiles back has read it
      if (g >= 2 && !waitw(&sm.pv_done[w], (k - 1) & 1, a, abort_flag, 29)) break;
      tc_fence_after();
      float sum = 0.f;
      if (any) {
        const float negM = Mn > -INFINITY ? -Mn : 0.f;
        float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
        for (int cc = 0; cc < 128; cc += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float x0, x1;
            fma2(x0, x1, __uint_as_float(v[cc + e]), __uint_as_float(v[cc + e + 1]), sl2, negM);
            x0 = ex2(x0);
            x1 = ex2(x1);
            if (e & 2) add2(s0, s1, x0, x1);
            else add2(s2, s3, x0, x1);
            pk[e >> 1] = pack_bf16(x0, x1);
          }
          tmem_st16(pcol + (cc >> 1), pk);
        }
        sum = mine ? (s0 + s1) + (s2 + s3) : 0.f;
        tmem_st_wait();
      }
      tc_fence_before();
      mbar_arrive(&sm.p_full[w]);
      // l goes from tile to tile as M does, in the order of the tiles
      float l = 0.f;
      if (g > 0 && !take(&sm.l_next[w ^ 1][r], g - 1, &l, a, abort_flag, 30)) break;
      if (Mp != Mn) l *= ex2(Mp - Mn);
      hand_over(&sm.l_next[w][r], g, l + sum);
    }
  }
  __syncthreads();
  if (!idle && warp < kProd0) {
    // The last tile's M and l hold for O.  Warpgroup w moves dims [64 w, 64 w + 64) of
    // O to where the key tiles were.
    const int w = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t ocol = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + kColO + 64 * w;
    if (w == 0) {
      int t0, t1, t2;
      const float m0 = handed(&sm.m_next[0][r], &t0), m1 = handed(&sm.m_next[1][r], &t1);
      sm.m[r] = t1 > t0 ? m1 : m0;
      sm.l[r] = handed(&sm.l_next[t1 > t0 ? 1 : 0][r], &t2);
    }
    uint8_t* dst = &sm.kv[0][0] + r * (kDim * 4);
    tc_fence_after();
    uint32_t x[64];
    PA_TMEM_LD_X32(ocol, x);
    PA_TMEM_LD_X32(ocol + 32, x + 32);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 64; e += 4)
      *reinterpret_cast<uint4*>(dst + ((((64 * w + e) >> 2) ^ lane) << 4)) = make_uint4(x[e], x[e + 1], x[e + 2], x[e + 3]);
  }
  tc_fence_before();
  cluster_arrive();
  cluster_wait();
  // Each rank finishes every c-th row: a warp a row, a lane 4 dims.  Three rows' parts
  // from every rank are on their way before the first is used.
  constexpr int kFly = 3;
  const bool finish = !idle && !*abort_flag;
  const int step = a.c * (kThreads / 32), rows_all = idle ? 0 : sm.npair * a.H;
  for (int r0 = rank + a.c * warp; finish && r0 < rows_all; r0 += kFly * step) {
    float4 o[kFly][kMaxCluster];
    float mi[kFly], li[kFly];
#pragma unroll
    for (int x = 0; x < kFly; ++x) {
      const int r = min(r0 + x * step, rows_all - 1);
      const float* orow = reinterpret_cast<const float*>(&sm.kv[0][0] + r * (kDim * 4) + ((lane ^ (r & 31)) << 4));
      mi[x] = -INFINITY;
      li[x] = 0.f;
      if (lane < a.c) {
        mi[x] = ld_peer(peer_addr(&sm.m[r], lane));
        li[x] = ld_peer(peer_addr(&sm.l[r], lane));
      }
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k)
        if (k < a.c) o[x][k] = ld_peer4(peer_addr(orow, k));
    }
#pragma unroll
    for (int x = 0; x < kFly; ++x) {
      const int r = r0 + x * step;
      const int u = static_cast<int>((static_cast<uint32_t>(r) * a.h_inv) >> 16);
      if (r >= rows_all) continue;
      const Pair pr = sm.pair[u];
      if (pr.b < 0) continue;
      float M = mi[x];
#pragma unroll
      for (int y = 4; y > 0; y >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, y));
      M = __shfl_sync(0xffffffffu, M, 0);
      const float fi = mi[x] > -INFINITY ? ex2(mi[x] - M) : 0.f;
      float L = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) {
        if (k >= a.c) break;
        const float f = __shfl_sync(0xffffffffu, fi, k), lk = __shfl_sync(0xffffffffu, li[x], k);
        L = fmaf(f, lk, L);
        acc[0] = fmaf(f, o[x][k].x, acc[0]);
        acc[1] = fmaf(f, o[x][k].y, acc[1]);
        acc[2] = fmaf(f, o[x][k].z, acc[2]);
        acc[3] = fmaf(f, o[x][k].w, acc[3]);
      }
      const int h = r - u * a.H;
      const size_t row = (static_cast<size_t>(pr.b) * a.T + pr.t) * a.H + h;
      float sc = 0.f, lse = -INFINITY;
      if (L != 0.f) {
        const float sg = sm.sink_l2[h];
        const float X = fmaxf(M, sg), fm = ex2(M - X);
        sc = __fdiv_rn(fm, fmaf(L, fm, ex2(sg - X)));
        lse = (M + log2f(L)) * 0.6931471805599453f;
      }
      uint2 o2;
      o2.x = pack_bf16(acc[0] * sc, acc[1] * sc);
      o2.y = pack_bf16(acc[2] * sc, acc[3] * sc);
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row * kDim + lane * 4) = o2;
      if (a.lse && lane == 0) a.lse[row] = lse;
    }
  }
  __syncwarp();
  cluster_arrive();        // peers may not leave before their rows are read
  if (warp == kQkWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  cluster_wait();
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
  // TMA boxes: the largest power of two of rows (8, a swizzle atom, to a warp's 64) in a page
  a.box = a.P & -a.P;
  a.box = a.box > 64 ? 64 : a.box < 8 ? 0 : a.box;
  CUtensorMap map = {};
  if (a.N == 0) a.box = 0;
  if (a.box && !make_pool_map(&map, a.pool, static_cast<uint64_t>(a.N) * a.P, a.box)) return CSA_ERR_CUDA;
  CSA_REQUIRE(static_cast<long long>(a.N) * a.P < (1ll << 31), CSA_ERR_UNSUPPORTED);
  CSA_REQUIRE(a.W == 0 || static_cast<long long>(a.B) * a.raw_cap < (1ll << 31), CSA_ERR_UNSUPPORTED);
  a.ppt = 128 / a.H < kPairs ? 128 / a.H : kPairs;
  // Ranks for the longest sequence that the cache can hold.
  const long long tiles = (static_cast<long long>(a.max_pages) * a.P + kTile - 1) / kTile;
  a.c = tiles < 8 ? 1 : tiles < 16 ? 2 : tiles < 128 ? 4 : 8;
  if (const char* e = getenv("PA_C")) a.c = atoi(e);
  a.win_run = ((a.W + a.c - 1) / a.c + 15) / 16 * 16;
  int dev = 0;
  cudaGetDevice(&dev);
  const long long pairs = static_cast<long long>(a.n_seq) * a.T;
  CSA_REQUIRE(pairs < (1ll << 30), CSA_ERR_UNSUPPORTED);
  const long long jobs = pairs / a.ppt + a.G;       // at most: each group may leave one part full
  CSA_REQUIRE(jobs * a.c < (1ll << 31), CSA_ERR_UNSUPPORTED);
  a.wait_ns = wait_limit_ns();
  a.hint_ns = static_cast<unsigned>(a.wait_ns < 200000ull ? a.wait_ns : 200000ull);
  const size_t smem = sizeof(Smem) + 1024;
  static bool attr_set[64] = {};
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(prefix_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return set_cuda_error(e);
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(jobs * a.c));
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, prefix_attn_kernel, a, map);
  if (e != cudaSuccess) return set_cuda_error(e);
  return check_launch();
}

}  // namespace csa
