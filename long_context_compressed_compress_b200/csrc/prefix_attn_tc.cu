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
// Split.  A cluster of c CTAs shares each job, and two halves (softmax
// warpgroup, S and O of their own) share a CTA: entry tile i goes to rank i % c,
// half (i / c) % 2; each window in equal runs of 16 tokens to the ranks' second
// halves.  The halves join in tensor memory, the ranks in distributed shared
// memory, in rank order, each rank finishing every c-th row.  c depends on
// the cache's capacity alone, tiles sit at multiples of 128 entries, and a row's
// rescaling depends on the row: its bits do not depend on batch or grouping.
//
// Softmax.  Exact online form with a lazy stabiliser: a row's M starts as its
// first maximum and moves (rescaling O in tensor memory) only when a later one
// exceeds it by more than 2^8, so weights stay below 2^8 and sums in fp32.
// P is rounded to bf16 for the MMA (a half step of 2^-9 a weight, of the size
// of the output's own rounding); the row sum adds the unrounded weights.
//
// Roles (12 warps): softmax warpgroup w for half w (warps 4w .. 4w + 3); producer
// warps 8, 9 (64 tile rows each, 16-byte asynchronous copies, so any page
// size); MMA warps 10, 11, one a half: one half's softmax overlaps the other's
// MMAs.  Tile slots alternate between the halves; a slot the order leaves over
// is skipped.
//
// All waits are bounded in time and every thread reaches the cluster barriers.
#include <cstdlib>
#include "common.cuh"
#include "prefix_attn.cuh"

namespace csa {
namespace pa {

constexpr int kTile = 128, kDim = 128;
constexpr int kStages = 4;
constexpr int kTileBytes = kTile * kDim * 2;
constexpr int kRegion = kTile * 128;          // the 64-dim half of a tile
constexpr int kMaxCluster = 8;
constexpr int kPairs = 16;                    // most pairs of a job
constexpr int kProdWarps = 2, kProd0 = 8, kMma0 = 10;
constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;    // S of half w at 128 w, O at 256 + 128 w
constexpr float kLazy = 8.f;                  // log2 of the growth a stabiliser lets pass

enum : int { kShared = 0, kOwn = 1, kWindow = 2, kSkip = 3, kEnd = 4 };

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
  uint64_t kv_full[kStages], kv_empty[kStages], q_full, s_full[2], p_full[2], drain[2];
  float m[2][kTile], l[2][kTile];      // the halves', then [0] the CTA's
  uint32_t valid[kStages][4];
  Desc desc[kStages];
  int s_stage[2];
  Pair pair[kPairs];
  int npair;
  int group, tile, shared, leader;
  uint32_t tmem;
  int abort_flag;
};

struct Args : PrefixAttnArgs {
  float scale_log2;     // |tau| log2(e)
  int negate;           // tau < 0: Q is negated on load
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
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
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
__device__ __forceinline__ int group_start(const Args& a, int g) { return min(max(a.group_off[g], 0), a.n_seq); }

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

// ---------------------------------------------------------------- softmax
// One tile of one row: the row's weights replace S as bf16, M and l move on.
// w: which of the 128 columns the row sees (all of them when full).
__device__ __forceinline__ void softmax_tile(uint32_t scol, uint32_t ocol, const uint32_t w[4], bool full, float sl2, float& M,
                                             float& l) {
  uint32_t v[128];
  auto load_s = [&]() {
    PA_TMEM_LD_X32(scol, v);
    PA_TMEM_LD_X32(scol + 32, v + 32);
    PA_TMEM_LD_X32(scol + 64, v + 64);
    PA_TMEM_LD_X32(scol + 96, v + 96);
    tmem_ld_wait();
    if (!full) {
#pragma unroll
      for (int e = 0; e < 128; ++e)
        if (!((w[e >> 5] >> (e & 31)) & 1u)) v[e] = 0xff800000u;   // -inf: weight 0
    }
  };
  load_s();
  float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int e = 0; e < 128; ++e) mx4[e & 3] = fmaxf(mx4[e & 3], __uint_as_float(v[e]));
  float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
  mx *= sl2;
  float f = 1.f;
  if (M == -INFINITY) {
    M = mx;                        // nothing summed yet (O and l are 0)
  } else if (mx > M + kLazy) {
    f = ex2(M - mx);
    M = mx;
  }
  if (__any_sync(0xffffffffu, f != 1.f)) {
    // (S came behind the last PV: O is at rest)
    l *= f;
#pragma unroll
    for (int cc = 0; cc < kDim; cc += 16) {
      uint32_t o[16];
      tmem_ld16(ocol + cc, o);
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
      tmem_st16(ocol + cc, o);
    }
    load_s();                      // (again, rather than held over this rare branch)
  }
  const float negM = M > -INFINITY ? -M : 0.f;
  float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
  for (int cc = 0; cc < 128; cc += 32) {
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      float x0, x1;
      fma2(x0, x1, __uint_as_float(v[cc + e]), __uint_as_float(v[cc + e + 1]), sl2, negM);
      float p0 = ex2(x0), p1 = ex2(x1);
      if (e & 2) add2(s0, s1, p0, p1);
      else add2(s2, s3, p0, p1);
      pk[e >> 1] = pack_bf16(p0, p1);
    }
    tmem_st16(scol + (cc >> 1), pk);
  }
  l += (s0 + s1) + (s2 + s3);
  tmem_st_wait();
}

__global__ void __launch_bounds__(kThreads, 1) prefix_attn_kernel(const __grid_constant__ Args a) {
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
      mbar_init(&sm.p_full[w], 128);
      mbar_init(&sm.drain[w], 1);
    }
    sm.abort_flag = 0;
    fence_mbar_init();
  } else if (warp == kMma0) {
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
    // One tile: src(r) gives the row of the pool (or ring) for tile row r, or -1.
    auto put = [&](const Desc& d, auto&& src) {
      const int stage = g % kStages, use = g / kStages;
      if (use >= 1 && !waitw(&sm.kv_empty[stage], (use - 1) & 1, a, abort_flag, 20)) return false;
      const bool data = d.kind < kSkip;
      const int r0 = 64 * pw + lane;
      const int x0 = data ? src(r0) : -1, x1 = data ? src(r0 + 32) : -1;
      const uint32_t v0 = __ballot_sync(0xffffffffu, x0 >= 0), v1 = __ballot_sync(0xffffffffu, x1 >= 0);
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
        sm.valid[stage][2 * pw] = v0;
        sm.valid[stage][2 * pw + 1] = v1;
        if (pw == 0) sm.desc[stage] = d;
        mbar_arrive(&sm.kv_full[stage]);
      }
      ++g;
      return true;
    };
    auto nothing = [](int) { return -1; };
    // The next slot belongs to half w.
    auto turn = [&](int w) { return (g & 1) == w || put(Desc{kSkip, 0, 0, 0}, nothing); };
    auto entry = [&](int b, int key, int n) {
      if (key >= n) return -1;
      const int id = a.table[static_cast<size_t>(b) * a.max_pages + key / a.P];
      return id >= 0 && id < a.N ? id * a.P + key % a.P : -1;
    };
    for (int i = rank; ok && i < sm.shared; i += a.c)
      ok = put(Desc{kShared, 0, 8, 0}, [&](int r) { return entry(sm.leader, i * kTile + r, INT32_MAX); });
    // the first tile of this rank behind the shared ones
    const int own0 = sm.shared + (rank - sm.shared % a.c + a.c) % a.c;
    for (int u = 0; u < sm.npair && ok; ++u) {
      const Pair pr = sm.pair[u];
      for (int i = own0; ok && i * kTile < pr.n; i += a.c)
        ok = turn((i / a.c) & 1) && put(Desc{kOwn, u, (min(kTile, pr.n - i * kTile) + 15) / 16, 0},
                                        [&](int r) { return entry(pr.b, i * kTile + r, pr.n); });
    }
    const int segs = a.win_run / 16;
    if (rank * a.win_run < a.W) {
      for (int k0 = 0; ok && k0 < sm.npair * segs; k0 += 8)
        ok = turn(1) && put(Desc{kWindow, 0, min(8, sm.npair * segs - k0), k0}, [&](int r) {
               const int sg = k0 + (r >> 4), u = sg / segs;
               if (u >= sm.npair) return -1;
               const Pair pr = sm.pair[u];
               // how many tokens before the query's own
               const int back = rank * a.win_run + (sg - u * segs) * 16 + (r & 15);
               return back < pr.nw ? pr.b * a.raw_cap + (pr.p - back) % a.raw_cap : -1;
             });
    }
    ok = ok && put(Desc{kEnd, 0, 0, 0}, nothing) && put(Desc{kEnd, 0, 0, 0}, nothing);
    cp_async_wait<0>();
  } else if (!idle && warp >= kMma0) {
    // ================================================================= MMA issuer of half w
    constexpr uint32_t idesc_qk = idesc_bf16(128, 128, 0, 0);
    constexpr uint32_t idesc_pv = idesc_bf16(128, 128, 0, 1);
    const int w = warp - kMma0;
    const int segs = max(a.win_run / 16, 1);
    const uint32_t scol = tmem + kColS + 128 * w, ocol = tmem + kColO + 128 * w;
    const uint32_t qb = smem_u32(sm.q);
    int k = 0;                      // tiles of this half
    bool ok = waitw(&sm.q_full, 0, a, abort_flag, 21);
    for (int g = w; ok; g += 2) {
      const int stage = g % kStages;
      ok = waitw(&sm.kv_full[stage], (g / kStages) & 1, a, abort_flag, 25);
      if (!ok) break;
      const Desc d = sm.desc[stage];
      if (d.kind == kEnd) break;
      if (d.kind == kSkip) {
        if (elect_one()) mbar_arrive(&sm.kv_empty[stage]);
        __syncwarp();
        continue;
      }
      fence_proxy_async();
      tc_fence_after();
      const uint32_t kb = smem_u32(sm.kv[stage]);
      if (elect_one()) {
#pragma unroll
        for (int j = 0; j < kDim / 16; ++j)
          mma_bf16(scol, desc_kmajor(qb, j), desc_kmajor(kb, j), idesc_qk, j > 0);
        tc_commit(&sm.s_full[w]);
        sm.s_stage[w] = stage;
        mbar_arrive(&sm.s_full[w]);
      }
      __syncwarp();
      ok = waitw(&sm.p_full[w], k & 1, a, abort_flag, 26);
      if (!ok) break;
      tc_fence_after();
      if (d.kind == kShared) {
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < kTile / 16; ++j) mma_ts(ocol, scol + 8 * j, desc_mnmajor(kb, j), idesc_pv);
          tc_commit(&sm.kv_empty[stage]);
        }
      } else if (elect_one()) {
        int u = d.kind == kWindow ? d.seg0 / segs : d.u;
        int left = d.kind == kWindow ? segs - d.seg0 % segs : kTile;
        uint32_t off[4];
        lanes_off(off, u * a.H, u * a.H + a.H);
        for (int j = 0; j < d.nk; ++j) {
          mma_ts_lanes(ocol, scol + 8 * j, desc_mnmajor(kb, j), idesc_pv, off);
          if (--left == 0) {        // the next run is the next pair's
            ++u;
            left = segs;
            lanes_off(off, u * a.H, u * a.H + a.H);
          }
        }
        tc_commit(&sm.kv_empty[stage]);
      }
      __syncwarp();
      ++k;
    }
    // The end: behind the last PV.  Whatever was issued has finished before tensor
    // memory is released.
    if (elect_one()) {
      if (ok) {
        tc_commit(&sm.s_full[w]);
        sm.s_stage[w] = -1;
        mbar_arrive(&sm.s_full[w]);
      }
      tc_commit(&sm.drain[w]);
      drain_wait(&sm.drain[w], 0);
    }
    __syncwarp();
  } else if (!idle && warp < kProd0) {
    // ================================================================= softmax of half w
    const int w = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t scol = tmem + lane_addr + kColS + 128 * w, ocol = tmem + lane_addr + kColO + 128 * w;
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
      for (int cc = 0; cc < kDim; cc += 16) tmem_st16(ocol + cc, z);
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
      fence_proxy_async();
      mbar_arrive(&sm.q_full);
    }
    const int u = r < rows ? static_cast<int>((static_cast<uint32_t>(r) * a.h_inv) >> 16) : -1;
    const int segs = max(a.win_run / 16, 1);
    float M = -INFINITY, l = 0.f;
    for (int k = 0;; ++k) {
      if (!waitw(&sm.s_full[w], k & 1, a, abort_flag, 22)) break;
      tc_fence_after();
      const int stage = sm.s_stage[w];
      if (stage < 0) break;
      const Desc d = sm.desc[stage];
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
      bool full = d.kind == kShared;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        see[i] = sm.valid[stage][i];
        full = full && see[i] == 0xffffffffu;
      }
      if (!full) {
        uint32_t off[4];
        lanes_off(off, lo, hi);
#pragma unroll
        for (int i = 0; i < 4; ++i) see[i] = mine ? see[i] & ~off[i] : 0u;
      }
      if (__any_sync(0xffffffffu, mine)) softmax_tile(scol, ocol, see, full, a.scale_log2, M, l);
      tc_fence_before();
      mbar_arrive(&sm.p_full[w]);
    }
    sm.m[w][r] = M;
    sm.l[w][r] = l;
  }
  __syncthreads();
  if (!idle && warp < kProd0) {
    // The halves join where both can be read, in tensor memory: half w takes dims
    // [64 w, 64 w + 64).  The CTA's O goes where the key tiles were.
    const int w = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t ocol = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + kColO + 64 * w;
    const float m0 = sm.m[0][r], m1 = sm.m[1][r], l0 = sm.l[0][r], l1 = sm.l[1][r];
    const float M = fmaxf(m0, m1);
    const float f0 = m0 > -INFINITY ? ex2(m0 - M) : 0.f, f1 = m1 > -INFINITY ? ex2(m1 - M) : 0.f;
    uint8_t* dst = &sm.kv[0][0] + r * (kDim * 4);
    tc_fence_after();
#pragma unroll
    for (int cc = 0; cc < 64; cc += 32) {
      uint32_t x[32], y[32];
      PA_TMEM_LD_X32(ocol + cc, x);
      PA_TMEM_LD_X32(ocol + 128 + cc, y);
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 32; e += 4) {
        float o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o[i] = fmaf(__uint_as_float(y[e + i]), f1, __uint_as_float(x[e + i]) * f0);
        *reinterpret_cast<float4*>(dst + ((((64 * w + cc + e) >> 2) ^ lane) << 4)) = make_float4(o[0], o[1], o[2], o[3]);
      }
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");    // both halves have read the other's M and l
    if (w == 0) {
      sm.m[0][r] = M;
      sm.l[0][r] = fmaf(l1, f1, l0 * f0);
    }
  }
  tc_fence_before();
  cluster_sync_all();
  if (!idle && !*abort_flag) {
    // Each rank finishes every c-th row: a warp a row, a lane 4 dims.
    for (int r = rank + a.c * warp; r < kTile; r += a.c * (kThreads / 32)) {
      const int u = static_cast<int>((static_cast<uint32_t>(r) * a.h_inv) >> 16);
      if (u >= sm.npair) continue;
      const Pair pr = sm.pair[u];
      if (pr.b < 0) continue;
      const float* orow = reinterpret_cast<const float*>(&sm.kv[0][0] + r * (kDim * 4) + ((lane ^ (r & 31)) << 4));
      // every rank's part is on its way before the first is used
      float4 o[kMaxCluster];
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k)
        if (k < a.c) o[k] = ld_peer4(peer_addr(orow, k));
      float mi = -INFINITY, li = 0.f;
      if (lane < a.c) {
        mi = ld_peer(peer_addr(&sm.m[0][r], lane));
        li = ld_peer(peer_addr(&sm.l[0][r], lane));
      }
      float M = mi;
#pragma unroll
      for (int x = 4; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
      M = __shfl_sync(0xffffffffu, M, 0);
      const float fi = mi > -INFINITY ? ex2(mi - M) : 0.f;
      float L = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) {
        if (k >= a.c) break;
        const float f = __shfl_sync(0xffffffffu, fi, k), lk = __shfl_sync(0xffffffffu, li, k);
        L = fmaf(f, lk, L);
        acc[0] = fmaf(f, o[k].x, acc[0]);
        acc[1] = fmaf(f, o[k].y, acc[1]);
        acc[2] = fmaf(f, o[k].z, acc[2]);
        acc[3] = fmaf(f, o[k].w, acc[3]);
      }
      const int h = r - u * a.H;
      const size_t row = (static_cast<size_t>(pr.b) * a.T + pr.t) * a.H + h;
      float sc = 0.f, lse = -INFINITY;
      if (L != 0.f) {
        const float sg = a.sink ? a.sink[h] * 1.4426950408889634f : -INFINITY;
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
  cluster_sync_all();      // peers have read this CTA's rows
  if (warp == kMma0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
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
  CSA_REQUIRE(static_cast<long long>(a.N) * a.P < (1ll << 31), CSA_ERR_UNSUPPORTED);
  CSA_REQUIRE(a.W == 0 || static_cast<long long>(a.B) * a.raw_cap < (1ll << 31), CSA_ERR_UNSUPPORTED);
  a.ppt = 128 / a.H < kPairs ? 128 / a.H : kPairs;
  // Ranks for the longest sequence that the cache can hold.
  const long long tiles = (static_cast<long long>(a.max_pages) * a.P + kTile - 1) / kTile;
  a.c = tiles < 8 ? 1 : tiles < 16 ? 2 : tiles < 32 ? 4 : 8;
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, prefix_attn_kernel, a);
  if (e != cudaSuccess) return set_cuda_error(e);
  return check_launch();
}

}  // namespace csa
