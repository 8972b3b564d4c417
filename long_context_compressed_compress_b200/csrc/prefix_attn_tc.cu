// hca_prefix_attn_fwd in bf16 on tcgen05: attention of a batch over paged entries
// that groups of sequences share, the raw window and the sink.
//
//   l_j = tau <q, k_j>;  out = sum_j e^{l_j} k_j / (e^sigma + sum_j e^{l_j})
//
// A stream is up to 128 query rows, whole (sequence, token) pairs of H heads of
// one group, as the M side of the MMAs; thread = row in the softmax:
//   S [128 rows x 128 keys] = Q K^T   (Q and the key tile in shared memory)
//   O [128 rows x 128 dims] += P K    (P in tensor memory over S; the same tile
//                                      read with its dims as N)
// Key tiles come in three kinds:
//   shared  128 entries that every row of the CTA's streams sees, loaded once for
//           all of them;
//   own     128 entries of one pair's sequence;
//   window  8 runs of 16 raw tokens, each of one pair.
// Own and window tiles concern some rows only.  The PV MMA of such a tile writes
// those rows' lanes alone (its lane mask), so a row's sum holds its own keys
// and nothing else: an infinity or NaN in one sequence's keys cannot reach
// another's row as 0 * inf.  Keys a row must not see inside its own tiles are
// zero-filled in shared memory and get P = 0.
//
// Split.  A cluster of c CTAs shares each job (one or two streams): entry tile i
// goes to rank i % c, each window to the ranks in equal runs of 16 tokens.  The
// ranks' (O, M, l) meet in distributed shared memory, joined in rank order by
// the rank that owns the row.  c depends on the cache's capacity alone, tiles sit
// at multiples of 128 entries, and a row's rescaling depends on the row: its bits
// do not depend on the batch, the grouping or how many streams a job has.
//
// Softmax.  Exact online form with a lazy stabiliser: a row's M starts as its
// first maximum and moves (rescaling O in tensor memory) only when a later one
// exceeds it by more than 2^8, so weights stay below 2^8 and sums in fp32.
// P is rounded to bf16 for the MMA (a half step of 2^-9 a weight, of the size
// of the output's own rounding); the row sum adds the unrounded weights.
//
// Roles (12 warps): softmax warpgroup s (warps 4s .. 4s + 3) for stream s;
// producer warps 8, 9 (64 tile rows each, 16-byte asynchronous copies, so any
// page size); MMA warp 10.  With two streams one's softmax overlaps the other's
// MMAs; a single stream alternates between both S buffers.
//
// All waits are bounded in time and every thread reaches the cluster barriers.
#include "common.cuh"
#include "prefix_attn.cuh"

namespace csa {
namespace pa {

constexpr int kTile = 128, kDim = 128;
constexpr int kStages = 4;
constexpr int kTileBytes = kTile * kDim * 2;
constexpr int kRegion = kTile * 128;          // the 64-dim half of a tile
constexpr int kPairs = 16;                    // most pairs of a stream
constexpr int kProdWarps = 2, kProd0 = 8, kMmaWarp = 10;
constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;    // S buffers at 0, 128; O of stream s at 256 + 128 s
constexpr float kLazy = 8.f;                  // log2 of the growth a stabiliser lets pass

enum : int { kShared = 0, kOwn = 1, kWindow = 2, kEnd = 3 };

struct Pair {
  int b, t, n, nw;        // sequence, token; visible entries; window rows (0 .. W)
  int p;                  // position
};
struct Desc {
  int kind, stream, u, nk, seg0;   // nk: 16-key steps of the PV
};

struct __align__(1024) Smem {
  uint8_t q[2][kTileBytes];
  uint8_t kv[kStages][kTileBytes];     // reused for the streams' O (64 KB each) at the end
  uint64_t kv_full[kStages], kv_empty[kStages], q_full[2], s_full[2], p_full[2], o_done[2], drain;
  float m[2][kTile], l[2][kTile];
  uint32_t valid[kStages][4];
  Desc desc[kStages];
  int s_stage[2];
  Pair pair[2][kPairs];
  int npair[2];
  int group, tile0, shared, leader;
  uint32_t tmem;
  int abort_flag;
};

struct Args : PrefixAttnArgs {
  float scale_log2;     // |tau| log2(e)
  int negate;           // tau < 0: Q is negated on load
  int c;                // cluster size
  int ppt;              // pairs a stream
  int streams;          // per job
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
__device__ __forceinline__ bool test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
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
// K-major operand, 16-element step j; the same tile with its rows as K.
__device__ __forceinline__ uint64_t desc_kmajor(uint32_t base, int j) {
  return make_sdesc(base + (j >> 2) * kRegion + (j & 3) * 32, 16, 1024, kLayoutSw128);
}
__device__ __forceinline__ uint64_t desc_mnmajor(uint32_t base, int j) {
  return make_sdesc(base + j * 2048, kRegion, 1024, kLayoutSw128);
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

// Warp 0: the job's group and first stream tile (job = rank of this cluster among
// the groups' jobs); false when there is no such job.
__device__ bool find_job(const Args& a, int job, Smem& sm) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int g0 = 0; g0 < a.G; g0 += 32) {
    const int g = g0 + lane;
    int jobs = 0, o0 = 0;
    if (g < a.G) {
      o0 = group_start(a, g);
      const long long pairs = static_cast<long long>(max(group_start(a, g + 1) - o0, 0)) * a.T;
      const long long tiles = (pairs + a.ppt - 1) / a.ppt;
      jobs = static_cast<int>((tiles + a.streams - 1) / a.streams);
    }
    const int incl = warp_incl_scan(jobs);
    const uint32_t hit = __ballot_sync(0xffffffffu, before + incl > job);
    if (hit) {
      const int src = __ffs(hit) - 1;
      if (lane == src) {
        sm.group = g;
        sm.tile0 = (job - (before + incl - jobs)) * a.streams;
      }
      return true;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

// Warp 0: the streams' pairs, and the entries that all of them share (whole tiles).
__device__ void load_pairs(const Args& a, Smem& sm) {
  const int lane = threadIdx.x & 31, g = sm.group;
  const int o0 = group_start(a, g), npg = (group_start(a, g + 1) - o0) * a.T;
  const int lead = a.group_seq[o0];
  int least = max(a.group_shared[g], 0);
  if (lead < 0 || lead >= a.B) least = 0;
  else least = static_cast<int>(min(static_cast<long long>(least),
                                    static_cast<long long>(max(min(a.held[lead], a.max_pages), 0)) * a.P));
  for (int s = 0; s < a.streams; ++s) {
    const int first = (sm.tile0 + s) * a.ppt;
    const int np = min(max(npg - first, 0), a.ppt);
    if (lane == 0) sm.npair[s] = np;
    int n = INT32_MAX;
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
      sm.pair[s][lane] = pr;
      n = pr.n;
    }
    least = min(least, static_cast<int>(__reduce_min_sync(0xffffffffu, n)));
  }
  if (lane == 0) {
    sm.shared = least / kTile;
    sm.leader = lead;
  }
}

// ---------------------------------------------------------------- softmax
// One tile of one row: the row's weights replace S as bf16, M and l move on.
// w: which of the 128 columns the row sees (all of them when full).
__device__ __forceinline__ void softmax_tile(uint32_t scol, uint32_t ocol, const uint32_t w[4], bool full, float sl2, float& M,
                                             float& l, uint64_t* o_done, uint32_t o_phase, bool o_any, const Args& a,
                                             volatile int* abort_flag) {
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
  if (__any_sync(0xffffffffu, f != 1.f) && o_any) {
    // every PV issued so far has to be in O (the next one waits for this tile's P)
    // (inline: a call here would spill the tile's 128 values)
    for (const uint64_t t0 = global_ns(); !try_wait(o_done, o_phase, a.hint_ns);)
      if (*abort_flag || global_ns() - t0 > a.wait_ns) {
        atomicCAS(a.status, 0, CSA_ERR_TIMEOUT | (24 << 8));
        *abort_flag = 1;
        break;
      }
    __syncwarp();
    tc_fence_after();
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
    const bool some = find_job(a, job, sm);
    __syncwarp();
    if (some) load_pairs(a, sm);
    else if (lane == 0) sm.group = -1;
    if (lane == 0) sm.abort_flag = 0;
  } else if (warp == 1 && lane == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.kv_full[s], 32 * kProdWarps + kProdWarps);
      mbar_init(&sm.kv_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.q_full[s], 128);
      mbar_init(&sm.s_full[s], 2);
      mbar_init(&sm.p_full[s], 128);
      mbar_init(&sm.o_done[s], 1);
    }
    mbar_init(&sm.drain, 1);
    fence_mbar_init();
  } else if (warp == kMmaWarp) {
    tmem_alloc(&sm.tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const bool idle = sm.group < 0;      // the same in every CTA of the cluster
  const int nstream = idle ? 0 : (a.streams == 2 && sm.npair[1] > 0 ? 2 : 1);

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
      const int r0 = 64 * pw + lane;
      const int x0 = d.kind == kEnd ? -1 : src(r0), x1 = d.kind == kEnd ? -1 : src(r0 + 32);
      const uint32_t v0 = __ballot_sync(0xffffffffu, x0 >= 0), v1 = __ballot_sync(0xffffffffu, x1 >= 0);
      if (d.kind != kEnd) {
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
    auto entry = [&](int b, int key, int n) {
      if (key >= n) return -1;
      const int id = a.table[static_cast<size_t>(b) * a.max_pages + key / a.P];
      return id >= 0 && id < a.N ? id * a.P + key % a.P : -1;
    };
    for (int i = rank; ok && i < sm.shared; i += a.c)
      ok = put(Desc{kShared, 3, 0, 8, 0}, [&](int r) { return entry(sm.leader, i * kTile + r, INT32_MAX); });
    for (int s = 0; s < nstream && ok; ++s) {
      for (int u = 0; u < sm.npair[s] && ok; ++u) {
        const Pair pr = sm.pair[s][u];
        // the first tile of this rank behind the shared ones
        int i = sm.shared + (rank - sm.shared % a.c + a.c) % a.c;
        for (; ok && i * kTile < pr.n; i += a.c)
          ok = put(Desc{kOwn, 1 << s, u, (min(kTile, pr.n - i * kTile) + 15) / 16, 0},
                   [&](int r) { return entry(pr.b, i * kTile + r, pr.n); });
      }
      const int segs = a.win_run / 16;
      if (rank * a.win_run < a.W) {
        for (int k0 = 0; ok && k0 < sm.npair[s] * segs; k0 += 8)
          ok = put(Desc{kWindow, 1 << s, 0, min(8, sm.npair[s] * segs - k0), k0}, [&](int r) {
            const int sg = k0 + (r >> 4), u = sg / segs;
            if (u >= sm.npair[s]) return -1;
            const Pair pr = sm.pair[s][u];
            const int in_run = (sg % segs) * 16 + (r & 15);
            const int back = rank * a.win_run + in_run;      // tokens before the query's own
            if (back >= pr.nw) return -1;
            return pr.b * a.raw_cap + (pr.p - back) % a.raw_cap;
          });
      }
    }
    if (ok) put(Desc{kEnd, 3, 0, 0, 0}, [](int) { return -1; });
    cp_async_wait<0>();
  } else if (!idle && warp == kMmaWarp) {
    // ================================================================= MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc_qk = idesc_bf16(128, 128, 0, 0);
      constexpr uint32_t idesc_pv = idesc_bf16(128, 128, 0, 1);
      int gq[2] = {0, 0};           // next tile of each stream's QK
      int nq[2] = {0, 0}, np[2] = {0, 0};
      int pend[2][2] = {{0, 0}, {0, 0}};   // stages of the QKs whose PV is to come
      bool fin[2] = {false, nstream < 2};
      uint32_t done = 0;            // streams through with each stage (2 bits a stage)
      const uint32_t all = nstream == 2 ? 3u : 1u;
      const int ahead = nstream == 2 ? 1 : 2;
      bool q_ok[2] = {false, false};
      auto through = [&](int stage, int s) {
        done |= (1u << s) << (2 * stage);
        if (((done >> (2 * stage)) & 3u) == all) {
          tc_commit(&sm.kv_empty[stage]);
          done &= ~(3u << (2 * stage));
        }
      };
      uint64_t t_last = global_ns();
      while (true) {
        bool did = false, left = false;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (s >= nstream) continue;
          if (np[s] < nq[s]) {
            left = true;
            const int buf = nstream == 2 ? s : (np[s] & 1);
            const int use = nstream == 2 ? np[s] : (np[s] >> 1);
            if (test_wait(&sm.p_full[buf], use & 1)) {
              tc_fence_after();
              const int stage = pend[s][np[s] & 1];
              const Desc d = sm.desc[stage];
              const uint32_t kb = smem_u32(sm.kv[stage]);
              const uint32_t pcol = tmem + kColS + 128 * buf, ocol = tmem + kColO + 128 * s;
              if (d.kind == kWindow) {
                const int segs = a.win_run / 16;
                for (int j = 0; j < d.nk; ++j) {
                  const int u = (d.seg0 + j) / segs;
                  uint32_t off[4];
                  lanes_off(off, u * a.H, u * a.H + a.H);
                  mma_ts_lanes(ocol, pcol + 8 * j, desc_mnmajor(kb, j), idesc_pv, off);
                }
              } else {
                uint32_t off[4];
                lanes_off(off, d.kind == kOwn ? d.u * a.H : 0, d.kind == kOwn ? d.u * a.H + a.H : 128);
                for (int j = 0; j < d.nk; ++j)
                  mma_ts_lanes(ocol, pcol + 8 * j, desc_mnmajor(kb, j), idesc_pv, off);
              }
              tc_commit(&sm.o_done[s]);
              through(stage, s);
              ++np[s];
              did = true;
            }
          }
          if (!fin[s]) {
            left = true;
            if (nq[s] - np[s] < ahead) {
              const int stage = gq[s] % kStages;
              if (!q_ok[s]) q_ok[s] = test_wait(&sm.q_full[s], 0);
              if (q_ok[s] && test_wait(&sm.kv_full[stage], (gq[s] / kStages) & 1)) {
                const Desc d = sm.desc[stage];
                const int buf = nstream == 2 ? s : (nq[s] & 1);
                if (d.kind == kEnd) {
                  sm.s_stage[buf] = -1;
                  mbar_arrive(&sm.s_full[buf]);
                  mbar_arrive(&sm.s_full[buf]);
                  fin[s] = true;
                } else if (!(d.stream & (1 << s))) {
                  through(stage, s);
                  ++gq[s];
                } else {
                  fence_proxy_async();
                  tc_fence_after();
                  const uint32_t qb = smem_u32(sm.q[s]), kb = smem_u32(sm.kv[stage]);
#pragma unroll
                  for (int j = 0; j < kDim / 16; ++j)
                    mma_bf16(tmem + kColS + 128 * buf, desc_kmajor(qb, j), desc_kmajor(kb, j), idesc_qk, j > 0);
                  sm.s_stage[buf] = stage;
                  tc_commit(&sm.s_full[buf]);
                  mbar_arrive(&sm.s_full[buf]);
                  pend[s][nq[s] & 1] = stage;
                  ++nq[s];
                  ++gq[s];
                }
                did = true;
              }
            }
          }
        }
        if (!left) break;
        if (did) {
          t_last = global_ns();
        } else {
          if (*abort_flag) break;
          __nanosleep(20);
          if (global_ns() - t_last > a.wait_ns) {
            atomicCAS(a.status, 0, CSA_ERR_TIMEOUT | (21 << 8));
            *abort_flag = 1;
            break;
          }
        }
      }
      // whatever was issued has finished before tensor memory is released
      tc_commit(&sm.drain);
      drain_wait(&sm.drain, 0);
    }
    __syncwarp();
  } else if (!idle && warp < kProd0 && (warp >> 2) < nstream) {
    // ================================================================= softmax
    const int s = warp >> 2, tid = threadIdx.x & 127;
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ocol = tmem + lane_addr + kColO + 128 * s;
    const int rows = sm.npair[s] * a.H;
    {
      // Q: 16 lanes a row; rows beyond the stream's are zero
      const int c = tid & 15;
      const uint32_t flip = a.negate ? 0x80008000u : 0u;
#pragma unroll 4
      for (int r = tid >> 4; r < kTile; r += 8) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows) {
          const int u = r / a.H;
          const Pair pr = sm.pair[s][u];
          if (pr.b >= 0)
            x = *reinterpret_cast<const uint4*>(
                static_cast<const __nv_bfloat16*>(a.q) +
                ((static_cast<size_t>(pr.b) * a.T + pr.t) * a.H + (r - u * a.H)) * kDim + c * 8);
        }
        x.x ^= flip; x.y ^= flip; x.z ^= flip; x.w ^= flip;
        *reinterpret_cast<uint4*>(sm.q[s] + (c >> 3) * kRegion + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = x;
      }
      fence_proxy_async();
      mbar_arrive(&sm.q_full[s]);
    }
    {
      uint32_t z[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) z[e] = 0u;
#pragma unroll
      for (int cc = 0; cc < kDim; cc += 16) tmem_st16(ocol + cc, z);
      tmem_st_wait();
      tc_fence_before();
    }
    const int r = (warp & 3) * 32 + lane;
    const int u = r < rows ? r / a.H : -1;
    const int segs = max(a.win_run / 16, 1);
    float M = -INFINITY, l = 0.f;
    int k = 0;
    while (true) {
      const int buf = nstream == 2 ? s : (k & 1), use = nstream == 2 ? k : (k >> 1);
      if (!waitw(&sm.s_full[buf], use & 1, a, abort_flag, 22)) break;
      tc_fence_after();
      const int stage = sm.s_stage[buf];
      if (stage < 0) break;
      const Desc d = sm.desc[stage];
      uint32_t w[4];
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
        w[i] = sm.valid[stage][i];
        full = full && w[i] == 0xffffffffu;
        const int x = min(max(lo - 32 * i, 0), 32), y = min(max(hi - 32 * i, 0), 32);
        const uint32_t by = y >= 32 ? 0xffffffffu : (1u << y) - 1u, bx = x >= 32 ? 0xffffffffu : (1u << x) - 1u;
        w[i] = mine ? w[i] & by & ~bx : 0u;
      }
      if (__any_sync(0xffffffffu, mine)) {
        const uint32_t scol = tmem + lane_addr + kColS + 128 * buf;
        softmax_tile(scol, ocol, w, full, a.scale_log2, M, l, &sm.o_done[s], (k - 1) & 1, k > 0, a, abort_flag);
      }
      tc_fence_before();
      mbar_arrive(&sm.p_full[buf]);
      ++k;
    }
    if (k > 0) waitw(&sm.o_done[s], (k - 1) & 1, a, abort_flag, 23);
    tc_fence_after();
    sm.m[s][r] = M;
    sm.l[s][r] = l;
  }
  // The streams' O go where the key tiles were, once nothing reads those.
  __syncthreads();
  if (!idle && warp < kProd0 && (warp >> 2) < nstream) {
    const int s = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t ocol = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + kColO + 128 * s;
    uint8_t* dst = &sm.kv[0][0] + s * (kTile * kDim * 4) + r * (kDim * 4);
#pragma unroll
    for (int cc = 0; cc < kDim; cc += 32) {
      uint32_t v[32];
      PA_TMEM_LD_X32(ocol + cc, v);
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 8; ++e)
        *reinterpret_cast<uint4*>(dst + (((cc / 4 + e) ^ lane) << 4)) =
            make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
    }
  }
  tc_fence_before();
  cluster_sync_all();
  if (!idle && !*abort_flag) {
    // Each rank finishes every c-th row: a warp a row, a lane 4 dims.
    for (int i = rank + a.c * warp; i < nstream * kTile; i += a.c * (kThreads / 32)) {
      const int s = i / kTile, r = i % kTile;
      const int u = r / a.H;
      if (u >= sm.npair[s]) continue;
      const Pair pr = sm.pair[s][u];
      if (pr.b < 0) continue;
      float mi = -INFINITY, li = 0.f;
      if (lane < a.c) {
        mi = ld_peer(peer_addr(&sm.m[s][r], lane));
        li = ld_peer(peer_addr(&sm.l[s][r], lane));
      }
      float M = mi;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      const float fi = M > -INFINITY ? ex2(mi - M) : 0.f;
      const float* orow = reinterpret_cast<const float*>(&sm.kv[0][0] + s * (kTile * kDim * 4) + r * (kDim * 4) +
                                                         ((lane ^ (r & 31)) << 4));
      float L = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
      for (int k = 0; k < a.c; ++k) {
        const float f = __shfl_sync(0xffffffffu, fi, k), lk = __shfl_sync(0xffffffffu, li, k);
        const float4 o = ld_peer4(peer_addr(orow, k));
        if (f == 0.f) continue;          // this rank saw none of the row's keys
        L = fmaf(f, lk, L);
        acc[0] = fmaf(f, o.x, acc[0]);
        acc[1] = fmaf(f, o.y, acc[1]);
        acc[2] = fmaf(f, o.z, acc[2]);
        acc[3] = fmaf(f, o.w, acc[3]);
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
  if (warp == kMmaWarp) {
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
  CSA_REQUIRE(static_cast<long long>(a.N) * a.P < (1ll << 31), CSA_ERR_UNSUPPORTED);
  CSA_REQUIRE(a.W == 0 || static_cast<long long>(a.B) * a.raw_cap < (1ll << 31), CSA_ERR_UNSUPPORTED);
  a.ppt = 128 / a.H < kPairs ? 128 / a.H : kPairs;
  // Ranks for the longest sequence the cache can hold, two entry tiles each at least.
  const long long tiles = (static_cast<long long>(a.max_pages) * a.P + kTile - 1) / kTile;
  a.c = tiles <= 2 ? 1 : tiles <= 4 ? 2 : tiles <= 8 ? 4 : 8;
  a.win_run = ((a.W + a.c - 1) / a.c + 15) / 16 * 16;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const long long pairs = static_cast<long long>(a.n_seq) * a.T;
  CSA_REQUIRE(pairs < (1ll << 30), CSA_ERR_UNSUPPORTED);
  const long long most = pairs / a.ppt + a.G;       // streams, at most
  // Two streams share a job's key tiles and overlap each other's softmax and MMAs;
  // one each while that leaves every cluster its own SMs.
  a.streams = most * a.c > sms ? 2 : 1;
  const long long jobs = a.streams == 2 ? pairs / (2 * a.ppt) + a.G : most;
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
