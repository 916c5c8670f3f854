// Shared-KV attention over the compressed cache on sm_100a (include/kvc.h,
// shared_kv_attention and shared_kv_attention_topk).
//
// What it computes, per query t and head h over the query's rows s (listed or visible cache
// entries, then its window), with K_s = [nope_s / fp8_scale ; rope_s] both key and value:
//     x_s = scale q[t,h].K_s,  out[t,h] = sum_s exp(x_s) K_s / D,  D = sum_s exp(x_s) (+ sink)
// in one pass over the rows with the running maximum and sum of the softmax.
//
// One query's heads share every row, so a query is a pair of GEMMs with the heads on M:
// S = Q K^T [128 heads x 64 rows] and O += P K [128 heads x c].  At 128 heads that is 455
// flop per cache byte, above the 246 the machine has per byte: the tensor cores bound it; at
// 64 heads and below HBM does.
//
// Split.  O for 128 heads x 512 channels in fp32 is all of an SM's TMEM, so a cluster of two
// CTAs takes a query, each with half of the channels: it gathers, widens and holds only its
// half of every row, as key and as value alike.  Each CTA's MMA gives the half-sum of S over
// its channels; the CTAs push their halves into each other's shared memory (st.async on an
// mbarrier) and both take the softmax of the sum.  TMEM: O 256 columns, two S buffers of
// 128; the weights P overwrite the S they came from and are the MMA's A operand from there.
//
// Types.  An E4M3 byte is exact in fp16, and a bf16 query row is exact in fp16 once scaled by
// a power of two (its largest value to 2^15: what is lost lies 2^-40 below it), so the FP8
// channels run as fp16 MMAs with the weights rounded to fp16 (2^-11); the bf16 channels keep
// bf16 for its exponent range, with weights rounded to bf16 (2^-8).  The two parts have
// accumulators of their own (S_n, S_r), because only S_n carries the row's power of two and
// 1 / fp8_scale.  Both parts accumulate in fp32.
//
// Roles (17 working warps): warps 0-3 and 4-7 are two softmax groups taking alternate 64-row tiles (a
// thread is a head), warps 8-15 gather the rows (global memory -> registers -> widened,
// swizzled shared memory, two tiles in flight), warp 16 issues the MMAs.  A persistent grid
// walks segments (query, row tiles); a query's tiles are split among clusters when there are
// too few queries, and a second kernel joins the parts in a fixed order.
#include <cuda_fp16.h>

#include "kvc_common.cuh"
#include "kvc_host.h"
#include "kvc_launch.h"
#include "tc_ptx.cuh"

namespace kvc {

// bit 0: a bounded wait gave up; bit 1: a query's rows or a listed entry out of range.
__device__ unsigned int g_attention_error = 0;

namespace attn {

using namespace tcx;

constexpr int kRows = 64;         // rows of a tile (MMA N of S, K of P K)
constexpr int kHeads = 128;       // heads of an item (MMA M, TMEM lanes)
constexpr int kStages = 3;        // row-tile ring
constexpr int kSoftWarps = 8;     // two groups of four
constexpr int kLoadWarps = 8;
constexpr int kMmaWarp = kSoftWarps + kLoadWarps;
constexpr int kThreads = 32 * (kMmaWarp + 4);  // whole warpgroups for setmaxnreg
// Registers a thread: 96 at launch (640 threads); a softmax thread holds a head's 64 scores,
// a gather thread two tiles' loads, the MMA thread little.
constexpr int kSoftRegs = 144, kLoadRegs = 80, kMmaRegs = 24;
static_assert(128 * (2 * kSoftRegs + 2 * kLoadRegs + kMmaRegs) <= kThreads * 96, "register split");
constexpr int kMaxAtoms = 4;      // 64-channel blocks per CTA
constexpr int kQAtom = kHeads * 128;      // one [128 heads x 64] 16-bit block, 16 KB
constexpr int kKAtom = kRows * 128;       // one [64 rows x 64] block, 8 KB
constexpr int kStage = kMaxAtoms * kKAtom;
constexpr int kXBuf = kHeads * kRows * 4; // the peer's half of S, fp32
constexpr uint32_t kWaitLimitNs = 2000000000u;  // of a 32-bit timer
// Weights are exp2(x - m + kBias): with m at most kSlack below the running maximum they stay
// below 2^15 in fp16 and vanish only 2^-31 below the maximum.
constexpr float kBias = 7.f;
constexpr float kSlack = 8.f;

// Shared memory (bytes).
constexpr int kSmQ = 0;
constexpr int kSmK = kSmQ + kMaxAtoms * kQAtom;
constexpr int kSmX = kSmK + kStages * kStage;
constexpr int kSmBars = kSmX + 2 * kXBuf;
constexpr int kNumBars = 2 * kStages + 2 + 2 + 2 + 2 + 2 + 2 + 1 + 4 + 4 + 1;
constexpr int kSmMask = kSmBars + kNumBars * 8;      // u8 [kStages][8]
constexpr int kSmMisc = kSmMask + kStages * 8;       // tmem address, abort flag
constexpr int kSmExp = kSmMisc + 8;                  // u8 [4][kHeads] exponents of Q rows
constexpr int kSmM = kSmExp + 4 * kHeads;            // f32 [kHeads] running maximum
constexpr int kSmL = kSmM + kHeads * 4;              // f32 [2][kHeads] row sums
constexpr int kSmem = kSmL + 2 * kHeads * 4;
static_assert(kSmem <= 227 * 1024, "attention shared memory");
// TMEM columns
constexpr int kColS = 256;        // S buffer b at kColS + 128 b: S_n 64, S_r 64 columns
constexpr int kColR = 64;

struct Args {
  AttentionProblem p;
  int64_t items, units;     // (query, head group); units = items x tiles_per_item
  int tiles_per_item, groups, clusters, atoms;  // atoms: 64-channel blocks per CTA
  int cn, cnp;              // FP8 channels, padded to whole blocks
  bool strided;             // whole items, cluster by cluster (no splits)
  float* part_o;            // [clusters][2][kHeads][c] fp32
  float2* part_ml;          // [clusters][2][kHeads] (m, l)
};

// The rows of query t.
struct Query {
  int64_t key_start, win_start, n_visible;
  int n1, n2;  // cache rows, window rows
  bool ok;
};
__device__ __forceinline__ Query query_of(const AttentionProblem& a, int64_t t) {
  Query q;
  q.key_start = a.key_start[t];
  q.n_visible = a.n_visible[t];
  q.win_start = a.win_start ? a.win_start[t] : 0;
  const int64_t n2 = a.win_start ? a.win_len[t] : 0;
  const int64_t n1 = a.idx ? (q.n_visible < a.k ? q.n_visible : a.k) : q.n_visible;
  q.ok = q.n_visible >= 0 && (a.idx || q.n_visible <= a.max_visible) && q.key_start >= 0 &&
         q.key_start <= a.cache_rows - q.n_visible && n2 >= 0 && n2 <= a.max_win &&
         (n2 == 0 || (q.win_start >= 0 && q.win_start <= a.win_rows - n2));
  q.n1 = q.ok ? static_cast<int>(n1) : 0;
  q.n2 = q.ok ? static_cast<int>(n2) : 0;
  return q;
}

// The segments of one cluster, in order.  Every role walks the same ones.
struct Walker {
  const Args& a;
  int64_t at, end;  // items (strided) or units
  // the current segment
  int64_t t;
  int hg, j0, j1, part;  // tiles [j0, j1) of the query; part: -1 whole, else partial slot
  Query q;

  __device__ Walker(const Args& args, int cid) : a(args) {
    if (a.strided) {
      at = cid;
      end = a.items;
    } else {
      at = cid * a.units / a.clusters;
      end = (cid + 1) * a.units / a.clusters;
    }
  }
  __device__ __forceinline__ bool next() {
    if (at >= end) return false;
    int64_t item;
    int f0, f1;
    const int tpi = a.tiles_per_item;
    if (a.strided) {
      item = at;
      at += a.clusters;
      f0 = 0;
      f1 = tpi;
    } else {
      item = at / tpi;
      f0 = static_cast<int>(at - item * tpi);
      const int64_t left = end - at;
      f1 = left < tpi - f0 ? f0 + static_cast<int>(left) : tpi;
      at += f1 - f0;
    }
    part = (f0 == 0 && f1 == tpi) ? -1 : (f0 > 0 ? 0 : 1);
    t = item / a.groups;
    hg = static_cast<int>(item - t * a.groups);
    q = query_of(a.p, t);
    // a query shorter than the longest spreads its tiles over its clusters alike
    const int nt = (q.n1 + q.n2 + kRows - 1) / kRows;
    j0 = static_cast<int>(static_cast<int64_t>(f0) * nt / tpi);
    j1 = static_cast<int>(static_cast<int64_t>(f1) * nt / tpi);
    return true;
  }
  // The next segment that has tiles.
  __device__ __forceinline__ bool next_nonempty() {
    while (next())
      if (j1 > j0) return true;
    return false;
  }
};

// ------------------------------------------------------------------ PTX

__device__ __forceinline__ uint32_t peer_addr(uint32_t local, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
  return r;
}
__device__ __forceinline__ void push_v4(uint32_t addr, float4 v, uint32_t bar) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
          addr),
      "r"(__float_as_uint(v.x)), "r"(__float_as_uint(v.y)), "r"(__float_as_uint(v.z)),
      "r"(__float_as_uint(v.w)), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_remote(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr)
               : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// D[tmem] (+)= A[tmem] x B[smem]: A one 32-bit column per two K elements, lane = row.
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, "
      "%19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, "
      "%19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Instruction descriptor of kind::f16: D fp32, A and B of one 16-bit type, A K-major, M = 128;
// bn: B MN-major.
__host__ __device__ constexpr uint32_t idesc(bool bf16, bool bn, int n) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (bn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(kHeads >> 4) << 24);
}

__device__ __forceinline__ uint32_t timer_lo() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}
// Bounded wait of a whole warp, acquiring at cluster scope; one answer for its lanes.  (No
// function call: calls do not go with setmaxnreg.)
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (__all_sync(0xffffffffu, try_wait_cluster(bar, parity))) return true;
  const uint32_t t0 = timer_lo();
  while (!__all_sync(0xffffffffu, try_wait_cluster(bar, parity))) {
    const bool late = timer_lo() - t0 > kWaitLimitNs;
    if (__any_sync(0xffffffffu, late || *abort_flag)) {
      if (late) {
        *abort_flag = 1;
        atomicOr(&g_attention_error, 1u);
      }
      return false;
    }
  }
  return true;
}
// Whether the phase of this parity has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
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

// Channel of slot `s` (a multiple of 8) of the padded row; -1 for padding.  `nope`: whether
// the slot lies in the FP8 part.
__device__ __forceinline__ int channel_of(const Args& a, int s, bool* nope) {
  *nope = s < a.cnp;
  if (*nope) return s < a.cn ? s : -1;
  return s - a.cnp < a.p.r ? a.cn + s - a.cnp : -1;
}

// ------------------------------------------------------------------ the kernel

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    attention_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kSmBars);
  uint64_t* kfull = bars;                 // [kStages] a row tile is in place
  uint64_t* kempty = kfull + kStages;     // [kStages] the MMAs are done with it
  uint64_t* qfull = kempty + kStages;     // Q in place (per segment)
  uint64_t* qempty = qfull + 1;           // the MMAs are done with Q
  uint64_t* sfull = qempty + 1;           // [2] this CTA's half of S complete
  uint64_t* pfull = sfull + 2;            // [2] weights in place
  uint64_t* pvdone = pfull + 2;           // [2] O includes the tile
  uint64_t* xfull = pvdone + 2;           // [2] the peer's half of S has landed
  uint64_t* xempty = xfull + 2;           // [2] the peer has read what this CTA pushed
  uint64_t* ofree = xempty + 2;           // O has been read (per segment)
  uint64_t* mh = ofree + 1;               // [4] running maximum handed on (per tile)
  uint64_t* lsync = mh + 4;               // [4] row sums of both groups posted (per segment)
  uint64_t* final_bar = lsync + 4;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + kSmMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kSmMisc + 4);
  uint8_t* mask = smem + kSmMask;
  uint8_t* qexp = smem + kSmExp;
  float* mrow = reinterpret_cast<float*>(smem + kSmM);
  float* lrow = reinterpret_cast<float*>(smem + kSmL);

  if ((smem_u32(smem) & 1023u) != 0) {  // the 128-byte swizzle counts on it
    if (threadIdx.x == 0) atomicOr(&g_attention_error, 1u);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t rank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int cid = blockIdx.x >> 1;
  const int A = a.atoms;
  // this CTA's blocks: the first na hold FP8 channels, the other nr bf16 ones
  const int na_all = a.cnp / 64 - static_cast<int>(rank) * A;
  const int na = na_all < 0 ? 0 : (na_all < A ? na_all : A);
  const int nr = A - na;
  const int slot0 = static_cast<int>(rank) * A * 64;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&kfull[s], kLoadWarps);
      mbar_init(&kempty[s], 1);
    }
    mbar_init(qfull, kLoadWarps);
    mbar_init(qempty, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sfull[b], 1);
      mbar_init(&pfull[b], 4);
      mbar_init(&pvdone[b], 1);
      mbar_init(&xfull[b], 1);
      mbar_init(&xempty[b], 4);
    }
    mbar_init(ofree, kSoftWarps);
    for (int w = 0; w < 4; ++w) {
      mbar_init(&mh[w], 1);
      mbar_init(&lsync[w], 2);
    }
    mbar_init(final_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(const_cast<uint32_t*>(tmem_slot))),
                 "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  // the peer's barriers are initialised before anything is pushed to it
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  Walker wk(a, cid);

  if (warp < kSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ------------------------------------------------------------ softmax groups
    const int grp = warp >> 2, w4 = warp & 3;
    const int row = w4 * 32 + lane;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(w4 * 32) << 16);
    const uint32_t sbuf = lane_addr + kColS + 128 * grp;
    const uint32_t peer = rank ^ 1u;
    const float4* xin = reinterpret_cast<const float4*>(smem + kSmX + grp * kXBuf) + row;
    const uint32_t xout = peer_addr(smem_u32(smem + kSmX + grp * kXBuf), peer) + row * 16;
    const uint32_t xout_bar = peer_addr(smem_u32(&xfull[grp]), peer);
    const uint32_t xempty_peer = peer_addr(smem_u32(&xempty[grp]), peer);
    const float b_scale = a.p.scale * kLog2e;
    const float inv_fp8 = 1.f / a.p.fp8_scale;
    uint32_t g = 0;     // tiles before this segment (all groups)
    uint32_t seg = 0;   // segments with tiles
    bool ok = true;
    while (ok && wk.next()) {
      const int nt = wk.j1 - wk.j0;
      if (!wk.q.ok && rank == 0 && threadIdx.x == 0) atomicOr(&g_attention_error, 2u);
      const int heads = a.p.H - wk.hg * kHeads < kHeads ? a.p.H - wk.hg * kHeads : kHeads;
      const bool active = w4 * 32 < heads;  // else the warp only keeps step
      float m_last = -INFINITY, l = 0.f, a_scale = 0.f;
      if (nt > 0) {
        bool mine = false;  // this group has had a tile of the segment
        for (int i = 0; i < nt && ok; ++i) {
          const uint32_t gt = g + i;
          if ((gt & 1u) != static_cast<uint32_t>(grp)) continue;
          const uint32_t n = gt >> 1;  // this group's tile count
          // S complete; the tile before it in this buffer is in O
          if (n > 0 && !wait_warp(&pvdone[grp], (n - 1) & 1u, abort_flag)) {
            ok = false;
            break;
          }
          if (w4 == 0 && lane == 0)
            mbar_arrive_expect_tx(&xfull[grp], ((heads + 31) >> 5) * 32 * kRows * 4);
          const uint32_t st = gt % kStages, ph = (gt / kStages) & 1u;
          if (!wait_warp(&sfull[grp], n & 1u, abort_flag) ||
              !wait_warp(&kfull[st], ph, abort_flag) ||
              (n > 0 && active && !wait_warp(&xempty[grp], (n - 1) & 1u, abort_flag))) {
            ok = false;
            break;
          }
          tc_fence_after();
          float x[kRows];
          float tmax = -INFINITY;
          if (active) {
            if (!mine) {
              // x = S_n * (2^(E - 142) scale / fp8_scale) + S_r * scale, in units of log 2
              const int e = qexp[(seg & 3u) * kHeads + row];
              a_scale = b_scale * inv_fp8 * __int_as_float((e - 15) << 23);
            }
#pragma unroll
            for (int c0 = 0; c0 < kRows; c0 += 16) {
              float (&xc)[16] = *reinterpret_cast<float(*)[16]>(x + c0);
              if (na > 0) {
                tmem_ld16(sbuf + c0, xc);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 16; ++c) xc[c] *= a_scale;
              }
              if (nr > 0) {
                float v[16];
                tmem_ld16(sbuf + kColR + c0, v);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 16; ++c)
                  xc[c] = na > 0 ? fmaf(v[c], b_scale, xc[c]) : v[c] * b_scale;
              }
#pragma unroll
              for (int c = 0; c < 16; c += 4)
                push_v4(xout + ((c0 + c) >> 2) * (kHeads * 16),
                        make_float4(x[c0 + c], x[c0 + c + 1], x[c0 + c + 2], x[c0 + c + 3]),
                        xout_bar);
            }
            if (!wait_warp(&xfull[grp], n & 1u, abort_flag)) {
              ok = false;
              break;
            }
#pragma unroll
            for (int c = 0; c < kRows; c += 4) {
              const float4 v = xin[(c >> 2) * kHeads];
              x[c] += v.x;
              x[c + 1] += v.y;
              x[c + 2] += v.z;
              x[c + 3] += v.w;
            }
            const uint2 live = *reinterpret_cast<const uint2*>(mask + st * 8);
            if ((live.x & live.y) != 0xffffffffu) {
#pragma unroll
              for (int c = 0; c < kRows; ++c)
                if (!(((c < 32 ? live.x : live.y) >> (c & 31)) & 1u)) x[c] = -INFINITY;
            }
#pragma unroll
            for (int c = 0; c < kRows; ++c) tmax = fmaxf(tmax, x[c]);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(xempty_peer);
          // the reference: the running maximum, or up to kSlack below it
          float m_old = -INFINITY;
          if (i > 0) {
            if (!wait_warp(&mh[w4], (gt - 1) & 1u, abort_flag)) {
              ok = false;
              break;
            }
            m_old = mrow[row];
          }
          const float m_new = i == 0 || tmax > m_old + kSlack ? tmax : m_old;
          mrow[row] = m_new;
          __syncwarp();
          if (lane == 0) mbar_arrive(&mh[w4]);
          if (active) {
            if (i > 0 && __any_sync(0xffffffffu, m_new != m_old)) {
              // O so far moves to the new reference, once the tile before this one is in it
              if (!wait_warp(&pvdone[grp ^ 1], ((gt - 1) >> 1) & 1u, abort_flag)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const float f = m_new != m_old ? ex2_ftz(m_old - m_new) : 1.f;
              for (int c0 = 0; c0 < A * 64; c0 += 32) {
                uint32_t v[32];
                tmem_ld32(lane_addr + c0, v);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) * f);
                tmem_st32(lane_addr + c0, v);
              }
            }
            const float ref = (m_new == -INFINITY ? 0.f : m_new) - kBias;
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int c = 0; c < kRows; c += 2) {
              x[c] = ex2_ftz(x[c] - ref);
              x[c + 1] = ex2_ftz(x[c + 1] - ref);
              s0 += x[c];
              s1 += x[c + 1];
            }
            uint32_t pk[16];
#pragma unroll
            for (int c0 = 0; c0 < 32; c0 += 16) {
              if (na > 0) {
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                  const __half2 h = __floats2half2_rn(x[2 * (c0 + c)], x[2 * (c0 + c) + 1]);
                  pk[c] = *reinterpret_cast<const uint32_t*>(&h);
                }
                tmem_st16(sbuf + c0, pk);
              }
              if (nr > 0) {
#pragma unroll
                for (int c = 0; c < 16; ++c)
                  pk[c] = pack_bf16x2(x[2 * (c0 + c)], x[2 * (c0 + c) + 1]);
                tmem_st16(sbuf + 32 + c0, pk);
              }
            }
            tmem_wait_st();
            if (mine && m_last != m_new) l *= ex2_ftz(m_last - m_new);
            l += s0 + s1;
          }
          m_last = m_new;
          mine = true;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&pfull[grp]);
        }
        if (!ok) break;
        // ---- both groups: the final maximum and sum of every row
        const uint32_t gl = g + nt - 1;
        float m_fin = m_last;
        if ((gl & 1u) != static_cast<uint32_t>(grp)) {
          if (!wait_warp(&mh[w4], gl & 1u, abort_flag)) break;
          m_fin = mrow[row];
        }
        if (l != 0.f && m_last != m_fin) l *= ex2_ftz(m_last - m_fin);
        // every warp has read the row sums of the segment before
        if (seg > 0 && !wait_warp(ofree, (seg - 1) & 1u, abort_flag)) break;
        lrow[grp * kHeads + row] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(&lsync[w4]);
        if (!wait_warp(&lsync[w4], seg & 1u, abort_flag) ||
            !wait_warp(&pvdone[gl & 1u], (gl >> 1) & 1u, abort_flag))
          break;
        l = (lrow[row] + lrow[kHeads + row]) * (1.f / 128.f);  // without the 2^kBias
        m_last = m_fin;
        tc_fence_after();
        g += nt;
        ++seg;
      }
      // ---- store: out and lse of a whole query, or the part's O, m and l
      const int head = wk.hg * kHeads + row;
      const bool live = row < heads && wk.q.ok;
      float f_rope;
      if (wk.part < 0) {
        const float sink2 = a.p.sink && live ? a.p.sink[head] * kLog2e : -INFINITY;
        const float M = fmaxf(m_last, sink2);
        float f = 0.f, den = 0.f;
        if (M != -INFINITY) {
          f = ex2_ftz(m_last - M);
          den = l * f + (a.p.sink ? ex2_ftz(sink2 - M) : 0.f);
        } else if (l != l) {
          f = den = l;  // NaN scores only
        }
        f_rope = den != 0.f ? f / den * (1.f / 128.f) : 0.f;
        if (rank == 0 && grp == 0 && live && a.p.lse)
          a.p.lse[wk.t * a.p.H + head] =
              m_last == -INFINITY && l == 0.f  // no row: the sink's logit as it is
                  ? (a.p.sink ? a.p.sink[head] : -INFINITY)
                  : (M == -INFINITY ? 0.f : M) * 0.6931471805599453f + logf(den);
      } else {
        f_rope = 1.f / 128.f;
        if (rank == 0 && grp == 0 && live)
          a.part_ml[(cid * 2 + wk.part) * kHeads + row] = make_float2(m_last, l);
      }
      const float f_nope = f_rope * inv_fp8;
      __nv_bfloat16* out =
          static_cast<__nv_bfloat16*>(a.p.out) + (wk.t * a.p.H + head) * a.p.c;
      float* po = a.part_o + (static_cast<int64_t>(cid * 2 + (wk.part > 0 ? 1 : 0)) * kHeads + row) *
                                 a.p.c;
      // each group takes half of this CTA's columns
      for (int c0 = grp * A * 32; c0 < (grp + 1) * A * 32; c0 += 32) {
        uint32_t v[32];
        __syncwarp();
        if (nt > 0) {
          tmem_ld32(lane_addr + c0, v);
          tmem_wait_ld();
        } else {
          if (wk.part >= 0) break;
#pragma unroll
          for (int c = 0; c < 32; ++c) v[c] = 0u;
        }
        if (!live) continue;
#pragma unroll
        for (int c = 0; c < 32; c += 8) {
          bool nope;
          const int ch = channel_of(a, slot0 + c0 + c, &nope);
          const float f = nope ? f_nope : f_rope;
          float o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = __uint_as_float(v[c + e]) * f;
          if (ch >= 0) {
            if (wk.part < 0) {
              *reinterpret_cast<uint4*>(out + ch) =
                  make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]),
                             pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7]));
            } else {
              *reinterpret_cast<float4*>(po + ch) = make_float4(o[0], o[1], o[2], o[3]);
              *reinterpret_cast<float4*>(po + ch + 4) = make_float4(o[4], o[5], o[6], o[7]);
            }
          }
        }
      }
      if (nt > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ofree);
      }
    }
  } else if (warp < kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
    // ------------------------------------------------------------ row gather
    const int pw = warp - kSoftWarps;
    const int cs = slot0 + lane * 8;  // this lane's 8-channel slot of every row
    bool nope = false;
    const int ch = lane < A * 8 ? channel_of(a, cs, &nope) : -1;
    const int64_t rch = ch - a.cn;    // offset in the bf16 part
    // swizzled place of (row, this lane's slot): 16-byte chunk lane % 8 of block lane / 8
    const uint32_t katom = (lane >> 3) * kKAtom, qatom = (lane >> 3) * kQAtom;
    const int lc = lane & 7;

    // A tile whose row numbers are on their way: lane i < 8 has row pw * 8 + i.
    struct Pending {
      bool live, first;
      int64_t t, base, n_visible;
      int hg, kind, raw;  // kind: 0 none, 1 listed (raw pending), 2 cache row, 3 window row
    };
    bool seg_live = wk.next_nonempty();
    int j = wk.j0;
    auto fetch = [&](Pending& p) {
      p.live = seg_live;
      if (!seg_live) return;
      p.first = j == wk.j0;
      p.t = wk.t;
      p.hg = wk.hg;
      p.n_visible = wk.q.n_visible;
      p.kind = 0;
      p.raw = 0;
      p.base = 0;
      const int e = j * kRows + pw * 8 + (lane & 7);
      if (e < wk.q.n1) {
        p.base = wk.q.key_start + e;
        p.kind = 2;
        if (a.p.idx) {
          p.base = wk.q.key_start;
          p.kind = 1;
          p.raw = a.p.idx[wk.t * a.p.k + e];
        }
      } else if (e < wk.q.n1 + wk.q.n2) {
        p.base = wk.q.win_start + (e - wk.q.n1);
        p.kind = 3;
      }
      if (++j == wk.j1) {
        seg_live = wk.next_nonempty();
        j = wk.j0;
      }
    };
    uint4 data[8];
    uint32_t bits = 0;  // which of the 8 rows count
    auto load = [&](const Pending& p, uint4 (&d)[8], uint32_t& valid) {
      int64_t r = p.base;
      bool v = p.kind != 0;
      if (p.kind == 1) {
        v = p.raw >= 0 && p.raw < p.n_visible;
        r += p.raw;
        if (!v && p.raw != -1 && lane < 8 && rank == 0) atomicOr(&g_attention_error, 2u);
      }
      // one word per row: the row number, the window flag, the validity flag
      const unsigned long long code =
          (v ? (1ull << 63) : 0ull) | (p.kind == 3 ? (1ull << 62) : 0ull) |
          (v ? static_cast<unsigned long long>(r) : 0ull);
      valid = __ballot_sync(0xffffffffu, v) & 0xffu;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const unsigned long long cd = __shfl_sync(0xffffffffu, code, i);
        d[i] = make_uint4(0u, 0u, 0u, 0u);
        if ((cd >> 63) && ch >= 0) {
          const bool win = (cd >> 62) & 1ull;
          const int64_t rr = static_cast<int64_t>(cd & ((1ull << 62) - 1));
          if (nope) {
            const uint8_t* b = static_cast<const uint8_t*>(win ? a.p.win_nope : a.p.nope);
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(b + rr * a.cn + ch));
            d[i].x = w.x;
            d[i].y = w.y;
          } else {
            const __nv_bfloat16* b =
                static_cast<const __nv_bfloat16*>(win ? a.p.win_rope : a.p.rope);
            d[i] = __ldg(reinterpret_cast<const uint4*>(b + rr * a.p.r + rch));
          }
        }
      }
    };
    Pending nxt, cur;
    fetch(cur);
    if (cur.live) load(cur, data, bits);
    fetch(nxt);
    uint32_t gt = 0, seg = 0;
    while (cur.live) {
      if (cur.first) {
        // ---- Q of the segment: 16 rows per warp, FP8 channels to scaled fp16
        if (!wait_warp(qempty, (seg & 1u) ^ 1u, abort_flag)) break;
        const int heads = a.p.H - cur.hg * kHeads;
        const __nv_bfloat16* qb = static_cast<const __nv_bfloat16*>(a.p.q) +
                                  (cur.t * a.p.H + cur.hg * kHeads) * a.p.c;
#pragma unroll
        for (int r0 = 0; r0 < 16; r0 += 8) {
          uint4 qv[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = pw * 16 + r0 + i;
            qv[i] = make_uint4(0u, 0u, 0u, 0u);
            if (rr < heads && ch >= 0)
              qv[i] = __ldg(reinterpret_cast<const uint4*>(qb + rr * a.p.c + ch));
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = pw * 16 + r0 + i;
            const uint32_t w[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t lo = w[k] & 0x7fffu, hi = (w[k] >> 16) & 0x7fffu;
              top = max(top, max(lo, hi));
            }
            int e = static_cast<int>(__reduce_max_sync(0xffffffffu, nope ? top : 0u) >> 7);
            if (e == 255) e = 142;  // an infinity or NaN: no scaling
            if (e < 16) e = 16;     // 2^(142 - e) stays finite
            if (lane == 0) qexp[(seg & 3u) * kHeads + rr] = static_cast<uint8_t>(e);
            uint32_t h[4] = {w[0], w[1], w[2], w[3]};
            if (nope) {
              const float mul = __int_as_float((142 - e + 127) << 23);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const __half2 hh =
                    __floats2half2_rn(__uint_as_float(w[k] << 16) * mul,
                                      __uint_as_float(w[k] & 0xffff0000u) * mul);
                h[k] = *reinterpret_cast<const uint32_t*>(&hh);
              }
            }
            if (lane < A * 8)
              *reinterpret_cast<uint4*>(smem + kSmQ + qatom + rr * 128 + ((lc ^ (rr & 7)) << 4)) =
                  make_uint4(h[0], h[1], h[2], h[3]);
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(qfull);
        ++seg;
      }
      // the next tile's rows set out before this tile's are needed
      uint4 dnext[8];
      uint32_t bnext = 0;
      if (nxt.live) load(nxt, dnext, bnext);
      const bool nlive = nxt.live, nfirst = nxt.first;
      const int64_t n_t = nxt.t;
      const int n_hg = nxt.hg;
      fetch(nxt);
      const uint32_t st = gt % kStages;
      if (!wait_warp(&kempty[st], ((gt / kStages) & 1u) ^ 1u, abort_flag)) break;
      uint8_t* kb = smem + kSmK + st * kStage + katom;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int rr = pw * 8 + i;
        uint4 v = data[i];
        if (nope) {
          const uint32_t w0 = data[i].x, w1 = data[i].y;
          const __half2_raw h0 = __nv_cvt_fp8x2_to_halfraw2(w0 & 0xffffu, __NV_E4M3);
          const __half2_raw h1 = __nv_cvt_fp8x2_to_halfraw2(w0 >> 16, __NV_E4M3);
          const __half2_raw h2 = __nv_cvt_fp8x2_to_halfraw2(w1 & 0xffffu, __NV_E4M3);
          const __half2_raw h3 = __nv_cvt_fp8x2_to_halfraw2(w1 >> 16, __NV_E4M3);
          v = make_uint4(h0.x | (uint32_t(h0.y) << 16), h1.x | (uint32_t(h1.y) << 16),
                         h2.x | (uint32_t(h2.y) << 16), h3.x | (uint32_t(h3.y) << 16));
        }
        if (lane < A * 8) *reinterpret_cast<uint4*>(kb + rr * 128 + ((lc ^ (rr & 7)) << 4)) = v;
      }
      if (lane == 0) mask[st * 8 + pw] = static_cast<uint8_t>(bits);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&kfull[st]);
      ++gt;
      cur.live = nlive;
      cur.first = nfirst;
      cur.t = n_t;
      cur.hg = n_hg;
      bits = bnext;
#pragma unroll
      for (int i = 0; i < 8; ++i) data[i] = dnext[i];
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
    if (warp == kMmaWarp && lane == 0) {
    // ------------------------------------------------------------ MMA issuer
    const uint64_t qd = smem_desc(smem_u32(smem + kSmQ), 16, 1024, 2);
    const uint64_t kd = smem_desc(smem_u32(smem + kSmK), 16, 1024, 2);        // K-major (S)
    const uint64_t vd = smem_desc(smem_u32(smem + kSmK), kKAtom, 1024, 2);    // MN-major (P K)
    const uint32_t is_n = idesc(false, false, kRows), is_r = idesc(true, false, kRows);
    const uint32_t io_n = idesc(false, true, na * 64), io_r = idesc(true, true, nr * 64);
    bool s_live = wk.next_nonempty();
    int j = wk.j0;
    uint32_t s = 0, pv = 0;         // tiles whose S / P K has been issued
    uint32_t s_seg = 0, pv_seg = 0; // segments begun
    uint32_t first_bits = 0;        // tile & 3: first of its segment
    uint64_t t0 = global_timer_ns();
    uint32_t spins = 0;
    while (s_live || pv < s) {
      bool moved = false;
      if (pv < s) {
        const uint32_t b = pv & 1u;
        const bool first = (first_bits >> (pv & 3u)) & 1u;
        if (mbar_test(&pfull[b], (pv >> 1) & 1u) &&
            (!first || pv_seg == 0 || mbar_test(ofree, (pv_seg - 1) & 1u))) {
          tc_fence_after();
          const uint32_t st = pv % kStages;
          const uint32_t pt = tmem + kColS + 128 * b;
          for (int ks = 0; ks < kRows / 16; ++ks) {
            const uint64_t d = vd + ((st * kStage + ks * 16 * 128) >> 4);
            const uint32_t acc = (!first || ks > 0) ? 1u : 0u;
            if (na > 0) umma_ts(tmem, pt + ks * 8, d, io_n, acc);
            if (nr > 0)
              umma_ts(tmem + na * 64, pt + 32 + ks * 8, d + ((na * kKAtom) >> 4), io_r, acc);
          }
          umma_commit(&kempty[st]);
          umma_commit(&pvdone[b]);
          if (first) ++pv_seg;
          ++pv;
          moved = true;
        }
      }
      if (s_live && s < pv + 2) {
        const uint32_t b = s & 1u, st = s % kStages;
        const bool first = j == wk.j0;
        if ((!first || mbar_test(qfull, s_seg & 1u)) &&
            mbar_test(&kfull[st], (s / kStages) & 1u)) {
          tc_fence_after();
          const uint32_t dt = tmem + kColS + 128 * b;
          for (int at = 0; at < A; ++at) {
            const bool r = at >= na;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              umma_bf16(dt + (r ? kColR : 0), qd + ((at * kQAtom + ks * 32) >> 4),
                        kd + ((st * kStage + at * kKAtom + ks * 32) >> 4), r ? is_r : is_n,
                        ((at != 0 && at != na) || ks > 0) ? 1u : 0u);
          }
          umma_commit(&sfull[b]);
          first_bits = (first_bits & ~(1u << (s & 3u))) | ((first ? 1u : 0u) << (s & 3u));
          if (first) ++s_seg;
          ++s;
          if (++j == wk.j1) {
            umma_commit(qempty);
            s_live = wk.next_nonempty();
            j = wk.j0;
          }
          moved = true;
        }
      }
      if (moved) {
        spins = 0;
      } else if (++spins >= 64) {
        if (spins == 64) t0 = global_timer_ns();
        if (*abort_flag) break;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
          *abort_flag = 1;
          atomicOr(&g_attention_error, 1u);
          break;
        }
      }
    }
    umma_commit(final_bar);  // every MMA issued above has finished before TMEM is freed
    const uint64_t tf = global_timer_ns();
    while (!mbar_try_wait(final_bar, 0) && global_timer_ns() - tf < kWaitLimitNs) {
    }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
  // neither CTA leaves while the other may still push into it
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// ------------------------------------------------------------------ joining the parts

constexpr int kJoinThreads = 128;

// A query whose units begin in cluster k - 1 and go on in cluster k (and perhaps further) was
// split: block (k, head) adds its parts in cluster order.
__global__ void __launch_bounds__(kJoinThreads) attention_join_kernel(const Args a) {
  const int64_t k = blockIdx.x, U = a.units, C = a.clusters;
  const int tpi = a.tiles_per_item;
  const int64_t lo = k * U / C;
  const int64_t item = lo / tpi;
  if (lo == item * tpi) return;
  const int64_t kf = ((item * tpi + 1) * C - 1) / U;
  if (kf != k - 1) return;
  const int64_t kl = ((item + 1) * tpi * C - 1) / U;
  const int64_t t = item / a.groups;
  const int hg = static_cast<int>(item - t * a.groups);
  const int row = blockIdx.y, head = hg * kHeads + row;
  if (head >= a.p.H || !query_of(a.p, t).ok) return;
  auto slot = [&](int64_t c) { return (c * 2 + (c == kf ? 1 : 0)) * kHeads + row; };
  float M = a.p.sink ? a.p.sink[head] * kLog2e : -INFINITY;
  const float sink2 = M;
  bool nan = false, rows = false;
  for (int64_t c = kf; c <= kl; ++c) {
    const float2 ml = a.part_ml[slot(c)];
    M = fmaxf(M, ml.x);
    nan = nan || ml.y != ml.y;
    rows = rows || ml.y != 0.f;
  }
  float den = 0.f;
  const float ref = M == -INFINITY ? 0.f : M;
  for (int64_t c = kf; c <= kl; ++c) {
    const float2 ml = a.part_ml[slot(c)];
    if (ml.y != 0.f) den += ml.y * ex2_ftz(ml.x - ref);
  }
  if (a.p.sink) den += ex2_ftz(sink2 - ref);
  if (nan) den = NAN;
  if (threadIdx.x == 0 && a.p.lse)
    a.p.lse[t * a.p.H + head] = !rows ? (a.p.sink ? a.p.sink[head] : -INFINITY)
                                      : ref * 0.6931471805599453f + logf(den);
  const float inv = den != 0.f ? 1.f / den : 0.f;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.p.out) + (t * a.p.H + head) * a.p.c;
  for (int ch = threadIdx.x * 4; ch < a.p.c; ch += kJoinThreads * 4) {
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int64_t c = kf; c <= kl; ++c) {
      const int64_t s = slot(c);
      const float2 ml = a.part_ml[s];
      if (ml.y == 0.f) continue;  // the part had no row: its O is not written
      const float f = ex2_ftz(ml.x - ref);
      const float4 v = *reinterpret_cast<const float4*>(a.part_o + s * a.p.c + ch);
      o.x = fmaf(v.x, f, o.x);
      o.y = fmaf(v.y, f, o.y);
      o.z = fmaf(v.z, f, o.z);
      o.w = fmaf(v.w, f, o.w);
    }
    *reinterpret_cast<uint2*>(out + ch) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  }
}

// ------------------------------------------------------------------ launch

constexpr int kMaxClusters = 74;     // pairs of the 148 SMs
constexpr int kMinTiles = 2;         // tiles per cluster below which a query is not split
constexpr int64_t kStridedItems = 8; // items per cluster from which queries are never split

struct Plan {
  int64_t items, units;
  int tiles_per_item, groups, clusters;
  bool strided;
};
Plan plan_of(int64_t T, int H, int64_t most, int max_clusters) {
  Plan p;
  p.groups = static_cast<int>(ceil_div(H, kHeads));
  p.items = T * p.groups;
  p.tiles_per_item = most > 0 ? static_cast<int>(ceil_div(most, kRows)) : 1;
  p.units = p.items * p.tiles_per_item;
  p.strided = p.items >= kStridedItems * max_clusters;
  if (p.strided) {
    p.clusters = max_clusters;
  } else {
    int64_t c = p.units / kMinTiles;
    if (c < p.items) c = p.items;
    p.clusters = static_cast<int>(c < max_clusters ? c : max_clusters);
  }
  return p;
}
int64_t ml_bytes(int clusters) { return int64_t(clusters) * 2 * kHeads * sizeof(float2); }

}  // namespace attn

int64_t attention_workspace_bytes(int64_t T, int H, int64_t c, int, int64_t most) {
  using namespace attn;
  const Plan p = plan_of(T, H, most, kMaxClusters);
  if (p.strided || p.tiles_per_item == 1) return 0;  // no query is split
  return ml_bytes(p.clusters) + int64_t(p.clusters) * 2 * kHeads * c * 4;
}

kvc_status launch_attention(const AttentionProblem& p, cudaStream_t st) {
  using namespace attn;
  if (!raise_smem_limit(reinterpret_cast<const void*>(attention_kernel))) return KVC_ERR_CUDA;
  // clusters that fit the device at once (waits between the CTAs of one cluster only)
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KVC_ERR_CUDA;
  static std::mutex mu;
  static int fit[64] = {};
  int max_clusters;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (fit[dev] == 0) {
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = 2;
      at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(2 * kMaxClusters, 1, 1);
      cfg.blockDim = dim3(kThreads, 1, 1);
      cfg.dynamicSmemBytes = kSmem;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, attention_kernel, &cfg) != cudaSuccess || n < 1) {
        (void)cudaGetLastError();
        return KVC_ERR_CUDA;
      }
      fit[dev] = n < kMaxClusters ? n : kMaxClusters;
    }
    max_clusters = fit[dev];
  }
  const int64_t most = (p.idx ? p.k : p.max_visible) + (p.win_start ? p.max_win : 0);
  const Plan pl = plan_of(p.T, p.H, most, max_clusters);
  Args a{};
  a.p = p;
  a.items = pl.items;
  a.units = pl.units;
  a.tiles_per_item = pl.tiles_per_item;
  a.groups = pl.groups;
  a.clusters = pl.clusters;
  a.strided = pl.strided;
  a.cn = static_cast<int>(p.c) - p.r;
  a.cnp = (a.cn + 63) / 64 * 64;
  a.atoms = (a.cnp / 64 + (p.r + 63) / 64 + 1) / 2;
  a.part_ml = static_cast<float2*>(p.workspace);
  a.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(p.workspace) + ml_bytes(pl.clusters));
  attention_kernel<<<2 * pl.clusters, kThreads, kSmem, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return KVC_ERR_CUDA;
  const bool whole =
      pl.units % pl.clusters == 0 && (pl.units / pl.clusters) % pl.tiles_per_item == 0;
  if (!pl.strided && !whole) {  // some query is split
    attention_join_kernel<<<dim3(pl.clusters, p.H < kHeads ? p.H : kHeads), kJoinThreads, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return KVC_ERR_CUDA;
  }
  last_kernel() = "attention_kernel";
  return KVC_OK;
}

unsigned int read_and_clear_attention_error(bool* failed) {
  unsigned int v = 0;
  const unsigned int zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_attention_error, sizeof(v)) != cudaSuccess) {
    *failed = true;
    return 0;
  }
  if (v != 0 && cudaMemcpyToSymbol(g_attention_error, &zero, sizeof(zero)) != cudaSuccess)
    *failed = true;
  return v;
}

}  // namespace kvc
