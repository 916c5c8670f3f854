// Shared-KV attention over the compressed cache on sm_100a (include/kvc.h,
// shared_kv_attention and shared_kv_attention_topk).
//
// What it computes, per query t and head h over the query's rows s (listed or visible cache
// entries, then its window), with K_s = [nope_s / fp8_scale ; rope_s] both key and value:
//     x_s = scale q[t,h].K_s,  out[t,h] = sum_s exp(x_s) K_s / D,  D = sum_s exp(x_s) (+ sink)
// in one pass over the rows with the running maximum and sum of the softmax.
//
// One query's heads share every row, so a query is a pair of GEMMs with the heads on M:
// S = Q K^T [heads x 64 rows] and O += P K [heads x c].  At 128 heads that is 455 flop per
// cache byte, above the 246 the machine has per byte: the tensor cores bound it; at 64 heads
// and below HBM does.
//
// Split.  A CTA takes 64 heads of a query: O for 64 heads x 512 channels in fp32 is half of the
// SM's TMEM (channels 0-255 in the lower 16 lanes of each quarter, 256-511 in the upper 16),
// S double-buffered in the other half, and a tile of 64 rows is held once in shared memory as
// the B operand of both GEMMs (K-major for S, MN-major for P K).  An M = 64 MMA takes as long
// as one with M = 128 of the same N from N = 128 on (measured: 32 cycles at N = 64, 128 at
// N = 256), so a tile costs 2060 tensor cycles, twice its share of the peak.  128 heads a CTA
// would need all of TMEM for O alone.  Measured against it: two CTAs per query with 128 heads
// and half of the channels each halve the MMA time on paper, but the half-sums of S they must
// exchange cross the SM-to-SM network at 20 bytes a cycle and its latency (about 4000 cycles)
// sits in every tile's chain: 5300 cycles a tile.
//
// What a tile takes: 4250 cycles (chunk of 1024 queries x 1152 rows x 128 heads: 575 us, 529
// TFLOP/s).  With every load, conversion, exponential and store taken out 3100 remain, and the
// hand-overs alone (no MMAs either) take 1000: S of a tile, its softmax, P K and the refill of
// its place follow one another, two tiles in turn, and S reads Q and K from shared memory at
// nearly all the bytes a cycle that it has, so that everything beside it waits: a wait that is
// over already takes 170 to 250 cycles.  So no barrier stands where another one implies it.
//
// Types.  An E4M3 byte is exact in fp16, and a bf16 query row is exact in fp16 once scaled by
// a power of two (its largest value to 2^15: what is lost lies 2^-40 below it), so the FP8
// channels run as fp16 MMAs with the weights rounded to fp16 (2^-11); the bf16 channels keep
// bf16 for its exponent range, with weights rounded to bf16 (2^-8).  The two parts have
// accumulators of their own (S_n, S_r), because only S_n carries the row's power of two and
// 1 / fp8_scale.  Both parts accumulate in fp32.
//
// Roles of the 28 warps.  0-3 take the softmax, 4-7 store finished queries, 8-23 gather the
// rows' FP8 channels (global memory -> registers -> widened, swizzled shared memory), 24
// issues the MMAs, 25 walks the segments (query, row tiles) of its CTA and posts them to the
// others, 26-27 find each tile's rows, tell the gather and copy the bf16 channels.  A query's
// tiles are split among CTAs when there are too few queries, and a second kernel joins the
// parts in a fixed order.  Work is dealt by the longest length a call allows, which the host
// knows, not by each query's own, which only the device does: queries of one length fill the
// CTAs alike, ragged ones do not (see plan_of).
#include <cuda_fp16.h>

#include "kvc_common.cuh"
#include "kvc_host.h"
#include "kvc_launch.h"
#include "tc_ptx.cuh"

namespace kvc {

// bit 0: a bounded wait gave up; bit 1: a query's rows or a listed entry out of range.
__device__ unsigned int g_attention_error = 0;
// What a row that does not count reads: E4M3 zeros.
__device__ __align__(16) const uint8_t g_zero_row[512] = {};

namespace attn {

using namespace tcx;

// A segment of work, as the scheduler warp posts it in shared memory: tiles [j0, j1) of one
// query's rows for one group of heads.  part: -1 the whole query, else this CTA's slot for the
// partial result; t < 0 ends the list.  Segments without a tile are not posted: the store
// warps, which have their outputs to write, walk the CTA's units themselves.  (Posted, a run of
// them longer than the ring would stop the roles that read ahead of the store.)
struct Seg {
  int64_t t, key_start, win_start, n_visible;
  int hg, j0, j1, n1, n2, part, ok, item;
};
static_assert(sizeof(Seg) == 64, "segment record");

constexpr int kRows = 64;         // rows of a tile (MMA N of S, K of P K)
constexpr int kHeads = 64;        // heads of an item (MMA M)
constexpr int kStages = 2;        // row-tile ring
constexpr int kSoftWarps = 4, kStoreWarps = 4, kLoadWarps = 16;
constexpr int kOwn = kRows / kLoadWarps;          // rows of a tile per gather warp
constexpr int kLoad0 = kSoftWarps + kStoreWarps;  // first gather warp
constexpr int kMmaWarp = kLoad0 + kLoadWarps;
constexpr int kThreads = 32 * (kMmaWarp + 4);  // whole warpgroups for setmaxnreg
// Registers a thread: 72 at launch (896 threads), split so that no role spills.
constexpr int kSoftRegs = 104, kStoreRegs = 56, kLoadRegs = 72, kMmaRegs = 56;
static_assert(kSoftRegs + kStoreRegs + 4 * kLoadRegs + kMmaRegs <= 7 * 72, "register split");
constexpr int kMaxAtoms = 8;      // 64-channel blocks of a row
constexpr int kAtom = 64 * 128;   // one [64 rows or heads x 64] block of 16-bit values, 8 KB
constexpr int kStage = kMaxAtoms * kAtom;
constexpr int kSegs = 8;          // segment records under way
constexpr int kExps = 4;          // and exponents of Q rows
// Bounded waits: every wait of a CTA gives up once the CTA has not gone on for kWaitTicks ticks
// of 2^16 cycles (2 to 3 s).  It goes on when a tile's rows are in place (microseconds) and when
// the scheduler or a store warp walks over a query, so neither a long query (many tiles before
// the store warps' next output) nor a padded batch (2^28 queries of which six have rows: 4.2 s
// in which the other roles have nothing to do; a limit of 2^18 polls gave up there) is taken for
// a standstill.  The cycle counter is read at every 16th poll of a wait; reading the nanosecond
// timer between polls took thousands of cycles and made every wait that long.
constexpr uint32_t kWaitTicks = 1u << 16;
// Weights are exp2(x - m + kBias): with m at most kSlack below the running maximum they stay
// below 2^15 in fp16 and vanish only 2^-31 below the maximum.
constexpr float kBias = 7.f;
constexpr float kUnbias = 1.f / 128.f;
constexpr float kSlack = 8.f;

// Shared memory (bytes).
constexpr int kSmQ = 0;
constexpr int kSmK = kSmQ + kMaxAtoms * kAtom;
constexpr int kSmP = kSmK + kStages * kStage;        // [2][fp16, bf16] weights
constexpr int kSmSeg = kSmP + 4 * kAtom;
constexpr int kSmRow = kSmSeg + kSegs * int(sizeof(Seg));  // u64 [2][kRows] where rows begin
constexpr int kSmMl = kSmRow + 2 * kRows * 8;        // float2 [kHeads] (m, l)
constexpr int kSmExp = kSmMl + kHeads * 8;           // u8 [kExps][kHeads] exponents of Q rows
constexpr int kSmMask = kSmExp + kExps * kHeads;     // u32 [kStages][2] rows that count
constexpr int kSmMisc = kSmMask + kStages * 8;       // tmem address, abort flag, tick of the last step
constexpr int kSmBars = kSmMisc + 16;
// mbarriers, by index
constexpr int kBKFull = 0;                  // [kStages] a row tile is in place
constexpr int kBKEmpty = kBKFull + kStages; // [kStages] the MMAs are done with it:
constexpr int kBPvDone = kBKEmpty;          // O includes the tile, its weights have been used
static_assert(kStages == 2, "as many as S and weight buffers");
constexpr int kBQFull = kBKEmpty + kStages; // Q in place (per segment)
constexpr int kBQEmpty = kBQFull + 1;       // the MMAs are done with Q
constexpr int kBSFull = kBQEmpty + 1;       // [2] S complete
constexpr int kBPFull = kBSFull + 2;        // [2] weights in place, S has been read
constexpr int kBOFree = kBPFull + 2;        // O has been read (per segment)
constexpr int kBLFull = kBOFree + 1;        // [kSegs] (m, l) posted
constexpr int kBSegFull = kBLFull + kSegs;  // [kSegs] a segment record is posted
constexpr int kBSegEmpty = kBSegFull + kSegs;  // [kSegs] every role has read it
constexpr int kBRowFull = kBSegEmpty + kSegs;  // [2] a tile's rows are known
constexpr int kBRowEmpty = kBRowFull + 2;   // [2] their loads have set out
constexpr int kBFinal = kBRowEmpty + 2;
constexpr int kNumBars = kBFinal + 1;
constexpr int kSmem = kSmBars + kNumBars * 8;
static_assert(kSmBars % 8 == 0 && kSmRow % 16 == 0 && kSmMask % 8 == 0 && kOwn == 4, "layout");
static_assert(kSmem <= 227 * 1024, "attention shared memory");
// TMEM columns: O 0-255; S buffer b 64 columns, S_n in the lower, S_r in the upper 16 lanes of
// each quarter (as O's channels below and above 256).
constexpr int kColS = 256;
constexpr uint32_t kUpper = 16u << 16;

struct Args {
  AttentionProblem p;
  int items, tiles_per_item;  // an item: a query and a group of heads
  int groups, ctas;
  int per_cta, extra;       // units (items x tiles_per_item) per CTA, one more in the first `extra`
  int na, nr;               // 64-channel blocks: FP8, then bf16
  int cn;                   // FP8 channels
  bool strided;             // whole items, CTA by CTA (no splits)
  bool wide_out;            // 32-byte stores to out are aligned (16 channels at a multiple of 16)
  float4* part_o;           // [ctas][2][c / 4][kHeads] fp32, 4 channels each
  float2* part_ml;          // [ctas][2][kHeads] (m, l)
};

// First unit of CTA k, and the CTA that has unit u.
__device__ __forceinline__ int first_unit(const Args& a, int k) {
  return k * a.per_cta + (k < a.extra ? k : a.extra);
}
__device__ __forceinline__ int cta_of(const Args& a, int u) {
  const int long_ones = a.extra * (a.per_cta + 1);
  return u < long_ones ? u / (a.per_cta + 1) : a.extra + (u - long_ones) / a.per_cta;
}

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

// The CTA's units (items, if strided), and the next segment of them (t = -1 after the last).
__device__ __forceinline__ void cta_range(const Args& a, int* at, int* end) {
  const int cta = blockIdx.x;
  *at = a.strided ? cta : first_unit(a, cta);
  *end = a.strided ? a.items : first_unit(a, cta + 1);
}
__device__ __forceinline__ Seg next_segment(const Args& a, int* at, int end) {
  Seg q;
  q.t = -1;
  q.j0 = q.j1 = 0;
  if (*at >= end) return q;
  const int tpi = a.tiles_per_item;
  int item = *at, f0 = 0, f1 = tpi;
  if (a.strided) {
    *at += a.ctas;
  } else {
    item = *at / tpi;
    f0 = *at - item * tpi;
    if (end - *at < tpi - f0) f1 = f0 + end - *at;
    *at += f1 - f0;
  }
  q.part = (f0 == 0 && f1 == tpi) ? -1 : (f0 > 0 ? 0 : 1);
  q.item = item;
  q.t = item / a.groups;
  q.hg = item - static_cast<int>(q.t) * a.groups;
  const Query y = query_of(a.p, q.t);
  q.key_start = y.key_start;
  q.win_start = y.win_start;
  q.n_visible = y.n_visible;
  q.n1 = y.n1;
  q.n2 = y.n2;
  q.ok = y.ok;
  // a query shorter than the longest spreads its tiles over its CTAs alike
  const int nt = (y.n1 + y.n2 + kRows - 1) / kRows;
  q.j0 = f0 == 0 ? 0 : static_cast<int>(static_cast<int64_t>(f0) * nt / tpi);
  q.j1 = f1 == tpi ? nt : static_cast<int>(static_cast<int64_t>(f1) * nt / tpi);
  return q;
}

// ------------------------------------------------------------------ PTX

// TMEM <-> registers: 16 columns of a lane each (also tmem_ld16); tmem_ld_rows: 16 lanes x 64
// columns, lane i holding of rows i / 4 (v[4k], v[4k + 1]) and i / 4 + 8 (v[4k + 2], v[4k + 3])
// the columns 8k + 2 (i % 4) and the next.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"f"(v[0]),
      "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]),
      "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]),
      "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, "
      "%10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, "
      "%26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]),
        "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]),
        "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// 8 bytes, not kept in L1, which is small beside this much shared memory.  (No predicate: with
// one, and zeros otherwise, each load was waited for before the next.)
__device__ __forceinline__ uint2 ld_chunk(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "l"(p));
  return v;
}
// Two E4M3 bytes each (low, high half of w) as fp16 pairs, exactly.
__device__ __forceinline__ uint2 widen4(uint32_t w) {
  uint2 v;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(v.x), "=r"(v.y)
      : "r"(w));
  return v;
}
__device__ __forceinline__ void st_global32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void st_shared16(uint32_t addr, uint2 lo, uint2 hi) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(lo.x), "r"(lo.y),
               "r"(hi.x), "r"(hi.y)
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// Larger magnitude (as 16-bit patterns: NaN above infinity above the rest) in either half.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t top, uint32_t w) {
  return __vmaxu2(top, w & 0x7fff7fffu);
}
// A pair of bf16 values times a power of two, as fp16.
__device__ __forceinline__ uint32_t scale_narrow(uint32_t w, float mul) {
  const __half2 h =
      __floats2half2_rn(__uint_as_float(w << 16) * mul, __uint_as_float(w & 0xffff0000u) * mul);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 16 bytes from global to shared memory, asynchronously; zeros if not wanted.
__device__ __forceinline__ void copy_chunk(uint32_t dst, const void* p, bool want) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(p),
               "r"(want ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// Instruction descriptor of kind::f16: D fp32, A and B of one 16-bit type, A K-major, M = 64;
// bn: B MN-major.
__host__ __device__ constexpr uint32_t idesc(bool bf16, bool bn, int n) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (bn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(kHeads >> 4) << 24);
}

// Whether the phase of this parity has completed, after at most some ten microseconds in which
// the thread may sleep.
__device__ __forceinline__ bool try_wait_long(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(20000)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ uint32_t ticks() { return static_cast<uint32_t>(clock64() >> 16); }
// Whether the CTA has stood still for too long, or has been told to stop.  abort_flag[1]: the
// tick at which it last went on.
__device__ __forceinline__ bool gave_up(volatile int* abort_flag) {
  const uint32_t last = static_cast<uint32_t>(abort_flag[1]);
  // (signed: another warp may note a later tick than this thread's between the two reads)
  if (static_cast<int32_t>(ticks() - last) > static_cast<int32_t>(kWaitTicks)) {
    *abort_flag = 1;
    atomicOr(&g_attention_error, 1u);
  }
  return *abort_flag != 0;
}
// Bounded wait of a whole warp; one answer for its lanes.  (No function call: calls do not go
// with setmaxnreg.)
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity,
                                          volatile int* abort_flag) {
#pragma unroll 1
  for (uint32_t spins = 1; !__all_sync(0xffffffffu, try_wait_long(bar, parity)); ++spins)
    if (spins % 16 == 0 && __any_sync(0xffffffffu, gave_up(abort_flag))) return false;
  return true;
}
// The same for one thread.
__device__ __forceinline__ bool wait_thread(uint64_t* bar, uint32_t parity,
                                            volatile int* abort_flag) {
#pragma unroll 1
  for (uint32_t spins = 1; !try_wait_long(bar, parity); ++spins)
    if (spins % 16 == 0 && gave_up(abort_flag)) return false;
  return true;
}
// One lane of a converged warp, in the form the compiler knows to leave a single thread: the
// MMAs' descriptors then need no per-lane handling (a lane == 0 test made each issue 4 times
// as long).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(p));
  return p != 0;
}
// Channel of slot `s` (a multiple of 8) of the padded row; -1 for padding.
__device__ __forceinline__ int channel_of(const Args& a, int s) {
  const int cnp = a.na * 64;
  if (s < cnp) return s < a.cn ? s : -1;
  return s - cnp < a.p.r ? a.cn + s - cnp : -1;
}

// What the roles of a CTA share.
struct Shared {
  uint8_t* smem;
  uint64_t* bars;
  volatile int* abort_flag;
  uint32_t tmem;
  __device__ __forceinline__ const Seg& seg(uint32_t sn) const {
    return reinterpret_cast<const Seg*>(smem + kSmSeg)[sn % kSegs];
  }
  __device__ __forceinline__ bool wait(int bar, uint32_t parity) const {
    return wait_warp(bars + bar, parity, abort_flag);
  }
  // the CTA goes on (see the bounded waits)
  __device__ __forceinline__ void went_on() const { abort_flag[1] = static_cast<int>(ticks()); }
  // one arrival for a warp, after all its lanes got here
  __device__ __forceinline__ void arrive(int bar) const {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bars + bar);
  }
};

// ------------------------------------------------------------------ rows of a tile

// Walks the tiles of the CTA's segments for the warps that bring rows.  A lane has one row of
// every tile, whose number may still be on its way after next() (a listed entry's load).
struct RowCursor {
  uint32_t sn = 0;     // segment records read
  int j = 0, j1 = 0;   // next tile of the current segment
  int item = -1;       // query and head group of the tile; -1: no more tiles
  bool first = false;  // the tile begins its segment
  int kind = 0;        // 0 none, 1 listed, 2 cache row, 3 window row
  int raw = 0, listed = 0;

  // The next tile, `r` of its rows.
  __device__ __forceinline__ void next(const Args& a, const Shared& sh, int r) {
    first = false;
    while (j == j1) {  // the next segment with tiles
      item = -1;
      if (sn > 0) sh.arrive(kBSegEmpty + (sn - 1) % kSegs);
      if (!sh.wait(kBSegFull + sn % kSegs, (sn / kSegs) & 1u)) return;
      const Seg& q = sh.seg(sn);
      ++sn;
      if (q.t < 0) return;
      j = q.j0;
      j1 = q.j1;
      first = true;
    }
    const Seg& q = sh.seg(sn - 1);
    item = q.item;
    const int e = j * kRows + r;
    kind = e < q.n1 ? (a.p.idx ? 1 : 2) : e < q.n1 + q.n2 ? 3 : 0;
    raw = e < q.n1 ? e : e - q.n1;
    if (kind == 1) listed = __ldg(a.p.idx + q.t * a.p.k + e);  // (a select would wait for it)
    ++j;
  }
  // The row's number in its array (*win: the window's), -1 for one that does not count.  The
  // tile's segment record is still there: it is given back by the next() that leaves it.
  __device__ __forceinline__ int64_t row(const Shared& sh, bool* win) {
    const Seg& q = sh.seg(sn - 1);
    *win = kind == 3;
    if (kind == 0) return -1;
    if (kind == 1) {
      raw = listed;
      if (raw < 0 || raw >= q.n_visible) {
        if (raw != -1) atomicOr(&g_attention_error, 2u);
        return -1;
      }
    }
    return (kind == 3 ? q.win_start : q.key_start) + raw;
  }
};

// ------------------------------------------------------------------ FP8 gather (16 warps)

// Brings Q (once per segment) and the rows' FP8 channels (tile by tile) into shared memory as
// the MMAs read them: 128-byte rows of 64 16-bit channels, swizzled, widened to fp16.  Warp pw
// has rows [4 pw, 4 pw + 4) of a tile, a lane the 8-channel chunks lane and lane + 32 of each
// (a warp reads 256 consecutive bytes).  A tile's loads set out as soon as the registers of the
// tile before are stored; its rows are in L2 by then.  Bound by instructions: 16 warps that
// each found their own rows issued a third of 9900 instructions a tile for it (6450 now; 600 us
// on the chunk of 1024 queries x 1152 rows, 580 so).  (8 warps with 8 rows each took twice as
// long over a tile; a second set of registers, one tile further ahead, measured 584 us.)
__device__ __forceinline__ void gather(const Args& a, const Shared& sh) {
  uint8_t* smem = sh.smem;
  const int pw = (threadIdx.x >> 5) - kLoad0, lane = threadIdx.x & 31;
  const int lc = lane & 7, rsub = lane >> 3;
  const int na = a.na;
  // channels of this lane's two chunks (of padding: others, which meet zeros of Q and are not
  // stored to out)
  const int off0 = lane * 8 < a.cn ? lane * 8 : 0;
  const int off1 = 256 + lane * 8 < a.cn ? 256 + lane * 8 : 0;
  uint2 d[kOwn][2];
  auto load = [&](uint32_t gt) {
    if (!sh.wait(kBRowFull + (gt & 1u), (gt >> 1) & 1u)) return false;
    if (na > 0) {
      const ulonglong2* rows =
          reinterpret_cast<const ulonglong2*>(smem + kSmRow + (gt & 1u) * (kRows * 8)) + pw * 2;
      const ulonglong2 r01 = rows[0], r23 = rows[1];
      const uint8_t* p[kOwn] = {
          reinterpret_cast<const uint8_t*>(r01.x), reinterpret_cast<const uint8_t*>(r01.y),
          reinterpret_cast<const uint8_t*>(r23.x), reinterpret_cast<const uint8_t*>(r23.y)};
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        d[i][0] = ld_chunk(p[i] + off0);
        d[i][1] = ld_chunk(p[i] + off1);
      }
    }
    sh.arrive(kBRowEmpty + (gt & 1u));
    return true;
  };
  auto store = [&](uint32_t st) {
    uint8_t* kb = smem + kSmK + st * kStage + rsub * kAtom;
    if (na > 0) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const int rr = pw * kOwn + i;
        uint8_t* place = kb + rr * 128 + ((lc ^ (rr & 7)) << 4);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint2 lo = widen4(d[i][h].x), hi = widen4(d[i][h].y);
          if (h * 4 + rsub < na)
            *reinterpret_cast<uint4*>(place + h * 4 * kAtom) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
      }
    }
  };
  // Q of a segment: 4 rows per warp, FP8 channels to scaled fp16.
  auto q_rows = [&](int item, int* heads) {
    const int t = item / a.groups, hg = item - t * a.groups;
    *heads = a.p.H - hg * kHeads;
    return static_cast<const __nv_bfloat16*>(a.p.q) +
           (static_cast<int64_t>(t) * a.p.H + hg * kHeads) * a.p.c;
  };
  // Copied to its place as it is, then scaled and narrowed there: loops of a few instructions,
  // since all of it runs once a segment, from cold.
  auto load_q = [&](int item, uint32_t seg) {
    int heads;
    const __nv_bfloat16* qb = q_rows(item, &heads);
    const int blocks = na + a.nr;
    const int qc0 = rsub < blocks ? channel_of(a, lane * 8) : -1;
    const int qc1 = rsub + 4 < blocks ? channel_of(a, 256 + lane * 8) : -1;
    const uint32_t to = smem_u32(smem + kSmQ) + rsub * kAtom + pw * (kOwn * 128);
#pragma unroll 1
    for (int i = 0; i < kOwn; ++i) {
      const int rr = pw * kOwn + i;
      const uint32_t at0 = to + i * 128 + ((lc ^ (rr & 7)) << 4);
      const __nv_bfloat16* src = qb + rr * a.p.c;
      const bool want0 = rr < heads && qc0 >= 0, want1 = rr < heads && qc1 >= 0;
      if (rsub < blocks) copy_chunk(at0, want0 ? src + qc0 : a.p.q, want0);
      if (rsub + 4 < blocks) copy_chunk(at0 + 4 * kAtom, want1 ? src + qc1 : a.p.q, want1);
    }
    copies_done();
#pragma unroll 1
    for (int i = 0; i < kOwn; ++i) {
      const int rr = pw * kOwn + i;
      const uint32_t at0 = to + i * 128 + ((lc ^ (rr & 7)) << 4);
      uint4 v[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
      if (rsub < na) v[0] = ld_shared16(at0);
      if (rsub + 4 < na) v[1] = ld_shared16(at0 + 4 * kAtom);
      uint32_t top = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        top = max_abs_bf16x2(top, v[h].x);
        top = max_abs_bf16x2(top, v[h].y);
        top = max_abs_bf16x2(top, v[h].z);
        top = max_abs_bf16x2(top, v[h].w);
      }
      top = max(top & 0xffffu, top >> 16);
      int e = static_cast<int>(__reduce_max_sync(0xffffffffu, top) >> 7);
      if (e == 255) e = 142;  // an infinity or NaN: no scaling
      if (e < 16) e = 16;     // 2^(142 - e) stays finite
      if (lane == 0) smem[kSmExp + (seg % kExps) * kHeads + rr] = static_cast<uint8_t>(e);
      const float mul = __int_as_float((142 - e + 127) << 23);
      if (rsub < na)
        st_shared16(at0, make_uint2(scale_narrow(v[0].x, mul), scale_narrow(v[0].y, mul)),
                    make_uint2(scale_narrow(v[0].z, mul), scale_narrow(v[0].w, mul)));
      if (rsub + 4 < na)
        st_shared16(at0 + 4 * kAtom,
                    make_uint2(scale_narrow(v[1].x, mul), scale_narrow(v[1].y, mul)),
                    make_uint2(scale_narrow(v[1].z, mul), scale_narrow(v[1].w, mul)));
    }
  };

  uint32_t gt = 0, sn = 0, seg = 0;
  while (true) {
    if (!sh.wait(kBSegFull + sn % kSegs, (sn / kSegs) & 1u)) return;
    const Seg& q = sh.seg(sn);
    const int nt = q.j1 - q.j0, item = q.item;
    const bool end = q.t < 0;
    sh.arrive(kBSegEmpty + sn % kSegs);
    if (end) return;
    ++sn;
    for (int i = 0; i < nt; ++i, ++gt) {
      const uint32_t st = gt % kStages;
      if (!load(gt)) return;
      if (i == 0) {
        if (!sh.wait(kBQEmpty, (seg & 1u) ^ 1u)) return;
        load_q(item, seg);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        sh.arrive(kBQFull);
        ++seg;
      }
      if (!sh.wait(kBKEmpty + st, ((gt / kStages) & 1u) ^ 1u)) return;
      store(st);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      sh.arrive(kBKFull + st);
    }
  }
}

// ------------------------------------------------------------------ rows and bf16 copy (2 warps)

// A line of 64 channels after another of Q's row r: in L2 when its turn comes.
__device__ __forceinline__ void prefetch_q(const Args& a, int item, int r) {
  const int t = item / a.groups, head = (item - t * a.groups) * kHeads + r;
  if (head >= a.p.H) return;
  const __nv_bfloat16* q =
      static_cast<const __nv_bfloat16*>(a.p.q) + (static_cast<int64_t>(t) * a.p.H + head) * a.p.c;
#pragma unroll 1
  for (int c = 0; c < a.p.c; c += 64) prefetch_l2(q + c);
}

// Where a tile's rows begin, for the gather, two tiles ahead of it and with a prefetch into L2;
// and the rows' bf16 channels, which go to their place as they are.  A lane has one row of
// every tile and copies it, 16 bytes at a time, once the place is free.
__device__ __forceinline__ void copy_rows(const Args& a, const Shared& sh) {
  const int r = threadIdx.x & 63;  // (the two warps begin at a multiple of 64 threads)
  const int nr = a.nr;
  RowCursor cur;
  uint32_t known = 0, ahead = 0;  // tiles whose rows have been handed on; looked for
  // the row's bf16 channels in the next tiles to copy (nullptr: it does not count)
  const __nv_bfloat16 *s0 = nullptr, *s1 = nullptr, *s2 = nullptr;
  cur.next(a, sh, r);
  for (uint32_t gt = 0;; ++gt) {
#pragma unroll 1
    while (true) {
      s2 = nullptr;
      if (cur.item >= 0) {
        if (cur.first) prefetch_q(a, cur.item, r);
        bool win;
        const int64_t row = cur.row(sh, &win);
        const uint8_t* nope = g_zero_row;
        if (row >= 0) {
          if (a.cn > 0) {
            nope = static_cast<const uint8_t*>(win ? a.p.win_nope : a.p.nope) + row * a.cn;
#pragma unroll 1
            for (int c = 0; c < a.cn; c += 128) prefetch_l2(nope + c);
          }
          s2 = static_cast<const __nv_bfloat16*>(nr == 0 ? a.p.q
                                                         : win ? a.p.win_rope : a.p.rope) +
               row * a.p.r;
#pragma unroll 1
          for (int c = 0; c < a.p.r; c += 64) prefetch_l2(s2 + c);
        }
        const uint32_t b = known & 1u;
        if (!sh.wait(kBRowEmpty + b, ((known >> 1) & 1u) ^ 1u)) return;
        reinterpret_cast<const uint8_t**>(sh.smem + kSmRow)[b * kRows + r] = nope;
        sh.arrive(kBRowFull + b);
        ++known;
        cur.next(a, sh, r);
      }
      if (++ahead == gt + 3) break;
      s0 = s1;
      s1 = s2;
    }
    if (gt == known) return;
    const uint32_t st = gt % kStages;
    if (!sh.wait(kBKEmpty + st, ((gt / kStages) & 1u) ^ 1u)) return;
    const uint32_t live = __ballot_sync(0xffffffffu, s0 != nullptr);
    if ((r & 31) == 0) reinterpret_cast<uint32_t*>(sh.smem + kSmMask)[st * 2 + (r >> 5)] = live;
    const uint32_t dst = smem_u32(sh.smem + kSmK + st * kStage + a.na * kAtom) + r * 128;
#pragma unroll 1
    for (int k = 0; k < nr; ++k) {
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const bool want = s0 != nullptr && k * 64 + c * 8 < a.p.r;
        copy_chunk(dst + k * kAtom + ((c ^ (r & 7)) << 4), want ? s0 + k * 64 + c * 8 : a.p.q,
                   want);
      }
    }
    copies_done();
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    sh.arrive(kBKFull + st);
    if (r == 0) sh.went_on();
    s0 = s1;
    s1 = s2;
  }
}

// ------------------------------------------------------------------ softmax (4 warps)

// A thread has rows 16 w + lane / 4 and the one 8 below, 16 columns of each.  (8 warps, two to
// a row that exchange maxima, left the others too few registers and issue slots: 654 against
// 600 us on the chunk of 1024 queries x 1152 rows.)
__device__ __forceinline__ void softmax(const Args& a, const Shared& sh) {
  uint8_t* smem = sh.smem;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ra = w * 16 + (lane >> 2), q4 = lane & 3;
  const int na = a.na, nr = a.nr;
  const uint32_t lane_addr = sh.tmem + (static_cast<uint32_t>(w * 32) << 16);
  // the weights' place: 16-byte chunk k of row ra at chunk k ^ (ra % 8) of its 128 bytes
  uint8_t* prow = smem + kSmP + ra * 128 + q4 * 4;
  const float b_scale = a.p.scale * kLog2e;
  const float n_scale = b_scale / a.p.fp8_scale;
  uint32_t g = 0, seg = 0;  // tiles, segments with tiles
  for (uint32_t sn = 0;; ++sn) {
    if (!sh.wait(kBSegFull + sn % kSegs, (sn / kSegs) & 1u)) return;
    const Seg& q = sh.seg(sn);
    const bool end = q.t < 0;
    const int nt = q.j1 - q.j0;
    sh.arrive(kBSegEmpty + sn % kSegs);
    if (end) return;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, scale_n[2] = {0.f, 0.f};
#pragma unroll 1
    for (int i = 0; i < nt; ++i, ++g) {
      const uint32_t b = g & 1u, n = g >> 1, st = g % kStages;
      if (!sh.wait(kBSFull + b, n & 1u)) return;
      tc_fence_after();
      float x[32], u[32];
      const uint32_t sb = lane_addr + kColS + 64 * b;
      float2 (&x2)[16] = *reinterpret_cast<float2(*)[16]>(x);  // [2 k + row]: two columns
      const float2(&u2)[16] = *reinterpret_cast<const float2(*)[16]>(u);
      if (na > 0) {
        tmem_ld_rows(sb, x);
        if (nr > 0) tmem_ld_rows(sb + kUpper, u);
      } else {
        tmem_ld_rows(sb + kUpper, x);
      }
      // (complete since S is: for the mask's sight, while the loads are under way)
      const bool there = sh.wait(kBKFull + st, (g / kStages) & 1u);
      const uint2 live = *reinterpret_cast<const uint2*>(smem + kSmMask + st * 8);
      if (i == 0) {
        // x = S_n * (2^(E - 142) scale / fp8_scale) + S_r * scale, in units of log 2
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int e = smem[kSmExp + (seg % kExps) * kHeads + ra + 8 * r];
          scale_n[r] = n_scale * __int_as_float((e - 15) << 23);
        }
      }
      tmem_wait_ld();
      if (!there) return;
      if (na > 0 && nr > 0) {
#pragma unroll
        for (int c = 0; c < 16; ++c)
          x2[c] = f2_fma(x2[c], make_float2(scale_n[c & 1], scale_n[c & 1]),
                         f2_mul(u2[c], make_float2(b_scale, b_scale)));
      } else {
        const float f0 = na > 0 ? scale_n[0] : b_scale, f1 = na > 0 ? scale_n[1] : b_scale;
#pragma unroll
        for (int c = 0; c < 16; ++c)
          x2[c] = f2_mul(x2[c], c & 1 ? make_float2(f1, f1) : make_float2(f0, f0));
      }
      if ((live.x & live.y) != ~0u) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t two = (k < 4 ? live.x : live.y) >> (8 * (k & 3) + 2 * q4);
          if (!(two & 1u)) x[4 * k] = x[4 * k + 2] = -INFINITY;
          if (!(two & 2u)) x[4 * k + 1] = x[4 * k + 3] = -INFINITY;
        }
      }
      float ref[2], f[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float top = -INFINITY;
#pragma unroll
        for (int k = 0; k < 8; ++k) top = fmaxf(top, fmaxf(x[4 * k + 2 * r], x[4 * k + 2 * r + 1]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the reference: the running maximum, or up to kSlack below it.  (Weights formed at the
        // old reference beside this search, and again where it moves, measured 584 us against
        // 574 on the chunk of 1024 queries x 1152 rows.)
        const float m_new = i == 0 || top > m[r] + kSlack ? top : m[r];
        f[r] = m_new != m[r] ? ex2_ftz(m[r] - m_new) : 1.f;
        m[r] = m_new;
        ref[r] = (m_new == -INFINITY ? 0.f : m_new) - kBias;
      }
      if (i > 0 && __any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
        // O so far moves to the new reference, once the tile before this one is in it
        if (!sh.wait(kBPvDone + (b ^ 1u), ((g - 1) >> 1) & 1u)) return;
        tc_fence_after();
        l[0] *= f[0];
        l[1] *= f[1];
        const float fa = __shfl_sync(0xffffffffu, f[0], (lane & 7) * 4);
        const float fb = __shfl_sync(0xffffffffu, f[1], (lane & 7) * 4);
        const float fl = lane & 8 ? fb : fa;  // of row lane % 16
#pragma unroll 1
        for (int c0 = 0; c0 < 256; c0 += 16) {
          float v[16];
          tmem_ld16(lane_addr + c0, v);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 16; ++c) v[c] *= fl;
          tmem_st16(lane_addr + c0, v);
        }
        tmem_wait_st();
        tc_fence_before();
      }
      // (the weights of the tile two before this one have been used: its P K was issued before
      // S of this one, whose commit covers both)
      uint8_t* pb = prow + b * 2 * kAtom;
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int place = (k ^ (ra & 7)) << 4;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float2 p = f2_ex2(f2_sub(x2[2 * k + r], make_float2(ref[r], ref[r])));
          sum[r] = f2_add(sum[r], p);
          if (na > 0)
            *reinterpret_cast<__half2*>(pb + place + r * 1024) = __floats2half2_rn(p.x, p.y);
          if (nr > 0)
            *reinterpret_cast<uint32_t*>(pb + kAtom + place + r * 1024) = pack_bf16x2(p.x, p.y);
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) l[r] += sum[r].x + sum[r].y;
      tc_fence_before();
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      sh.arrive(kBPFull + b);
    }
    // the sums of the segment before this one have been read
    if (seg > 0 && !sh.wait(kBOFree, (seg - 1) & 1u)) return;
    float2* ml = reinterpret_cast<float2*>(smem + kSmMl);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (q4 == 0) ml[ra + 8 * r] = make_float2(m[r], l[r] * kUnbias);
    }
    sh.arrive(kBLFull + seg % kSegs);
    ++seg;
  }
}

// ------------------------------------------------------------------ store (4 warps)

// out and lse of a whole query, or the part's O, m and l.  A lane has row 16 w + lane % 16,
// channels below 256 (lanes 0-15) or above.
__device__ __forceinline__ void store_out_rows(const Args& a, const Shared& sh) {
  const int w = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const int row = w * 16 + (lane & 15), upper = lane >> 4;
  const uint32_t lane_addr = sh.tmem + (static_cast<uint32_t>(w * 32) << 16);
  const int slots = (a.na + a.nr) * 64;
  const float inv_fp8 = 1.f / a.p.fp8_scale;
  uint32_t g = 0, seg = 0;
  int at, end;
  cta_range(a, &at, &end);
  while (true) {
    const Seg q = next_segment(a, &at, end);
    const int64_t t = q.t;
    const int nt = q.j1 - q.j0, hg = q.hg, part = q.part;
    const bool ok = q.ok;
    if (t < 0) return;
    if (lane == 0) sh.went_on();
    if (!ok && w == 0 && lane == 0) atomicOr(&g_attention_error, 2u);
    float m = -INFINITY, l = 0.f;
    if (nt > 0) {
      g += nt;
      const uint32_t gl = g - 1;
      if (!sh.wait(kBLFull + seg % kSegs, (seg / kSegs) & 1u) ||
          !sh.wait(kBPvDone + (gl & 1u), (gl >> 1) & 1u))
        return;
      tc_fence_after();
      const float2 ml =
          reinterpret_cast<const float2*>(sh.smem + kSmMl)[row];
      m = ml.x;
      l = ml.y;
      ++seg;
    }
    const int head = hg * kHeads + row;
    const bool live = head < a.p.H && ok;
    float f_rope = kUnbias;
    if (part < 0) {
      const float sink = a.p.sink && live ? a.p.sink[head] : -INFINITY;
      const float sink2 = sink * kLog2e;
      const float M = fmaxf(m, sink2);
      float f = 0.f, den = 0.f;
      if (M != -INFINITY) {
        f = ex2_ftz(m - M);
        den = l * f + (a.p.sink ? ex2_ftz(sink2 - M) : 0.f);
      } else if (l != l) {
        f = den = l;  // NaN scores only
      }
      f_rope = den != 0.f ? f / den * kUnbias : 0.f;
      if (upper == 0 && live && a.p.lse)
        a.p.lse[t * a.p.H + head] =
            m == -INFINITY && l == 0.f  // no row: the sink's logit as it is
                ? sink
                : (M == -INFINITY ? 0.f : M) * 0.6931471805599453f + logf(den);
    } else if (upper == 0 && live) {
      a.part_ml[(blockIdx.x * 2 + part) * kHeads + row] = make_float2(m, l);
    }
    const float f_nope = f_rope * inv_fp8;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.p.out) + (t * a.p.H + head) * a.p.c;
    // (a part lies with its rows side by side, as the lanes have them)
    float4* po = a.part_o +
                 static_cast<int64_t>(blockIdx.x * 2 + (part > 0 ? 1 : 0)) * (a.p.c / 4) * kHeads +
                 row;
    const bool wide = a.wide_out;
    if (nt == 0 && part >= 0) continue;
#pragma unroll 1
    for (int c0 = 0; c0 < 256 && c0 < slots; c0 += 16) {
      float v[16];
      __syncwarp();
      if (nt > 0) {
        tmem_ld16(lane_addr + c0, v);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int c = 0; c < 16; ++c) v[c] = 0.f;
      }
      const int s0 = upper * 256 + c0;
      if (!live || s0 >= slots) continue;
      const float f = s0 < a.na * 64 ? f_nope : f_rope;
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] *= f;
      const int ch = channel_of(a, s0), ch8 = channel_of(a, s0 + 8);
      if (part < 0) {
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
        if (wide && ch8 >= 0) {  // a whole 32-byte sector: twice as fast as two halves
          st_global32(out + ch, o);
        } else {
          if (ch >= 0) *reinterpret_cast<uint4*>(out + ch) = make_uint4(o[0], o[1], o[2], o[3]);
          if (ch8 >= 0) *reinterpret_cast<uint4*>(out + ch8) = make_uint4(o[4], o[5], o[6], o[7]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const int c4 = e < 8 ? ch : ch8;
          if (c4 >= 0)
            po[static_cast<int64_t>(c4 / 4 + (e & 4) / 4) * kHeads] =
                make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
      }
    }
    if (nt > 0) {
      tc_fence_before();
      sh.arrive(kBOFree);
    }
  }
}

// ------------------------------------------------------------------ MMA issue (one thread)

__device__ __forceinline__ void issue_mmas(const Args& a, const Shared& sh) {
  uint64_t* bars = sh.bars;
  const uint32_t tmem = sh.tmem;
  const int na = a.na, blocks = a.na + a.nr;
  const int lo = blocks < 4 ? blocks : 4, hi = blocks - lo;     // blocks below / above 256
  const int na_lo = na < lo ? na : lo, na_hi = na - na_lo;
  const int nr_lo = lo - na_lo, nr_hi = hi - na_hi;
  const uint64_t qd = smem_desc(smem_u32(sh.smem + kSmQ), 16, 1024, 2);
  const uint64_t kd = smem_desc(smem_u32(sh.smem + kSmK), 16, 1024, 2);     // K-major (S)
  const uint64_t vd = smem_desc(smem_u32(sh.smem + kSmK), kAtom, 1024, 2);  // MN-major (P K)
  const uint64_t pd = smem_desc(smem_u32(sh.smem + kSmP), 16, 1024, 2);
  const uint32_t is_n = idesc(false, false, kRows), is_r = idesc(true, false, kRows);
  auto wait = [&](int bar, uint32_t parity) {
    return wait_thread(bars + bar, parity, sh.abort_flag);
  };
  uint32_t sn = 0;                // segment records read
  int j = 0, j1 = 0;              // tiles of the current segment
  bool ended = false, first = false;
  uint32_t s = 0, pv = 0;         // tiles whose S / P K has been issued
  uint32_t s_seg = 0, pv_seg = 0; // segments begun
  uint32_t first_bits = 0;        // tile & 1: first of its segment
  // Two S, then the two P K: while the softmax of one tile runs the tensor cores have the
  // other, and a tile's place in the ring is refilled during the second P K.  A segment's
  // first S waits for its Q, so what is pending goes first.  (Polling for whichever can go
  // measured 607 against 600 us on the chunk of 1024 queries x 1152 rows.)
  bool ok = true;
  while (ok) {
    while (ok && s < pv + 2) {
      if (j == j1) {
        while (ok && !ended && j == j1) {
          ok = wait(kBSegFull + sn % kSegs, (sn / kSegs) & 1u);
          if (!ok) break;
          const Seg& q = sh.seg(sn);
          j = q.j0;
          j1 = q.j1;
          ended = q.t < 0;
          mbar_arrive(bars + kBSegEmpty + sn % kSegs);
          ++sn;
        }
        first = true;
      }
      if (!ok || ended || (first && pv < s)) break;
      const uint32_t b = s & 1u, st = s % kStages;
      ok = (!first || wait(kBQFull, s_seg & 1u)) &&
           wait(kBKFull + st, (s / kStages) & 1u);
      if (!ok) break;
      tc_fence_after();  // (S of the tile two before has been read: its weights were there)
      const uint32_t dt = tmem + kColS + 64 * b;
#pragma unroll 1
      for (int at = 0; at < blocks; ++at) {
        const bool r = at >= na;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          umma_bf16(dt + (r ? kUpper : 0u), qd + ((at * kAtom + ks * 32) >> 4),
                    kd + ((st * kStage + at * kAtom + ks * 32) >> 4), r ? is_r : is_n,
                    ((at != 0 && at != na) || ks > 0) ? 1u : 0u);
      }
      umma_commit(bars + kBSFull + b);
      first_bits = (first_bits & ~(1u << b)) | ((first ? 1u : 0u) << b);
      if (first) ++s_seg;
      first = false;
      ++s;
      if (++j == j1) umma_commit(bars + kBQEmpty);
    }
    if (ok && ended && pv == s) break;
    while (ok && pv < s) {
      const uint32_t b = pv & 1u, st = pv % kStages;
      const bool begins = (first_bits >> b) & 1u;
      ok = wait(kBPFull + b, (pv >> 1) & 1u) &&
           (!begins || pv_seg == 0 || wait(kBOFree, (pv_seg - 1) & 1u));
      if (!ok) break;
      tc_fence_after();
      const uint64_t pn = pd + ((b * 2 * kAtom) >> 4), pr = pn + (kAtom >> 4);
#pragma unroll 1
      for (int ks = 0; ks < kRows / 16; ++ks) {
        const uint64_t d = vd + ((st * kStage + ks * 16 * 128) >> 4);
        const uint64_t an = pn + ((ks * 32) >> 4), ar = pr + ((ks * 32) >> 4);
        const uint32_t acc = (!begins || ks > 0) ? 1u : 0u;
        if (na_lo > 0) umma_bf16(tmem, an, d, idesc(false, true, na_lo * 64), acc);
        if (nr_lo > 0)
          umma_bf16(tmem + na_lo * 64, ar, d + ((na_lo * kAtom) >> 4),
                    idesc(true, true, nr_lo * 64), acc);
        if (na_hi > 0)
          umma_bf16(tmem + kUpper, an, d + ((4 * kAtom) >> 4), idesc(false, true, na_hi * 64), acc);
        if (nr_hi > 0)
          umma_bf16(tmem + kUpper + na_hi * 64, ar, d + (((4 + na_hi) * kAtom) >> 4),
                    idesc(true, true, nr_hi * 64), acc);
      }
      umma_commit(bars + kBKEmpty + st);
      if (begins) ++pv_seg;
      ++pv;
    }
  }
  umma_commit(bars + kBFinal);  // every MMA issued above has finished before TMEM is freed
  for (const uint32_t t0 = ticks(); !try_wait_long(bars + kBFinal, 0) && ticks() - t0 < kWaitTicks;) {
  }
}

// ------------------------------------------------------------------ scheduler (one thread)

__device__ __forceinline__ void schedule(const Args& a, const Shared& sh) {
  Seg* segs = reinterpret_cast<Seg*>(sh.smem + kSmSeg);
  int at, end;
  cta_range(a, &at, &end);
  for (uint32_t sn = 0;; ++sn) {
    Seg q;
    do {
      q = next_segment(a, &at, end);
      sh.went_on();
    } while (q.t >= 0 && q.j0 == q.j1);
    if (!wait_thread(sh.bars + kBSegEmpty + sn % kSegs, ((sn / kSegs) & 1u) ^ 1u, sh.abort_flag))
      return;
    segs[sn % kSegs] = q;
    mbar_arrive(sh.bars + kBSegFull + sn % kSegs);
    if (q.t < 0) return;
  }
}

// ------------------------------------------------------------------ the kernel

// What the CTA's first segment needs, on its way into L2 while the CTA sets up: its query's row
// range, its Q, the list entries of its first tiles.
__device__ __forceinline__ void prefetch_first(const Args& a) {
  int item = blockIdx.x, tile = 0;
  if (!a.strided) {
    const int u = first_unit(a, blockIdx.x);
    item = u / a.tiles_per_item;
    tile = u - item * a.tiles_per_item;
  }
  if (item >= a.items) return;
  const int64_t t = item / a.groups;
  const int hg = item - static_cast<int>(t) * a.groups;
  const int i = threadIdx.x;
  if (i == 0) prefetch_l2(a.p.key_start + t);
  if (i == 1) prefetch_l2(a.p.n_visible + t);
  if (a.p.win_start) {
    if (i == 2) prefetch_l2(a.p.win_start + t);
    if (i == 3) prefetch_l2(a.p.win_len + t);
  }
  if (i >= 32 && i < 40 && a.p.idx) {
    const int64_t e = static_cast<int64_t>(tile) * kRows + (i - 32) * 32;
    if (e < a.p.k) prefetch_l2(a.p.idx + t * a.p.k + e);
  }
  // threads 64 .. : a row each 8, 64 channels a thread
  const int row = (i - 64) >> 3, ch = (i & 7) * 64;
  if (i >= 64 && row < kHeads && hg * kHeads + row < a.p.H && ch < a.p.c)
    prefetch_l2(static_cast<const __nv_bfloat16*>(a.p.q) + (t * a.p.H + hg * kHeads + row) * a.p.c +
                ch);
}

__global__ void __launch_bounds__(kThreads, 1) attention_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  griddep_launch_dependents();  // the join, which waits for this grid's end before it reads
  if ((smem_u32(smem) & 1023u) != 0) {  // the 128-byte swizzle counts on it
    if (threadIdx.x == 0) atomicOr(&g_attention_error, 1u);
    return;
  }
  prefetch_first(a);
  Shared sh;
  sh.smem = smem;
  sh.bars = reinterpret_cast<uint64_t*>(smem + kSmBars);
  sh.abort_flag = reinterpret_cast<volatile int*>(smem + kSmMisc + 4);
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + kSmMisc);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t count = 1;  // commits, the scheduler
      if (i >= kBKFull && i < kBKFull + kStages) count = kLoadWarps + 2;
      if (i == kBQFull) count = kLoadWarps;
      if (i >= kBPFull && i < kBPFull + 2) count = kSoftWarps;
      if (i == kBOFree) count = kStoreWarps;
      if (i >= kBLFull && i < kBLFull + kSegs) count = kSoftWarps;
      if (i >= kBSegEmpty && i < kBSegEmpty + kSegs) count = kMmaWarp + 3 - kStoreWarps;
      if (i >= kBRowFull && i < kBRowFull + 2) count = 2;
      if (i >= kBRowEmpty && i < kBRowEmpty + 2) count = kLoadWarps;
      mbar_init(sh.bars + i, count);
    }
    *sh.abort_flag = 0;
    sh.went_on();
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
  tc_fence_after();
  sh.tmem = *tmem_slot;

  if (warp < kSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    softmax(a, sh);
  } else if (warp < kLoad0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kStoreRegs));
    store_out_rows(a, sh);
  } else if (warp < kMmaWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
    gather(a, sh);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
    if (warp == kMmaWarp) {
      if (elect_one()) issue_mmas(a, sh);
    } else if (warp == kMmaWarp + 1) {
      if (elect_one()) schedule(a, sh);
    } else {
      copy_rows(a, sh);
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem), "r"(512));
  }
}

// ------------------------------------------------------------------ joining the parts

// A query (of one group of heads) whose units lie in several CTAs has that many parts to join:
//     out = sum_p 2^(m_p - M) O_p / D,  D = sum_p 2^(m_p - M) l_p (+ sink),  M = max m_p,
// in an order that the plan alone fixes.  A query with few parts takes a warp for each of its
// heads, one with many a block of 8 groups of 128 threads that take every eighth part.  Bound
// by the parts' bytes (fp32, from L2 as a rule) and by three dependent round trips, so all of
// it should be resident at once.  (A block for every head of every CTA boundary, most of
// them idle, took 26 to 40 us.)
constexpr int kMaxParts = 160;  // CTAs, with room
// Parts up to which a warp takes them one after the other (at most 16, two lanes for each): 64
// queries split in two 267 us so and 380 with a block a head pair; 5 parts 21.6 and 18.4, 3 to
// 9 parts 26.7 and 21.3.
constexpr int kFewParts = 4;
constexpr int kJoinWarps = 4;

struct Split {
  int kf, parts;    // first CTA, number of parts
  int64_t t;
  int hg;
  bool ok;
};
// The x-th query that may be split: with fewer queries than CTAs the x-th one, else the one that
// CTA x ends in and CTA x + 1 goes on with, if CTA x is its first.
__device__ __forceinline__ Split split_of(const Args& a, int x) {
  const int tpi = a.tiles_per_item;
  Split s;
  s.ok = false;
  int item = x;
  if (a.items >= a.ctas) {
    const int lo = first_unit(a, x + 1);
    item = lo / tpi;
    if (lo == item * tpi) return s;
  }
  s.kf = cta_of(a, item * tpi);
  if (a.items >= a.ctas && s.kf != x) return s;
  s.parts = cta_of(a, item * tpi + tpi - 1) - s.kf + 1;
  s.t = item / a.groups;
  s.hg = item - static_cast<int>(s.t) * a.groups;
  s.ok = s.parts > 1 && query_of(a.p, s.t).ok;
  return s;
}
// Part p of the workspace: slot 1 of the first CTA, slot 0 of the others.
__device__ __forceinline__ int64_t part_slot(const Split& s, int p) {
  return static_cast<int64_t>(s.kf + p) * 2 + (p == 0 ? 1 : 0);
}
// Weight of a part with maximum m and sum l: a part without a row has l = 0, and its O is not
// written; NaN scores leave l NaN, and perhaps m = -inf.
__device__ __forceinline__ float part_weight(float2 ml, float ref) {
  return ml.y == 0.f ? 0.f : ml.y != ml.y ? ml.y : ex2_ftz(ml.x - ref);
}
__device__ __forceinline__ float4 fma4(float4 v, float w, float4 o) {
  return make_float4(fmaf(v.x, w, o.x), fmaf(v.y, w, o.y), fmaf(v.z, w, o.z), fmaf(v.w, w, o.w));
}
__device__ __forceinline__ void store4(const Args& a, int64_t out_row, int ch, float4 o, float inv) {
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.p.out) + out_row * a.p.c + ch) =
      make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
}
__device__ __forceinline__ void store_lse(const Args& a, int64_t out_row, bool any, float sink,
                                          float ref, float den) {
  if (a.p.lse) a.p.lse[out_row] = any ? ref * 0.6931471805599453f + logf(den) : sink;
}

// A warp for two heads and 256 channels: lane i has head i % 2 and 4 of every 64 channels.
__global__ void __launch_bounds__(32 * kJoinWarps) attention_join_few_kernel(const Args a) {
  __shared__ Split sp;
  griddep_wait();  // the parts are complete
  if (threadIdx.x == 0) sp = split_of(a, blockIdx.x);
  __syncthreads();
  const int lane = threadIdx.x & 31, q4 = lane >> 1;
  const int row0 = (blockIdx.y * kJoinWarps + (threadIdx.x >> 5)) * 2, row = row0 + (lane & 1);
  if (!sp.ok || sp.hg * kHeads + row0 >= a.p.H) return;
  const int head = sp.hg * kHeads + row;
  const bool live = head < a.p.H;  // (an odd number of heads)
  const int parts = sp.parts;      // at most kFewParts
  const int64_t out_row = sp.t * a.p.H + head;
  const float sink = a.p.sink && live ? a.p.sink[head] : -INFINITY;
  // lane 2 p + (head % 2) has part p's m and l
  float2 ml = make_float2(-INFINITY, 0.f);
  if (q4 < parts) ml = a.part_ml[part_slot(sp, q4) * kHeads + row];
  float M = ml.x;
#pragma unroll
  for (int o = 16; o > 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  M = fmaxf(M, sink * kLog2e);
  const float ref = M == -INFINITY ? 0.f : M;
  const float w = part_weight(ml, ref);
  float den = ml.y == 0.f ? 0.f : w * ml.y;
  float any = ml.y == 0.f ? 0.f : 1.f;
#pragma unroll
  for (int o = 16; o > 1; o >>= 1) {
    den += __shfl_xor_sync(0xffffffffu, den, o);
    any += __shfl_xor_sync(0xffffffffu, any, o);
  }
  if (a.p.sink) den += ex2_ftz(sink * kLog2e - ref);
  if (lane < 2 && live && blockIdx.z == 0) store_lse(a, out_row, any != 0.f, sink, ref, den);
  const float inv = den != 0.f ? 1.f / den : 0.f;
  const int quads = static_cast<int>(a.p.c) / 4, c0 = blockIdx.z * 64 + q4;
  float4 o[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int p = 0; p < parts; ++p) {
    const float wp = __shfl_sync(0xffffffffu, w, 2 * p + (lane & 1));
    const float4* src = a.part_o + part_slot(sp, p) * quads * kHeads + row;
    float4 v[4];
    // (a part of weight 0 adds nothing, and perhaps was not written)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      v[q] = wp != 0.f && c0 + q * 16 < quads ? src[static_cast<int64_t>(c0 + q * 16) * kHeads]
                                              : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = fma4(v[q], wp, o[q]);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (live && c0 + q * 16 < quads) store4(a, out_row, (c0 + q * 16) * 4, o[q], inv);
}

// A block for two heads and 256 channels: thread i has head i % 2 and 4 channels.
constexpr int kJoinGroups = 8;
__global__ void __launch_bounds__(128 * kJoinGroups) attention_join_many_kernel(const Args a) {
  constexpr int G = kJoinGroups;
  __shared__ Split sp;
  __shared__ float weight[2][kMaxParts], red[3][2][4 * G];
  __shared__ float4 sums[G - 1][128];
  const int tid = threadIdx.x, odd = tid & 1;
  griddep_wait();  // the parts are complete
  if (tid == 0) sp = split_of(a, blockIdx.x);
  __syncthreads();
  const int row = blockIdx.y * 2 + odd, head = sp.hg * kHeads + row;
  if (!sp.ok || head - odd >= a.p.H) return;
  const bool live = head < a.p.H;
  const int parts = sp.parts;
  const int64_t out_row = sp.t * a.p.H + head;
  const float sink = a.p.sink && live ? a.p.sink[head] : -INFINITY;
  // every part's m and l at once (there are fewer than half as many parts as threads)
  float2 ml = make_float2(-INFINITY, 0.f);
  if (tid / 2 < parts) ml = a.part_ml[part_slot(sp, tid / 2) * kHeads + row];
  float M = ml.x;
#pragma unroll
  for (int o = 16; o > 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if ((tid & 31) < 2) red[0][odd][tid >> 5] = M;
  __syncthreads();
  M = sink * kLog2e;
#pragma unroll
  for (int w = 0; w < 4 * G; ++w) M = fmaxf(M, red[0][odd][w]);
  const float ref = M == -INFINITY ? 0.f : M;
  const float wt = part_weight(ml, ref);
  if (tid / 2 < parts) weight[odd][tid / 2] = wt;
  float den = ml.y == 0.f ? 0.f : wt * ml.y;
  float any = ml.y == 0.f ? 0.f : 1.f;
#pragma unroll
  for (int o = 16; o > 1; o >>= 1) {
    den += __shfl_xor_sync(0xffffffffu, den, o);
    any += __shfl_xor_sync(0xffffffffu, any, o);
  }
  if ((tid & 31) < 2) {
    red[1][odd][tid >> 5] = den;
    red[2][odd][tid >> 5] = any;
  }
  __syncthreads();
  den = a.p.sink ? ex2_ftz(sink * kLog2e - ref) : 0.f;
  any = 0.f;
#pragma unroll
  for (int w = 0; w < 4 * G; ++w) {
    den += red[1][odd][w];
    any += red[2][odd][w];
  }
  if (tid < 2 && live && blockIdx.z == 0) store_lse(a, out_row, any != 0.f, sink, ref, den);
  const float inv = den != 0.f ? 1.f / den : 0.f;
  const int g = tid >> 7, lane = tid & 127;
  const int quads = static_cast<int>(a.p.c) / 4, c4 = blockIdx.z * 64 + (lane >> 1);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c4 < quads) {
#pragma unroll 8
    for (int p = g; p < parts; p += G) {
      const float w = weight[odd][p];
      const float4 v = w != 0.f ? a.part_o[(part_slot(sp, p) * quads + c4) * kHeads + row]
                                : make_float4(0.f, 0.f, 0.f, 0.f);
      o = fma4(v, w, o);
    }
  }
  if (g > 0) sums[g - 1][lane] = o;
  __syncthreads();
  if (g == 0 && live && c4 < quads) {
#pragma unroll
    for (int i = 0; i < G - 1; ++i) o = fma4(sums[i][lane], 1.f, o);
    store4(a, out_row, c4 * 4, o, inv);
  }
}

// ------------------------------------------------------------------ launch

constexpr int kMaxCtas = 148;        // SMs: one CTA each
static_assert(kMaxCtas <= kMaxParts, "a query may be split among all CTAs");
// Tiles of a part at least, however few the queries (512 + 128 rows, one query: 18.4 us with 2,
// 29.0 with 1, 22.0 with 3), and more in long queries, whose join takes longer the more parts
// there are (8320 rows, one query of two groups: 32.0 us with 2, 30.0 with 3).
constexpr int kMinTiles = 2;
int least_tiles(int tiles_per_item) {
  int n = kMinTiles;
  while (16 * n * n < tiles_per_item) ++n;  // sqrt(tiles) / 4
  return n;
}
// Queries go whole, CTA by CTA, where the CTAs that get one less wait for few tiles.  Splitting
// evens that out but costs the parts' way through memory and the join, 20 to 25 us: with 128
// queries of 1152 rows (256 items, idle for 5 tiles on average) 96 us whole and 102 split, with
// 700 (9.7 tiles) 422 either way, with 300 (17 tiles) 214 whole and 199 split.
// Both ways count tiles by the longest length.  Of 64 queries of 1329 to 8320 rows x 128 heads
// (265 us) the fullest CTA has 113 tiles where the mean is 66.5; of one query of 100000 rows and
// 73 of 1000 x 128 heads, which go whole, 1563 where the mean is 37.
constexpr int64_t kIdleTiles = 8;

struct Plan {
  int64_t items, units;
  int tiles_per_item, groups, ctas;
  bool strided;
};
Plan plan_of(int64_t T, int H, int64_t most, int max_ctas) {
  Plan p;
  p.groups = static_cast<int>(ceil_div(H, kHeads));
  p.items = T * p.groups;
  p.tiles_per_item = most > 0 ? static_cast<int>(ceil_div(most, kRows)) : 1;
  p.units = p.items * p.tiles_per_item;
  // (decided for the full machine, as the workspace is; unit numbers are 32-bit)
  const int64_t idle = (ceil_div(p.items, kMaxCtas) * kMaxCtas - p.items) * p.tiles_per_item;
  p.strided = idle <= kIdleTiles * kMaxCtas || p.units > 0x7fffffff - 2 * kMaxCtas;
  if (p.strided) {
    p.ctas = static_cast<int>(p.items < max_ctas ? p.items : max_ctas);
  } else {
    int64_t c = p.units / least_tiles(p.tiles_per_item);
    if (c < p.items) c = p.items;
    p.ctas = static_cast<int>(c < max_ctas ? c : max_ctas);
  }
  return p;
}
int64_t ml_bytes(int ctas) { return int64_t(ctas) * 2 * kHeads * sizeof(float2); }

}  // namespace attn

int64_t attention_workspace_bytes(int64_t T, int H, int64_t c, int, int64_t most) {
  using namespace attn;
  const Plan p = plan_of(T, H, most, kMaxCtas);
  if (p.strided || p.tiles_per_item == 1) return 0;  // no query is split
  return ml_bytes(p.ctas) + int64_t(p.ctas) * 2 * kHeads * c * 4;
}

kvc_status launch_attention(const AttentionProblem& p, cudaStream_t st) {
  using namespace attn;
  if (!raise_smem_limit(reinterpret_cast<const void*>(attention_kernel))) return KVC_ERR_CUDA;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return KVC_ERR_CUDA;
  const int sms = device_info(dev).sms;
  if (sms < 1) return KVC_ERR_CUDA;
  const int64_t most = (p.idx ? p.k : p.max_visible) + (p.win_start ? p.max_win : 0);
  const Plan pl = plan_of(p.T, p.H, most, sms < kMaxCtas ? sms : kMaxCtas);
  Args a{};
  a.p = p;
  a.items = static_cast<int>(pl.items);
  if (!pl.strided) {
    a.per_cta = static_cast<int>(pl.units / pl.ctas);
    a.extra = static_cast<int>(pl.units % pl.ctas);
  }
  a.wide_out = reinterpret_cast<uintptr_t>(p.out) % 32 == 0 && p.c % 16 == 0 && p.r % 16 == 0;
  a.tiles_per_item = pl.tiles_per_item;
  a.groups = pl.groups;
  a.ctas = pl.ctas;
  a.strided = pl.strided;
  a.cn = static_cast<int>(p.c) - p.r;
  a.na = (a.cn + 63) / 64;
  a.nr = (p.r + 63) / 64;
  a.part_ml = static_cast<float2*>(p.workspace);
  a.part_o = reinterpret_cast<float4*>(static_cast<uint8_t*>(p.workspace) + ml_bytes(pl.ctas));
  attention_kernel<<<pl.ctas, kThreads, kSmem, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return KVC_ERR_CUDA;
  const bool whole = pl.units % pl.ctas == 0 && (pl.units / pl.ctas) % pl.tiles_per_item == 0;
  if (!pl.strided && !whole && pl.tiles_per_item > 1) {  // some query is split
    // launched as a programmatic dependent: it may set up while the parts are still made
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    const int rows = p.H < kHeads ? p.H : kHeads;
    const int64_t splits = pl.items < pl.ctas ? pl.items : pl.ctas - 1;
    // the most CTAs a query's units can lie in
    const int64_t parts = (pl.tiles_per_item - 2) / (pl.units / pl.ctas) + 2;
    const bool few = parts <= kFewParts;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(splits),
                       static_cast<unsigned>(few ? ceil_div(rows, 2 * kJoinWarps) : ceil_div(rows, 2)),
                       static_cast<unsigned>(ceil_div(p.c, 256)));
    cfg.blockDim = dim3(few ? 32 * kJoinWarps : 128 * kJoinGroups, 1, 1);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, few ? attention_join_few_kernel : attention_join_many_kernel, a) !=
        cudaSuccess)
      return KVC_ERR_CUDA;
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
