// Partial rotary positions on sm_100a: the last r of c channels of x [T, H, c], one position
// per token, forward or inverse, interleaved or half layout (include/kvc.h, partial_rope),
// and the host-side frequency table scaled for long contexts (kvc_rope_frequencies).
//
// Per token the r / 2 angles are shared by all H heads, so a CTA forms each (cos, sin) once in
// shared memory (angle and reduction in fp64, fp32's rest of the angle put back: within 1.84
// units in the last place of the angle's own) and applies it to
// every head it handles; the rotation itself is 3 flops a value, so the kernel is bound by
// memory traffic (long calls) or by launch and one dependent round trip (short ones).  A unit
// is one vector of up to 16 bytes (half layout: the vector and its partner r / 2 channels on);
// every thread has all its kUnits loads in flight before the angles are formed.  Measured:
// 4096 x 128 heads, r = 64 of c = 512 in place (134 MB, 128 of every 1024 bytes) 29.0 us, 0.71 of
// the copy bandwidth (1, 2 and 8 units a thread: 36.8, 29.0, 31.4; streaming loads and stores
// 28.8).  What the 128-byte pieces cost in that is not known apart: between events, with cold
// inputs, the call takes 32.8 us, an elementwise pass of torch in place over as many bytes in one
// piece 27.4, and over the same pieces 41.8.  128 x 128 heads 3.2 us and one token 2.6 us, a
// launch and its round trip; fp32 777 x 24 heads of 192 (29 MB, out of place) 7.0 us against 4.4
// at the copy bandwidth.
#include <math.h>

#include "kvc_common.cuh"
#include "kvc_host.h"
#include "kvc_launch.h"

namespace kvc {
namespace rope {

constexpr int kThreads = 256;
constexpr int kUnits = 4;          // units per thread
constexpr int kMaxPairs = 2048;    // (cos, sin) pairs a CTA keeps (16 KB)

struct Args {
  const void* x;
  void* out;
  const int64_t* pos;
  const float* inv_freq;
  int64_t T, c, chunks;  // chunks of one token's units (1 when a CTA takes whole tokens)
  int H, r, tokens;      // tokens per CTA (1 when chunks > 1)
  int copy_units, rot_units;  // units of one head: copied, rotated
  float magnitude, sign;
};

template <int BYTES>
struct Vec;
template <>
struct Vec<16> {
  using T = uint4;
};
template <>
struct Vec<8> {
  using T = uint2;
};

template <typename E, int N>
union Pack {
  typename Vec<sizeof(E) * N>::T v;
  E e[N];
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float* d, float v) { *d = v; }
__device__ __forceinline__ void from_f(__nv_bfloat16* d, float v) { *d = __float2bfloat16_rn(v); }

// E: element type, N: elements per unit vector, HALF: pairs (j, j + r/2) instead of (2j, 2j+1).
template <typename E, int N, bool HALF>
__global__ void __launch_bounds__(kThreads) partial_rope_kernel(const Args a) {
  extern __shared__ float2 cs[];  // [tokens][r / 2] (cos, sin), times the magnitude
  using P = Pack<E, N>;
  const int64_t tok0 = a.chunks > 1 ? blockIdx.x / a.chunks : blockIdx.x * int64_t(a.tokens);
  const int64_t chunk = a.chunks > 1 ? blockIdx.x - tok0 * a.chunks : 0;
  const int ntok = static_cast<int>(a.T - tok0 < a.tokens ? a.T - tok0 : a.tokens);
  const int per_head = a.copy_units + a.rot_units;
  const int64_t per_tok = int64_t(a.H) * per_head;
  const int64_t end = a.chunks > 1 ? per_tok : ntok * per_tok;
  const E* x = static_cast<const E*>(a.x) + tok0 * a.H * a.c;
  E* out = static_cast<E*>(a.out) + tok0 * a.H * a.c;
  const int64_t cn = a.c - a.r;

  P v[kUnits], w[kUnits];
  int64_t at[kUnits];
  int pair[kUnits];  // first (cos, sin) pair of the unit, -1: copied, -2: none
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int64_t u = chunk * (kThreads * kUnits) + i * kThreads + threadIdx.x;
    pair[i] = -2;
    if (u < end) {
      const uint32_t uu = static_cast<uint32_t>(u);  // at most tokens * H * c / N < 2^31
      const uint32_t row = uu / per_head;            // (token, head) within the CTA's tokens
      const int k = static_cast<int>(uu - row * per_head);
      if (k < a.copy_units) {
        pair[i] = -1;
        at[i] = row * a.c + k * N;
        v[i].v = *reinterpret_cast<const decltype(v[i].v)*>(x + at[i]);
      } else {
        const int q = k - a.copy_units;
        at[i] = row * a.c + cn + q * N;
        pair[i] = static_cast<int>(row / a.H) * (a.r / 2) + q * (HALF ? N : N / 2);
        v[i].v = *reinterpret_cast<const decltype(v[i].v)*>(x + at[i]);
        if constexpr (HALF)
          w[i].v = *reinterpret_cast<const decltype(w[i].v)*>(x + at[i] + a.r / 2);
      }
    }
  }
  const int np = a.r / 2;
  for (int p = threadIdx.x; p < ntok * np; p += kThreads) {
    const int tk = p / np, j = p - tk * np;
    const double ang = static_cast<double>(a.pos[tok0 + tk]) * static_cast<double>(a.inv_freq[j]);
    // 2 pi in two parts: at positions around 2^40 the first part alone is 1e-5 off
    const double turns = rint(ang * 0.15915494309189535);
    const double red =
        fma(-turns, 2.4492935982947064e-16, fma(-turns, 6.283185307179586, ang));
    // what the angle loses in fp32 (up to 2^-23, all of a sine next to a multiple of pi) is put
    // back by the first term of the addition theorem: sin(h + l) = sin h + l cos h to 2^-47
    const float high = static_cast<float>(red);
    const float low = static_cast<float>(red - high);
    float sn, cn_;
    sincosf(high, &sn, &cn_);
    const float s_ = fmaf(low, cn_, sn), c_ = fmaf(-low, sn, cn_);
    cs[p] = make_float2(c_ * a.magnitude, s_ * a.magnitude * a.sign);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    if (pair[i] == -2) continue;
    if (pair[i] >= 0) {
      if constexpr (HALF) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float2 t = cs[pair[i] + e];
          const float p = to_f(v[i].e[e]), q = to_f(w[i].e[e]);
          from_f(&v[i].e[e], fmaf(p, t.x, -q * t.y));
          from_f(&w[i].e[e], fmaf(p, t.y, q * t.x));
        }
        *reinterpret_cast<decltype(w[i].v)*>(out + at[i] + a.r / 2) = w[i].v;
      } else {
#pragma unroll
        for (int e = 0; e < N; e += 2) {
          const float2 t = cs[pair[i] + e / 2];
          const float p = to_f(v[i].e[e]), q = to_f(v[i].e[e + 1]);
          from_f(&v[i].e[e], fmaf(p, t.x, -q * t.y));
          from_f(&v[i].e[e + 1], fmaf(p, t.y, q * t.x));
        }
      }
    }
    *reinterpret_cast<decltype(v[i].v)*>(out + at[i]) = v[i].v;
  }
}

template <typename E, int N, bool HALF>
kvc_status launch(const RopeProblem& p, cudaStream_t st) {
  Args a{};
  a.x = p.x;
  a.out = p.out;
  a.pos = p.pos;
  a.inv_freq = p.inv_freq;
  a.T = p.T;
  a.c = p.c;
  a.H = p.H;
  a.r = p.r;
  a.copy_units = p.x == p.out ? 0 : static_cast<int>((p.c - p.r) / N);
  a.rot_units = HALF ? p.r / 2 / N : p.r / N;
  a.magnitude = p.magnitude;
  a.sign = p.inverse ? -1.f : 1.f;
  const int64_t per_tok = int64_t(p.H) * (a.copy_units + a.rot_units);
  if (per_tok == 0) return KVC_OK;
  constexpr int64_t kPerCta = kThreads * kUnits;
  if (per_tok > (int64_t(1) << 30)) return KVC_ERR_UNSUPPORTED;
  int64_t blocks;
  if (per_tok >= kPerCta) {
    a.tokens = 1;
    a.chunks = ceil_div(per_tok, kPerCta);
    blocks = p.T * a.chunks;
  } else {
    a.tokens = static_cast<int>(kPerCta / per_tok);
    const int fit = p.r > 0 ? kMaxPairs / (p.r / 2) : a.tokens;
    if (a.tokens > fit) a.tokens = fit > 0 ? fit : 1;
    a.chunks = 1;
    blocks = ceil_div(p.T, a.tokens);
  }
  if (blocks > 0x7fffffff) return KVC_ERR_UNSUPPORTED;
  const size_t smem = static_cast<size_t>(a.tokens) * (p.r / 2) * sizeof(float2);
  auto kern = partial_rope_kernel<E, N, HALF>;
  if (smem > 48 * 1024 && !raise_smem_limit(reinterpret_cast<const void*>(kern)))
    return KVC_ERR_CUDA;
  kern<<<static_cast<unsigned>(blocks), kThreads, smem, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return KVC_ERR_CUDA;
  last_kernel() = "partial_rope_kernel";
  return KVC_OK;
}

}  // namespace rope

kvc_status launch_partial_rope(const RopeProblem& p, cudaStream_t st) {
  using namespace rope;
  // 16-byte units (8 bf16 or 4 fp32); the half layout needs r / 2 to hold whole units, which
  // for bf16 at r % 16 == 8 means 8-byte ones (c % 8 == 0 and r % 8 == 0 hold throughout)
  if (p.bf16) {
    if (!p.half) return launch<__nv_bfloat16, 8, false>(p, st);
    return p.r % 16 == 0 ? launch<__nv_bfloat16, 8, true>(p, st)
                         : launch<__nv_bfloat16, 4, true>(p, st);
  }
  return p.half ? launch<float, 4, true>(p, st) : launch<float, 4, false>(p, st);
}

}  // namespace kvc
