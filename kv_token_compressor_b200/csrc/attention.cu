// Shared-KV attention over the compressed cache (include/kvc.h, shared_kv_attention and
// shared_kv_attention_topk): one pass over a query's rows with the running maximum and sum
// of the softmax.  A CTA takes one query and 8 heads, a warp one head; rows are widened to
// fp32 in shared memory 16 at a time.
#include "kvc_common.cuh"
#include "kvc_host.h"
#include "kvc_launch.h"

namespace kvc {

// bit 1: a query's rows or a listed entry out of range.
__device__ unsigned int g_attention_error = 0;

namespace attn {

constexpr int kRows = 16;
constexpr int kThreads = 256;
constexpr int kMaxPerLane = 16;  // channels per lane at c = 512

struct Query {
  int64_t key_start, n1, n2, win_start, n_visible;
  bool ok;
};
__device__ __forceinline__ Query query_of(const AttentionProblem& a, int64_t t) {
  Query q;
  q.key_start = a.key_start[t];
  q.n_visible = a.n_visible[t];
  q.n1 = a.idx ? (q.n_visible < a.k ? q.n_visible : a.k) : q.n_visible;
  q.win_start = a.win_start ? a.win_start[t] : 0;
  q.n2 = a.win_start ? a.win_len[t] : 0;
  q.ok = q.n_visible >= 0 && (a.idx || q.n_visible <= a.max_visible) && q.key_start >= 0 &&
         q.key_start <= a.cache_rows - q.n_visible && q.n2 >= 0 && q.n2 <= a.max_win &&
         (q.n2 == 0 || (q.win_start >= 0 && q.win_start <= a.win_rows - q.n2));
  return q;
}

__global__ void __launch_bounds__(kThreads) attention_simple_kernel(const AttentionProblem a) {
  extern __shared__ float kt[];  // [kRows][c]
  __shared__ int live[kRows];
  const int64_t t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y * 8 + warp;
  const Query q = query_of(a, t);
  if (!q.ok) {
    if (threadIdx.x == 0) atomicOr(&g_attention_error, 2u);
    return;
  }
  const int c = static_cast<int>(a.c), cn = c - a.r;
  const float inv_s = 1.f / a.fp8_scale;
  float qv[kMaxPerLane], o[kMaxPerLane];
#pragma unroll
  for (int i = 0; i < kMaxPerLane; ++i) {
    const int d = lane + 32 * i;
    o[i] = 0.f;
    qv[i] = h < a.H && d < c ? __bfloat162float(static_cast<const __nv_bfloat16*>(
                                   a.q)[(t * a.H + h) * a.c + d]) * a.scale
                             : 0.f;
  }
  float m = -INFINITY, l = 0.f;
  if (a.sink && h < a.H && a.sink[h] != -INFINITY) {
    m = a.sink[h];
    l = 1.f;
  }
  const int64_t n = q.n1 + q.n2;
  for (int64_t e0 = 0; e0 < n; e0 += kRows) {
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * c; i += kThreads) {
      const int rr = i / c, d = i - rr * c;
      const int64_t e = e0 + rr;
      float v = 0.f;
      bool ok = e < n;
      if (ok) {
        const bool win = e >= q.n1;
        int64_t row = win ? q.win_start + (e - q.n1) : q.key_start + e;
        if (!win && a.idx) {
          const int32_t ix = a.idx[t * a.k + e];
          ok = ix >= 0 && ix < q.n_visible;
          if (!ok && ix != -1) atomicOr(&g_attention_error, 2u);
          row = q.key_start + ix;
        }
        if (ok) {
          const uint8_t* nope = static_cast<const uint8_t*>(win ? a.win_nope : a.nope);
          const __nv_bfloat16* rp = static_cast<const __nv_bfloat16*>(win ? a.win_rope : a.rope);
          if (d < cn) {
            __nv_fp8_e4m3 b;
            b.__x = nope[row * cn + d];
            v = static_cast<float>(b) * inv_s;
          } else {
            v = __bfloat162float(rp[row * a.r + d - cn]);
          }
        }
      }
      kt[i] = v;
      if (d == 0) live[rr] = ok;
    }
    __syncthreads();
    for (int rr = 0; rr < kRows; ++rr) {
      if (!live[rr]) continue;
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kMaxPerLane; ++i) {
        const int d = lane + 32 * i;
        if (d < c) s = fmaf(qv[i], kt[rr * c + d], s);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      const float mn = fmaxf(m, s);
      const float f = mn == -INFINITY ? 1.f : __expf(m - mn);
      const float p = mn == -INFINITY ? 0.f : __expf(s - mn);
      m = mn;
      l = l * f + p;
#pragma unroll
      for (int i = 0; i < kMaxPerLane; ++i) {
        const int d = lane + 32 * i;
        if (d < c) o[i] = o[i] * f + p * kt[rr * c + d];
      }
    }
  }
  if (h >= a.H) return;
  const float il = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
  for (int i = 0; i < kMaxPerLane; ++i) {
    const int d = lane + 32 * i;
    if (d < c)
      static_cast<__nv_bfloat16*>(a.out)[(t * a.H + h) * a.c + d] = __float2bfloat16_rn(o[i] * il);
  }
  if (a.lse && lane == 0) a.lse[t * a.H + h] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace attn

int64_t attention_workspace_bytes(int64_t, int, int64_t, int, int64_t) { return 0; }

kvc_status launch_attention(const AttentionProblem& p, cudaStream_t st) {
  using namespace attn;
  const size_t smem = kRows * p.c * sizeof(float);
  const int64_t gy = ceil_div(p.H, 8);
  if (p.T > 0x7fffffff || gy > 65535) return KVC_ERR_UNSUPPORTED;
  attention_simple_kernel<<<dim3(static_cast<unsigned>(p.T), static_cast<unsigned>(gy)), kThreads,
                            smem, st>>>(p);
  if (cudaGetLastError() != cudaSuccess) return KVC_ERR_CUDA;
  last_kernel() = "attention_simple_kernel";
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
