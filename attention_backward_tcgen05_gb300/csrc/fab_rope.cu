// fab_rope.cu -- what stands between a projection and the attention: norms of
// the queries and keys per head, the position rotation, and the move from
// token rows to the attention's head-major tensors (or to a paged cache), with
// the gradient of it all.
//
//   n = x w / sqrt(mean(x^2) + eps),  y = R n  (pairs turned by the position's angle)
//   g = R^T dy, u = g w:  dx = r (u - r x mean(u r x)),  dw = sum g r x
//
// Memory bound: every value is read once and written once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fab.h"
#include "fab_device.cuh"
#include "fab_internal.h"

namespace fab {
namespace {

__device__ uint32_t g_err_rope;

constexpr int kWarps = 8;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f32(float& dst, float x) { dst = x; }
__device__ __forceinline__ void from_f32(__nv_bfloat16& dst, float x) { dst = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f32(__half& dst, float x) { dst = __float2half_rn(x); }

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// Where a token's rows go, and the position it is rotated by.
struct Place {
  int64_t pos;    // row of cos and sin, clamped into the tables
  int64_t page;   // paged: page of the cache, or -1: not stored
  int64_t slot;   // paged: row of the page
  bool live;      // paged: the token belongs to a sequence
};

// Token t's place.  A position, page or start out of range sets kErrIndex and
// yields a place that touches nothing out of bounds.
__device__ Place place_of(const RopeProblem& p, int64_t t) {
  Place x{0, -1, 0, true};
  bool bad = false;
  if (p.starts != nullptr) {
    // the last sequence that starts at or before t (empty ones before it share the start)
    int64_t lo = 0, hi = p.seqs;  // starts[lo] <= t is assumed for lo = 0
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) >> 1;
      if (p.starts[mid] <= t) lo = mid; else hi = mid;
    }
    const int64_t s0 = p.starts[lo], s1 = p.starts[lo + 1];
    if (t < s0 || t >= s1) {
      x.live = false;  // padding after the last sequence
      return x;
    }
    x.pos = (int64_t)p.lens[lo] - (s1 - t);
    const int64_t pi = x.pos >= 0 ? x.pos / p.page : -1;
    if (pi < 0 || pi >= p.max_pages) {
      bad = true;
    } else {
      x.page = p.table[lo * p.max_pages + pi];
      x.slot = x.pos - pi * p.page;
      if (x.page < 0 || x.page >= p.pages) {
        x.page = -1;
        bad = true;
      }
    }
  } else {
    x.pos = p.pos != nullptr ? p.pos[t] : t % p.N;
  }
  if (p.rot > 0 && (x.pos < 0 || x.pos >= p.P)) {
    bad = true;
    x.pos = x.pos < 0 ? 0 : p.P - 1;
  }
  if (bad) atomicOr(&g_err_rope, kErrIndex);
  return x;
}

// The partner column of i < rot, and whether i is the pair's first; f: the pair's index.
__device__ __forceinline__ int partner(int i, int half, int interleaved, int& f, bool& first) {
  if (interleaved) {
    f = i >> 1;
    first = (i & 1) == 0;
    return i ^ 1;
  }
  first = i < half;
  f = first ? i : i - half;
  return first ? i + half : i - half;
}

// A warp per row of any width, alignment and stride.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) rope_rows_kernel(const RopeProblem p) {
  if (p.starts != nullptr && blockIdx.x == 0)
    check_starts(p.starts, p.seqs, p.N, (int)threadIdx.x, (int)blockDim.x, &g_err_rope);
  const int lane = threadIdx.x & 31;
  const int64_t per = p.H + p.Hkv + (p.v != nullptr ? p.Hkv : 0);
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= p.B * p.N * per) return;
  const int64_t t = row / per;
  int64_t j = row - t * per;
  const Place at = place_of(p, t);
  if (!at.live) return;
  const int kind = j < p.H ? 0 : j < p.H + p.Hkv ? 1 : 2;
  if (kind == 1) j -= p.H;
  if (kind == 2) j -= p.H + p.Hkv;
  const int D = (int)(kind == 2 ? p.DV : p.DK);
  const T* x = static_cast<const T*>(kind == 0 ? p.q : kind == 1 ? p.k : p.v) +
               t * (kind == 0 ? p.ldq : kind == 1 ? p.ldk : p.ldv) + j * D;
  T* y;
  if (p.starts == nullptr) {
    const int64_t b = t / p.N, n = t - b * p.N, heads = kind == 0 ? p.H : p.Hkv;
    y = static_cast<T*>(kind == 0 ? p.q_out : kind == 1 ? p.k_out : p.v_out) + ((b * heads + j) * p.N + n) * D;
  } else if (kind == 0) {
    y = static_cast<T*>(p.q_out) + (t * p.H + j) * D;
  } else {
    if (at.page < 0) return;
    y = static_cast<T*>(kind == 1 ? p.k_out : p.v_out) + ((at.page * p.Hkv + j) * p.page + at.slot) * D;
  }
  if (kind == 2) {
    for (int i = lane; i < D; i += 32) y[i] = x[i];
    return;
  }
  const T* w = static_cast<const T*>(kind == 0 ? p.wq : p.wk);
  float r = 1.f;
  if (w != nullptr) {
    float ss = 0.f;
    for (int i = lane; i < D; i += 32) ss += to_f32(x[i]) * to_f32(x[i]);
    r = rsqrtf(warp_sum(ss) / (float)D + p.eps);
  }
  const int half = (int)p.rot / 2;
  const float* c = p.cos + at.pos * half;
  const float* s = p.sin + at.pos * half;
  for (int i = lane; i < D; i += 32) {
    float a = to_f32(x[i]) * r;
    if (w != nullptr) a *= to_f32(w[i]);
    if (i < 2 * half) {
      int f;
      bool first;
      const int o = partner(i, half, p.interleaved, f, first);
      float b = to_f32(x[o]) * r;
      if (w != nullptr) b *= to_f32(w[o]);
      a = first ? a * c[f] - b * s[f] : a * c[f] + b * s[f];
    }
    from_f32(y[i], a);
  }
}

// The gradient, a warp per row.  Blocks 0 .. nq-1 walk q's rows, the next nk
// k's, the rest v's; each of the former leaves its sum of dw in partial[block].
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) rope_rows_backward_kernel(const RopeProblem p, int nq, int nk, int nv) {
  __shared__ float acc_s[kWarps][kMaxWidth];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blk = (int)blockIdx.x;
  const int kind = blk < nq ? 0 : blk < nq + nk ? 1 : 2;
  const int first_blk = kind == 0 ? 0 : kind == 1 ? nq : nq + nk, blocks = kind == 0 ? nq : kind == 1 ? nk : nv;
  const int64_t heads = kind == 0 ? p.H : p.Hkv;
  const int D = (int)(kind == 2 ? p.DV : p.DK);
  const float* dy0 = kind == 0 ? p.dq : kind == 1 ? p.dk : p.dv;
  const T* x0 = static_cast<const T*>(kind == 0 ? p.q : p.k);
  const int64_t ldx = kind == 0 ? p.ldq : p.ldk, ldg = kind == 0 ? p.ldgq : kind == 1 ? p.ldgk : p.ldgv;
  T* g0 = static_cast<T*>(kind == 0 ? p.gq : kind == 1 ? p.gk : p.gv);
  const T* w = static_cast<const T*>(kind == 0 ? p.wq : kind == 1 ? p.wk : nullptr);
  const int half = kind == 2 ? 0 : (int)p.rot / 2;
  constexpr int R = (int)kMaxWidth / 32;
  float acc[R];
#pragma unroll
  for (int e = 0; e < R; ++e) acc[e] = 0.f;
  const int64_t rows = p.B * p.N * heads;
  for (int64_t row = (int64_t)(blk - first_blk) * kWarps + warp; row < rows; row += (int64_t)blocks * kWarps) {
    const int64_t t = row / heads, j = row - t * heads;
    const int64_t b = t / p.N, n = t - b * p.N;
    const float* dy = dy0 + ((b * heads + j) * p.N + n) * D;
    T* g = g0 + t * ldg + j * D;
    const Place at = half > 0 ? place_of(p, t) : Place{0, -1, 0, true};
    const float* c = p.cos + at.pos * half;
    const float* s = p.sin + at.pos * half;
    float u[R], xr[R];
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < R; ++e) {
      const int i = lane + 32 * e;
      u[e] = xr[e] = 0.f;
      if (i < D) {
        u[e] = dy[i];
        if (i < 2 * half) {
          int f;
          bool first;
          const int o = partner(i, half, p.interleaved, f, first);
          u[e] = first ? dy[i] * c[f] + dy[o] * s[f] : dy[i] * c[f] - dy[o] * s[f];
        }
        if (w != nullptr) {
          xr[e] = to_f32(x0[t * ldx + j * D + i]);
          ss += xr[e] * xr[e];
        }
      }
    }
    float r = 1.f, dot = 0.f;
    if (w != nullptr) {
      r = rsqrtf(warp_sum(ss) / (float)D + p.eps);
#pragma unroll
      for (int e = 0; e < R; ++e) {
        const int i = lane + 32 * e;
        if (i < D) {
          xr[e] *= r;
          acc[e] += u[e] * xr[e];
          u[e] *= to_f32(w[i]);
          dot += u[e] * xr[e];
        }
      }
      dot = warp_sum(dot) / (float)D;
    }
#pragma unroll
    for (int e = 0; e < R; ++e) {
      const int i = lane + 32 * e;
      if (i < D) from_f32(g[i], r * (u[e] - xr[e] * dot));
    }
  }
  if (w == nullptr) return;
#pragma unroll
  for (int e = 0; e < R; ++e) acc_s[warp][lane + 32 * e] = acc[e];
  __syncthreads();
  const int i = threadIdx.x;
  if (i < D) {
    float sum = 0.f;
    for (int q = 0; q < kWarps; ++q) sum += acc_s[q][i];
    p.partial[(int64_t)blk * D + i] = sum;
  }
}

// gw[i] = the sum of column i of `rows` partial rows; block 0 for q, 1 for k.
__global__ void __launch_bounds__(256) rope_partial_sum_kernel(const float* partial, int nq, int nk, int D, float* gwq,
                                                               float* gwk) {
  const int which = (int)blockIdx.y;
  float* gw = which == 0 ? gwq : gwk;
  if (gw == nullptr) return;
  const int rows = which == 0 ? nq : nk;
  const float* src = partial + (which == 0 ? 0 : (int64_t)nq * D);
  // a warp per column, lanes over the rows
  const int i = (int)blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (i >= D) return;
  float sum = 0.f;
  for (int r = lane; r < rows; r += 32) sum += src[(int64_t)r * D + i];
  sum = warp_sum(sum);
  if (lane == 0) gw[i] = sum;
}

template <typename T>
cudaError_t rope_t(const RopeProblem& p, cudaStream_t s) {
  const int64_t rows = p.B * p.N * (p.H + p.Hkv + (p.v != nullptr ? p.Hkv : 0));
  const int64_t grid = (rows + kWarps - 1) / kWarps;
  if (grid > 2147483647ll) return cudaErrorInvalidValue;
  rope_rows_kernel<T><<<(unsigned)grid, kWarps * 32, 0, s>>>(p);
  return cudaPeekAtLastError();
}

template <typename T>
cudaError_t rope_backward_t(const RopeProblem& p, cudaStream_t s) {
  const int64_t tok = p.B * p.N;
  auto blocks = [&](int64_t heads, int64_t most) {
    const int64_t b = (tok * heads + kWarps - 1) / kWarps;
    return (int)(b < most ? b : most);
  };
  const int nq = blocks(p.H, 768), nk = blocks(p.Hkv, 256), nv = p.dv != nullptr ? blocks(p.Hkv, 256) : 0;
  rope_rows_backward_kernel<T><<<(unsigned)(nq + nk + nv), kWarps * 32, 0, s>>>(p, nq, nk, nv);
  cudaError_t e = cudaPeekAtLastError();
  if (e != cudaSuccess || (p.gwq == nullptr && p.gwk == nullptr)) return e;
  rope_partial_sum_kernel<<<dim3((unsigned)((p.DK + 7) / 8), 2), 256, 0, s>>>(p.partial, nq, nk, (int)p.DK, p.gwq,
                                                                              p.gwk);
  return cudaPeekAtLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeProblem& p, cudaStream_t s) {
  if (p.dtype == FAB_BF16) return rope_t<__nv_bfloat16>(p, s);
  if (p.dtype == FAB_F16) return rope_t<__half>(p, s);
  return rope_t<float>(p, s);
}

cudaError_t launch_rope_backward(const RopeProblem& p, cudaStream_t s) {
  if (p.dtype == FAB_BF16) return rope_backward_t<__nv_bfloat16>(p, s);
  if (p.dtype == FAB_F16) return rope_backward_t<__half>(p, s);
  return rope_backward_t<float>(p, s);
}

uint32_t take_error_rope() {
  uint32_t v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_rope, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(g_err_rope, &z, sizeof(z));
  return v;
}

}  // namespace fab
