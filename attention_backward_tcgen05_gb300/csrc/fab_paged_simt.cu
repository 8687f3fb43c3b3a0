// fab_paged_simt.cu -- attention of new tokens over a paged key/value cache on
// the CUDA cores: every dtype, DK, DV <= 256, any page size.
//
//   token i of the n new ones of sequence b, head h:
//   s_m = scale q . k_m over m <= lens[b] - n + i (causal) or m < lens[b],
//   o = sum softmax(s)_m v_m,  lse = log sum exp(s_m)
//
// One pass over the keys with a running maximum and sum.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "fab.h"
#include "fab_device.cuh"
#include "fab_internal.h"

namespace fab {
namespace {

__device__ uint32_t g_err_paged;

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

// A warp per (token, head).
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) paged_rows_kernel(const PagedProblem p) {
  constexpr int R = (int)kMaxWidth / 32;
  if (blockIdx.x == 0) check_starts(p.starts, p.B, p.T, (int)threadIdx.x, (int)blockDim.x, &g_err_paged);
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= p.T * p.H) return;
  const int64_t t = row / p.H, h = row - t * p.H, hk = h / (p.H / p.Hkv);
  const int DK = (int)p.DK, DV = (int)p.DV;
  int64_t lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (p.starts[mid] <= t) lo = mid; else hi = mid;
  }
  const int64_t s0 = p.starts[lo], s1 = p.starts[lo + 1], len = p.lens[lo];
  if (t < s0 || t >= s1) return;  // padding after the last sequence
  int64_t mend = p.causal ? len - (s1 - t) + 1 : len;
  if (mend > p.max_pages * p.page) {
    mend = p.max_pages * p.page;
    atomicOr(&g_err_paged, kErrIndex);
  }
  const T* q = static_cast<const T*>(p.q) + row * DK;
  float qv[R], acc[R];
#pragma unroll
  for (int e = 0; e < R; ++e) {
    qv[e] = lane + 32 * e < DK ? to_f32(q[lane + 32 * e]) : 0.f;
    acc[e] = 0.f;
  }
  float mx = -INFINITY, l = 0.f;
  for (int64_t m = 0; m < mend; ++m) {
    const int64_t page = p.table[lo * p.max_pages + m / p.page];
    if (page < 0 || page >= p.pages) {
      atomicOr(&g_err_paged, kErrIndex);
      continue;
    }
    const int64_t at = (page * p.Hkv + hk) * p.page + m % p.page;
    const T* k = static_cast<const T*>(p.k) + at * DK;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < R; ++e)
      if (lane + 32 * e < DK) s += qv[e] * to_f32(k[lane + 32 * e]);
    s = warp_sum(s) * p.scale;
    if (s > mx) {
      const float corr = expf(mx - s);
      l *= corr;
#pragma unroll
      for (int e = 0; e < R; ++e) acc[e] *= corr;
      mx = s;
    }
    const float w = s == -INFINITY ? 0.f : expf(s - mx);
    l += w;
    const T* v = static_cast<const T*>(p.v) + at * DV;
#pragma unroll
    for (int e = 0; e < R; ++e)
      if (lane + 32 * e < DV) acc[e] += w * to_f32(v[lane + 32 * e]);
  }
  // (l is NaN when a score is: the row is then NaN, not empty)
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* o = static_cast<T*>(p.o) + row * DV;
#pragma unroll
  for (int e = 0; e < R; ++e)
    if (lane + 32 * e < DV) from_f32(o[lane + 32 * e], acc[e] * inv);
  if (p.lse != nullptr && lane == 0) p.lse[h * p.T + t] = l == 0.f ? INFINITY : mx + logf(l);
}

template <typename T>
cudaError_t paged_t(const PagedProblem& p, cudaStream_t s) {
  const int64_t grid = (p.T * p.H + kWarps - 1) / kWarps;
  if (grid > 2147483647ll) return cudaErrorInvalidValue;
  paged_rows_kernel<T><<<(unsigned)grid, kWarps * 32, 0, s>>>(p);
  return cudaPeekAtLastError();
}

}  // namespace

size_t paged_simt_workspace_bytes(const PagedProblem&) { return 256; }

cudaError_t launch_paged_simt(const PagedProblem& p, cudaStream_t s) {
  if (p.dtype == FAB_BF16) return paged_t<__nv_bfloat16>(p, s);
  if (p.dtype == FAB_F16) return paged_t<__half>(p, s);
  return paged_t<float>(p, s);
}

uint32_t take_error_paged() {
  uint32_t v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_paged, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(g_err_paged, &z, sizeof(z));
  return v;
}

}  // namespace fab
