// fab_rope.cu -- what stands between a projection and the attention: norms of
// the queries and keys per head, the position rotation, and the move from
// token rows to the attention's head-major tensors (or to a paged cache), with
// the gradient of it all.
//
//   n = x w / sqrt(mean(x^2) + eps),  y = R n  (pairs turned by the position's angle)
//   g = R^T dy, u = g w:  dx = r (u - r x mean(u r x)),  dw = sum g r x
//
// Memory bound: every value is read once and written once.  bf16, 4 sequences of
// 2,048 tokens, 32 query and 8 key heads of width 128: forward 33.5 us, 6.1 TB/s;
// gradient 70.8 us, 5.5 TB/s.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "fab.h"
#include "fab_device.cuh"
#include "fab_internal.h"
#include "fab_launch.cuh"

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

// The sequence of each lane's token t, the same in the L lanes of a group: the
// last that starts at or before it (empty ones before it share the start;
// starts[0] <= t is assumed).  The whole warp looks at 32 places at once, which all
// its groups share for the first look: two looks for up to 1,024 sequences, where
// halving takes ten, each as long as an access to memory (one token of 64 sequences
// 3.9 -> 3.4 us, drafts of up to 64 tokens of 64 sequences 16.0 -> 15.1, prompts of 8 the same).
template <int L>
__device__ __forceinline__ int64_t sequence_of(const RopeProblem& p, int64_t t) {
  const int lane = threadIdx.x & 31;
  int32_t lo = 0, n = (int32_t)p.seqs;  // this lane's sequence is one of the n from lo on
  int32_t step = (n - 1) / 32 + 1;
  if (n > 1) {
    const int64_t i = (int64_t)step * (lane + 1);
    const int64_t start = i < n ? (int64_t)p.starts[i] : INT64_MAX;
    int32_t over = 0;
#pragma unroll
    for (int g = 0; g < 32 / L; ++g) {
      const uint32_t at = __ballot_sync(0xffffffffu, start <= __shfl_sync(0xffffffffu, t, g * L));
      if (lane / L == g) over = __popc(at) * step;
    }
    lo = over;
    n = n - over < step ? n - over : step;
  }
  while (step > 1) {
    step = (step - 1) / 32 + 1;
    int32_t over = 0;
#pragma unroll
    for (int g = 0; g < 32 / L; ++g) {
      const int64_t tg = __shfl_sync(0xffffffffu, t, g * L);
      const int32_t lg = __shfl_sync(0xffffffffu, lo, g * L), ng = __shfl_sync(0xffffffffu, n, g * L);
      const int64_t i = (int64_t)step * (lane + 1);
      const uint32_t at = __ballot_sync(0xffffffffu, i < ng && p.starts[lg + i] <= tg);
      if (lane / L == g) over = __popc(at) * step;
    }
    lo += over;
    n = n - over < step ? n - over : step;
  }
  return lo;
}

// Token t's place, in sequence `lo` where there are sequences.  A position, page
// or start out of range sets kErrIndex and yields a place that touches nothing out
// of bounds.
__device__ Place place_of(const RopeProblem& p, int64_t t, int64_t lo) {
  Place x{0, -1, 0, true};
  bool bad = false;
  if (p.starts != nullptr) {
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
    if (p.seen != nullptr) {
      // a drafted token lies in the row of its number and stands as far behind
      // the past as it sees earlier ones
      const int i = (int)(t - s0);
      const uint32_t* row = p.seen + t * p.words;
      int deep = 0;
      for (int w = 0; w <= i >> 5 && w < p.words; ++w)
        deep += __popc(w < i >> 5 ? row[w] : row[w] & ((1u << (i & 31)) - 1u));
      bad |= i >= 32 * p.words;
      x.pos += deep - i;
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
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (launched early)
  if (p.starts != nullptr && blockIdx.x == 0)
    check_starts(p.starts, p.seqs, p.N, (int)threadIdx.x, (int)blockDim.x, &g_err_rope);
  const int lane = threadIdx.x & 31;
  const int64_t per = p.H + p.Hkv + (p.v != nullptr ? p.Hkv : 0);
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= p.B * p.N * per) return;
  const int64_t t = row / per;
  int64_t j = row - t * per;
  const Place at = place_of(p, t, p.starts != nullptr ? sequence_of<32>(p, t) : 0);
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
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
    const Place at = half > 0 ? place_of(p, t, 0) : Place{0, -1, 0, true};
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


// ------------------------------------------------------------------ 16-byte accesses
//
// L lanes (a power of two) share a row: each holds two chunks of 8 columns,
// which are the two halves of 8 pairs (or, interleaved, hold their pairs
// whole), so the rotation needs no exchange and a row's sum takes log2 L
// shuffles.  A group of L lanes keeps one token's cosines and sines and its
// operand's weights in registers and walks over heads; the next rows' loads are
// issued before the present ones are worked on, and rows wait in the type they
// were loaded in (half the registers of 32-bit values for the 16-bit types).

constexpr int kVecThreads = 128;

// 8 values as loaded.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) v[i] = ld_global_nc_v4(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[4 * i] = __uint_as_float(v[i].x);
        x[4 * i + 1] = __uint_as_float(v[i].y);
        x[4 * i + 2] = __uint_as_float(v[i].z);
        x[4 * i + 3] = __uint_as_float(v[i].w);
      }
    } else {
      const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<std::is_same<T, __half>::value>(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
  }
};

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    constexpr bool h = std::is_same<T, __half>::value;
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack2<h>(x[0], x[1]), pack2<h>(x[2], x[3]), pack2<h>(x[4], x[5]), pack2<h>(x[6], x[7]));
  }
}

// The chunks of lane slot `s` of a row of C chunks of which the first R are
// rotated: ca and cb (-1: none).  turned: both are rotated together (or, with
// IL, those below R by themselves).
template <bool IL>
__device__ __forceinline__ void chunks_of(int s, int C, int R, int& ca, int& cb, bool& ta, bool& tb) {
  if (IL || s >= R / 2) {
    ca = IL ? 2 * s : R + 2 * (s - R / 2);
    cb = ca + 1;
  } else {
    ca = s;
    cb = s + R / 2;
  }
  ta = ca < R;
  tb = cb < R;
  if (ca >= C) ca = -1;
  if (cb >= C) cb = -1;
}

// This lane's cosines and sines at a position: 8 pairs, or 4 of each chunk.
template <bool IL>
__device__ __forceinline__ void load_turn(const float* cos, const float* sin, int64_t pos, int half, int ca, int cb,
                                          bool ta, bool tb, float (&c)[8], float (&s)[8]) {
  const float* c0 = cos + pos * half;
  const float* s0 = sin + pos * half;
  if (IL) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (!(h ? tb : ta)) continue;
      const int at = (h ? cb : ca) * 4;
      const float4 x = __ldg(reinterpret_cast<const float4*>(c0 + at)), y = __ldg(reinterpret_cast<const float4*>(s0 + at));
      c[4 * h] = x.x, c[4 * h + 1] = x.y, c[4 * h + 2] = x.z, c[4 * h + 3] = x.w;
      s[4 * h] = y.x, s[4 * h + 1] = y.y, s[4 * h + 2] = y.z, s[4 * h + 3] = y.w;
    }
  } else if (ta) {
    load8(c0 + ca * 8, c);
    load8(s0 + ca * 8, s);
  }
}

// Rotates by the angle (BACK: by its negative).
template <bool IL, bool BACK>
__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const float (&c)[8], const float (&s)[8], bool ta,
                                     bool tb) {
  auto pair = [](float& x, float& y, float cc, float ss) {
    if (BACK) ss = -ss;
    const float x1 = x * cc - y * ss;
    y = y * cc + x * ss;
    x = x1;
  };
  if (IL) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (ta) pair(a[2 * i], a[2 * i + 1], c[i], s[i]);
      if (tb) pair(b[2 * i], b[2 * i + 1], c[4 + i], s[4 + i]);
    }
  } else if (ta) {
#pragma unroll
    for (int i = 0; i < 8; ++i) pair(a[i], b[i], c[i], s[i]);
  }
}

template <int L>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int off = L / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// One CTA: kVecThreads / L tokens times `hb` heads of one operand.  Blocks of
// heads: bq of q, bk of k, then v's.
template <typename T, int L, bool IL>
__global__ void __launch_bounds__(kVecThreads, sizeof(T) == 4 ? 4 : 5) rope_vec_kernel(const RopeProblem p, int hb,
                                                                                     int bq, int bk) {
  constexpr int U = sizeof(T) == 4 ? 1 : 2;  // rows a step
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (launched early)
  if (p.starts != nullptr && blockIdx.x == 0 && blockIdx.y == 0)
    check_starts(p.starts, p.seqs, p.N, (int)threadIdx.x, (int)blockDim.x, &g_err_rope);
  const int sub = threadIdx.x & (L - 1);
  const int64_t t = (int64_t)blockIdx.x * (kVecThreads / L) + threadIdx.x / L;
  const int by = (int)blockIdx.y;
  const int kind = by < bq ? 0 : by < bq + bk ? 1 : 2;
  const int heads = kind == 0 ? (int)p.H : (int)p.Hkv;
  // its heads are j0 .. j0 + nj - 1; j counts from j0, so that offsets from the
  // 64-bit addresses of head j0 fit 32 bits however long a token's row is
  const int j0 = (by - (kind == 0 ? 0 : kind == 1 ? bq : bq + bk)) * hb;
  const int nj = heads - j0 < hb ? heads - j0 : hb;
  const int D = (int)(kind == 2 ? p.DV : p.DK);
  const int half = kind == 2 ? 0 : (int)p.rot / 2;
  int ca, cb;
  bool ta, tb;
  chunks_of<IL>(sub, D / 8, half / 4, ca, cb, ta, tb);
  const bool row_ok = t < p.B * p.N;
  const bool oka = row_ok && ca >= 0, okb = row_ok && cb >= 0;
  const T* x0 = static_cast<const T*>(kind == 0 ? p.q : kind == 1 ? p.k : p.v) +
                t * (kind == 0 ? p.ldq : kind == 1 ? p.ldk : p.ldv) + (int64_t)j0 * D;
  Raw8<T> na[U], nb[U];
  auto fetch = [&](int j) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      na[u].zero();
      nb[u].zero();
      if (j + u < nj) {
        if (oka) na[u].load(x0 + (j + u) * D + ca * 8);
        if (okb) nb[u].load(x0 + (j + u) * D + cb * 8);
      }
    }
  };
  fetch(0);
  const T* w0 = static_cast<const T*>(kind == 0 ? p.wq : kind == 1 ? p.wk : nullptr);
  const bool norm = w0 != nullptr;
  Raw8<T> wa, wb;
  wa.zero();
  wb.zero();
  if (norm) {
    if (ca >= 0) wa.load(w0 + ca * 8);
    if (cb >= 0) wb.load(w0 + cb * 8);
  }
  Place at{0, -1, 0, false};
  const int64_t seq = p.starts != nullptr ? sequence_of<L>(p, t) : 0;  // (whole warps)
  if (row_ok) at = place_of(p, t, seq);
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
  if (row_ok && half > 0) load_turn<IL>(p.cos, p.sin, at.pos, half, ca, cb, ta, tb, c, s);
  // where this token's rows go: head j0 + j at y0 + j * ystep
  T* y0 = nullptr;
  int64_t ystep = 0;
  if (p.starts == nullptr) {
    const int64_t b = t / p.N, n = t - b * p.N;
    y0 = static_cast<T*>(kind == 0 ? p.q_out : kind == 1 ? p.k_out : p.v_out) + ((b * heads + j0) * p.N + n) * D;
    ystep = p.N * D;
  } else if (kind == 0) {
    y0 = static_cast<T*>(p.q_out) + (t * p.H + j0) * D;
    ystep = D;
  } else {
    y0 = static_cast<T*>(kind == 1 ? p.k_out : p.v_out) + ((at.page * p.Hkv + j0) * p.page + at.slot) * D;
    ystep = p.page * D;
  }
  const bool store = row_ok && at.live && (p.starts == nullptr || kind == 0 || at.page >= 0);
  const float inv_d = 1.f / (float)D;
  for (int j = 0; j < nj; j += U) {
    Raw8<T> ra[U], rb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) ra[u] = na[u], rb[u] = nb[u];
    if (j + U < nj) fetch(j + U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kind != 2) {
        float a[8], b[8];
        ra[u].get(a);
        rb[u].get(b);
        if (norm) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss += a[i] * a[i] + b[i] * b[i];
          const float r = rsqrtf(group_sum<L>(ss) * inv_d + p.eps);
          float w[8];
          wa.get(w);
#pragma unroll
          for (int i = 0; i < 8; ++i) a[i] *= r * w[i];
          wb.get(w);
#pragma unroll
          for (int i = 0; i < 8; ++i) b[i] *= r * w[i];
        }
        turn<IL, false>(a, b, c, s, ta, tb);
        if (store && j + u < nj) {
          T* y = y0 + (j + u) * ystep;
          if (oka) store8(y + ca * 8, a);
          if (okb) store8(y + cb * 8, b);
        }
      } else if (store && j + u < nj) {  // values move as they are
        T* y = y0 + (j + u) * ystep;
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i) {
          if (oka) reinterpret_cast<uint4*>(y + ca * 8)[i] = ra[u].v[i];
          if (okb) reinterpret_cast<uint4*>(y + cb * 8)[i] = rb[u].v[i];
        }
      }
    }
  }
}

// The gradient.  Blocks 0 .. nq-1 share q's items (kVecThreads / L tokens times hb
// heads), the next nk k's, the rest v's; each of the former leaves its sum of
// dw in partial[block].
template <typename T, int L, bool IL>
__global__ void __launch_bounds__(kVecThreads, 3) rope_vec_backward_kernel(const RopeProblem p, int hb, int nq, int nk,
                                                                           int nv) {
  __shared__ float acc_s[kVecThreads / 32][16 * L];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int sub = threadIdx.x & (L - 1), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blk = (int)blockIdx.x;
  const int kind = blk < nq ? 0 : blk < nq + nk ? 1 : 2;
  const int first_blk = kind == 0 ? 0 : kind == 1 ? nq : nq + nk, blocks = kind == 0 ? nq : kind == 1 ? nk : nv;
  const int heads = kind == 0 ? (int)p.H : (int)p.Hkv;
  const int D = (int)(kind == 2 ? p.DV : p.DK);
  const int half = kind == 2 ? 0 : (int)p.rot / 2;
  const float* dy0 = kind == 0 ? p.dq : kind == 1 ? p.dk : p.dv;
  const T* x0 = static_cast<const T*>(kind == 0 ? p.q : p.k);
  const int64_t ldx = kind == 0 ? p.ldq : p.ldk, ldg = kind == 0 ? p.ldgq : kind == 1 ? p.ldgk : p.ldgv;
  T* g0 = static_cast<T*>(kind == 0 ? p.gq : kind == 1 ? p.gk : p.gv);
  const T* w0 = static_cast<const T*>(kind == 0 ? p.wq : kind == 1 ? p.wk : nullptr);
  const bool norm = w0 != nullptr;
  int ca, cb;
  bool ta, tb;
  chunks_of<IL>(sub, D / 8, half / 4, ca, cb, ta, tb);
  float acc_a[8], acc_b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc_a[i] = acc_b[i] = 0.f;
  Raw8<T> wa, wb;
  wa.zero();
  wb.zero();
  if (norm) {
    if (ca >= 0) wa.load(w0 + ca * 8);
    if (cb >= 0) wb.load(w0 + cb * 8);
  }
  constexpr int A = sizeof(T) == 4 ? 1 : 2;  // rows on their way
  const float inv_d = 1.f / (float)D;
  const int64_t tokens = p.B * p.N, tblocks = (tokens + kVecThreads / L - 1) / (kVecThreads / L);
  const int64_t hblocks = (heads + hb - 1) / hb, items = tblocks * hblocks, dstep = p.N * D;
  for (int64_t it = blk - first_blk; it < items; it += blocks) {
    const int64_t tbk = it / hblocks;
    // heads j0 .. j0 + nj - 1; j counts from j0, as in rope_vec_kernel
    const int j0 = (int)(it - tbk * hblocks) * hb, nj = heads - j0 < hb ? heads - j0 : hb;
    const int64_t t = tbk * (kVecThreads / L) + threadIdx.x / L;
    const bool row_ok = t < tokens;
    const bool oka = row_ok && ca >= 0, okb = row_ok && cb >= 0;
    const int64_t b = t / p.N, n = t - b * p.N;
    const float* dy = dy0 + (b * heads * p.N + n) * D + j0 * dstep;
    const T* x = x0 + t * ldx + (int64_t)j0 * D;
    T* g = g0 + t * ldg + (int64_t)j0 * D;
    Raw8<float> nga[A], ngb[A];
    Raw8<T> nxa[A], nxb[A];
    auto fetch = [&](int j, int u) {
      nga[u].zero();
      ngb[u].zero();
      nxa[u].zero();
      nxb[u].zero();
      if (j >= nj) return;
      if (oka) nga[u].load(dy + j * dstep + ca * 8);
      if (okb) ngb[u].load(dy + j * dstep + cb * 8);
      if (norm) {
        if (oka) nxa[u].load(x + j * D + ca * 8);
        if (okb) nxb[u].load(x + j * D + cb * 8);
      }
    };
#pragma unroll
    for (int u = 0; u < A; ++u) fetch(u, u);
    // A row that is not there (past the last token, past the last head) adds
    // zeros to dw: by r = 0, as at eps = 0 its 1 / sqrt would be infinite.
    const int live = row_ok ? nj : 0;
    float c[8], s[8];  // (a lane past the last token turns zeros: by something finite)
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
    if (row_ok && half > 0) load_turn<IL>(p.cos, p.sin, place_of(p, t, 0).pos, half, ca, cb, ta, tb, c, s);
    for (int jj = 0; jj < nj; jj += A)
#pragma unroll
    for (int u = 0; u < A; ++u) {
      const int j = jj + u;
      float ga[8], gb[8];
      nga[u].get(ga);
      ngb[u].get(gb);
      const Raw8<T> rxa = nxa[u], rxb = nxb[u];
      fetch(j + A, u);
      if (kind != 2) turn<IL, true>(ga, gb, c, s, ta, tb);
      if (norm) {
        float xa[8], xb[8], w[8];
        rxa.get(xa);
        rxb.get(xb);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += xa[i] * xa[i] + xb[i] * xb[i];
        const float mean = group_sum<L>(ss) * inv_d;
        const float r = j < live ? rsqrtf(mean + p.eps) : 0.f;
        float dot = 0.f;
        wa.get(w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          xa[i] *= r;
          acc_a[i] += ga[i] * xa[i];
          ga[i] *= w[i];
          dot += ga[i] * xa[i];
        }
        wb.get(w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          xb[i] *= r;
          acc_b[i] += gb[i] * xb[i];
          gb[i] *= w[i];
          dot += gb[i] * xb[i];
        }
        dot = group_sum<L>(dot) * inv_d;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ga[i] = r * (ga[i] - xa[i] * dot);
          gb[i] = r * (gb[i] - xb[i] * dot);
        }
      }
      if (oka && j < nj) store8(g + j * D + ca * 8, ga);
      if (okb && j < nj) store8(g + j * D + cb * 8, gb);
    }
  }
  if (!norm) return;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int off = L; off < 32; off <<= 1) {
      acc_a[i] += __shfl_xor_sync(0xffffffffu, acc_a[i], off);
      acc_b[i] += __shfl_xor_sync(0xffffffffu, acc_b[i], off);
    }
  if (lane < L) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (ca >= 0) acc_s[warp][ca * 8 + i] = acc_a[i];
      if (cb >= 0) acc_s[warp][cb * 8 + i] = acc_b[i];
    }
  }
  __syncthreads();
  for (int i = (int)threadIdx.x; i < D; i += kVecThreads) {
    float sum = 0.f;
    for (int q = 0; q < kVecThreads / 32; ++q) sum += acc_s[q][i];
    p.partial[(int64_t)blk * D + i] = sum;
  }
}

// gw[i] = the sum of column i of the partial rows, nq of q then nk of k; a block
// takes 32 columns of one of them, its 32 rows of threads every 32nd row each.
__global__ void __launch_bounds__(1024) rope_partial_sum_kernel(const float* partial, int nq, int nk, int D, float* gwq,
                                                                float* gwk) {
  __shared__ float sum_s[32][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the rows are still being worked on
  float* gw = blockIdx.y == 0 ? gwq : gwk;
  if (gw == nullptr) return;
  const int rows = blockIdx.y == 0 ? nq : nk;
  const float* src = partial + (blockIdx.y == 0 ? 0 : (int64_t)nq * D);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = (int)blockIdx.x * 32 + lane;
  float sum = 0.f;
  if (i < D) {
#pragma unroll 8
    for (int r = warp; r < rows; r += 32) sum += src[(int64_t)r * D + i];
  }
  sum_s[warp][lane] = sum;
  __syncthreads();
  sum = warp_sum(sum_s[lane][warp]);
  const int o = (int)blockIdx.x * 32 + warp;
  if (lane == 0 && o < D) gw[o] = sum;
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Lanes a row of the 16-byte kernels needs for this width, 0 when it does not
// come in chunks of 8 columns with whole chunks rotated together.
int lanes_for(int64_t D, int64_t rot, int interleaved) {
  if (D % 8 != 0 || rot % (interleaved ? 8 : 16) != 0) return 0;
  const int64_t C = D / 8, R = rot / 8;
  const int64_t slots = interleaved ? (C + 1) / 2 : R / 2 + (C - R + 1) / 2;
  return slots <= 4 ? 4 : slots <= 8 ? 8 : 16;
}

// The 16-byte kernels' lanes for this call, 0 when some row or table is not
// 16-byte aligned: the kernels of a warp per row then serve it (the calls of the
// figures above in 204 and 402 us; one head of 128 tokens 3.5 us for 2.5).
int vec_lanes(const RopeProblem& p, bool backward) {
  const size_t e = p.dtype == FAB_F32 ? 4 : 2;
  const int lk = lanes_for(p.DK, p.rot, p.interleaved);
  const bool v = backward ? p.dv != nullptr : p.v != nullptr;
  const int lv = v ? lanes_for(p.DV, 0, p.interleaved) : lk;
  if (lk == 0 || lv == 0) return 0;
  auto rows = [&](const void* x, int64_t ld) { return aligned(x, 16) && (ld * (int64_t)e) % 16 == 0; };
  if ((p.wq && !aligned(p.wq, 16)) || (p.wk && !aligned(p.wk, 16))) return 0;
  if (p.rot > 0 && (!aligned(p.cos, 16) || !aligned(p.sin, 16))) return 0;
  if (!backward || p.wq)
    if (!rows(p.q, p.ldq)) return 0;
  if (!backward || p.wk)
    if (!rows(p.k, p.ldk)) return 0;
  if (!backward && v && !rows(p.v, p.ldv)) return 0;
  if (backward && (!rows(p.gq, p.ldgq) || !rows(p.gk, p.ldgk) || (v && !rows(p.gv, p.ldgv)))) return 0;
  return lk > lv ? lk : lv;
}

template <typename T, int L>
cudaError_t rope_vec(const RopeProblem& p, cudaStream_t s) {
  const int64_t gx = (p.B * p.N + kVecThreads / L - 1) / (kVecThreads / L);
  auto blocks = [&](int64_t hb) { return (p.H + hb - 1) / hb + (p.Hkv + hb - 1) / hb * (p.v != nullptr ? 2 : 1); };
  // heads a CTA walks over: 32, halved while the SMs have fewer than 8 CTAs each
  // (one token of 64 sequences, 32 and 8 heads: 4.0 us, never halved 12.1; prompts
  // of 8 sequences, 16 heads of width 64: 21.5 us, halved below 2 CTAs an SM only
  // 23.4, below 32 of them 23.5; the training step 33.4 us, below 32 37.2)
  int64_t hb = 32;
  while (hb > 1 && gx * blocks(hb) < 1216) hb /= 2;
  while (blocks(hb) > 65535) hb *= 2;  // (a grid's limit)
  const int64_t bq = (p.H + hb - 1) / hb, bk = (p.Hkv + hb - 1) / hb;
  if (gx > 2147483647ll) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)gx, (unsigned)blocks(hb));
  const auto kernel = p.interleaved ? rope_vec_kernel<T, L, true> : rope_vec_kernel<T, L, false>;
  return launch_early(kernel, grid, kVecThreads, 0, s, p, (int)hb, (int)bq, (int)bk);
}

template <typename T, int L>
cudaError_t rope_vec_backward(const RopeProblem& p, int* rows_q, int* rows_k, cudaStream_t s) {
  const int64_t tb = (p.B * p.N + kVecThreads / L - 1) / (kVecThreads / L);
  int64_t hb = 32;
  while (hb > 1 && tb * ((p.H + hb - 1) / hb + (p.Hkv + hb - 1) / hb * 2) < 456) hb /= 2;
  // blocks in the ratio of the operands' bytes, about 8 an SM (6: 74.1 us for
  // 70.4 on the training step; 3: 71.8, and 15.0 for 11.6 on 3 x 777 tokens of 12
  // and 4 heads of width 80, where an item of 32 heads takes 13.1, of fewer 20.7)
  auto blocks = [&](int64_t heads, int64_t most) {
    const int64_t items = tb * ((heads + hb - 1) / hb);
    return (int)(items < most ? items : most);
  };
  const int64_t all = 1216, sum = p.H + 2 * p.Hkv;
  const int nq = blocks(p.H, (all * p.H + sum - 1) / sum), nk = blocks(p.Hkv, (all * p.Hkv + sum - 1) / sum);
  const int nv = p.dv != nullptr ? blocks(p.Hkv, (all * p.Hkv + sum - 1) / sum) : 0;
  if (p.interleaved)
    rope_vec_backward_kernel<T, L, true><<<(unsigned)(nq + nk + nv), kVecThreads, 0, s>>>(p, (int)hb, nq, nk, nv);
  else
    rope_vec_backward_kernel<T, L, false><<<(unsigned)(nq + nk + nv), kVecThreads, 0, s>>>(p, (int)hb, nq, nk, nv);
  *rows_q = nq;
  *rows_k = nk;
  return cudaPeekAtLastError();
}

template <typename T>
cudaError_t rope_t(const RopeProblem& p, cudaStream_t s) {
  switch (vec_lanes(p, false)) {
    case 4: return rope_vec<T, 4>(p, s);
    case 8: return rope_vec<T, 8>(p, s);
    case 16: return rope_vec<T, 16>(p, s);
  }
  const int64_t rows = p.B * p.N * (p.H + p.Hkv + (p.v != nullptr ? p.Hkv : 0));
  const int64_t grid = (rows + kWarps - 1) / kWarps;
  if (grid > 2147483647ll) return cudaErrorInvalidValue;
  return launch_early(rope_rows_kernel<T>, dim3((unsigned)grid), kWarps * 32, 0, s, p);
}

template <typename T>
cudaError_t rope_backward_t(const RopeProblem& p, cudaStream_t s) {
  const int64_t tok = p.B * p.N;
  auto blocks = [&](int64_t heads, int64_t most) {
    const int64_t b = (tok * heads + kWarps - 1) / kWarps;
    return (int)(b < most ? b : most);
  };
  int nq = 0, nk = 0;
  cudaError_t e;
  switch (vec_lanes(p, true)) {
    case 4: e = rope_vec_backward<T, 4>(p, &nq, &nk, s); break;
    case 8: e = rope_vec_backward<T, 8>(p, &nq, &nk, s); break;
    case 16: e = rope_vec_backward<T, 16>(p, &nq, &nk, s); break;
    default: {
      nq = blocks(p.H, 768), nk = blocks(p.Hkv, 256);
      const int nv = p.dv != nullptr ? blocks(p.Hkv, 256) : 0;
      rope_rows_backward_kernel<T><<<(unsigned)(nq + nk + nv), kWarps * 32, 0, s>>>(p, nq, nk, nv);
      e = cudaPeekAtLastError();
    }
  }
  if (e != cudaSuccess || (p.gwq == nullptr && p.gwk == nullptr)) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((p.DK + 31) / 32), 2);
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_partial_sum_kernel, static_cast<const float*>(p.partial), nq, nk, (int)p.DK,
                            p.gwq, p.gwk);
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
