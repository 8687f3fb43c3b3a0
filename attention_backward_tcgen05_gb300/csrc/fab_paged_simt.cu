// fab_paged_simt.cu -- attention of new tokens over a paged key/value cache on
// the CUDA cores: every dtype, DK, DV <= 256, any page size.  It serves f32,
// whose accuracy the tensor cores' 16-bit products do not reach, and the
// widths and pages that the tensor-core kernel does not take.
//
//   token i of the n new ones of sequence b, head h:
//   s_m = scale q . k_m over m <= lens[b] - n + i (causal) or m < lens[b],
//   o = sum softmax(s)_m v_m,  lse = log sum exp(s_m)
// Drafted trees (TREE): causal, and of the new keys m = lens[b] - n + j only
// those whose bit j is set in the token's row of `seen`.
//
// The work is shared out as on the tensor cores (fab_paged.cuh), with tiles of
// R rows and key tiles of 64.  Each of a CTA's eight warps owns 8 keys of every
// key tile, from the copy to the sum: it fetches their rows into a ring of its
// own with bulk copies (a lane a row), keeps a running maximum and sum of its
// own, and adds its keys' share to an output of its own, so that the loop has no
// barrier for the block.  The warps' shares meet at the unit's end.  Scores: 64 / R
// lanes share a block of 4 rows and 4 keys, each summing its part of the
// columns (8 reads of shared memory for 64 multiply-adds), and add up by
// shuffles that leave each lane R / 4 rows of one key; the output: a lane takes
// CPL columns of all R rows, so a value is read from shared memory once for R
// rows.
//
// Few rows a sequence: bound by memory (f32, one sequence of 100,000 keys, 32
// heads on 8, width 128: 153 us, 5.4 TB/s).  More: by the latency of a tile's
// steps, of which two warps a scheduler hide only a part (chunks of 60 tokens on
// 2,000 keys 107 us).  Copies of 16 bytes by every lane in place of the bulk copies
// took 249 and 142 us: a third of the instructions and more was theirs.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "fab.h"
#include "fab_device.cuh"
#include "fab_internal.h"
#include "fab_paged.cuh"

namespace fab {
namespace {

__device__ uint32_t g_err_paged;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kKeys = 8;    // keys of a tile that a warp owns
constexpr int kStages = 4;  // of a warp's ring, at most
constexpr int kFewTiles = 4;  // key tiles of a unit that one CTA walks (paged_grid)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct SimtParams {
  PagedPlan plan;
  PagedParts parts;
  const int32_t* table;
  int64_t max_pages, pages;
  int page, H, Hkv, DK, DV;
  int ks, vs;          // bytes of a key and a value row in the ring (multiples of 16)
  int qs;              // floats of a query row in shared memory (a multiple of 4, zero past DK)
  int stages;          // of a warp's ring
  int bulk;            // rows come in whole aligned 16-byte pieces
  float c1;            // scale log2 e
  const uint32_t* seen;
  int words;
  const void *q, *k, *v;
  void* o;
  float* lse;
};

FAB_DEV float to_f32(float x) { return x; }
FAB_DEV float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
FAB_DEV float to_f32(__half x) { return __half2float(x); }

// Four values of a row in shared memory.
template <typename T>
FAB_DEV float4 lds4(const T* p) {
  if constexpr (sizeof(T) == 4) {
    return *reinterpret_cast<const float4*>(p);
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    constexpr bool h = std::is_same<T, __half>::value;
    const float2 a = unpack2<h>(v.x), b = unpack2<h>(v.y);
    return make_float4(a.x, a.y, b.x, b.y);
  }
}

// Of a pair of values in each of two lanes, `bit` apart: the lane whose bit is
// set gets the sum of both lanes' second, the other that of their first.
FAB_DEV float halve(bool set, float first, float second, int bit) {
  const float keep = set ? second : first, give = set ? first : second;
  return keep + __shfl_xor_sync(0xffffffffu, give, bit);
}

template <typename T, int R, int CPL, bool TREE>
__global__ void __launch_bounds__(kThreads, 1) paged_simt_kernel(const __grid_constant__ SimtParams p) {
  static_assert((R == 4 || R == 8 || R == 16) && CPL % 4 == 0, "");
  constexpr int RPL = R / 4;  // rows a lane scores
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ PagedShared sh;
  __shared__ uint64_t bars[kWarps][kStages];  // a ring slot's rows have landed
  __shared__ uint32_t abort_s;
  volatile uint32_t* abort_flag = &abort_s;
  const PagedPlan& plan = p.plan;
  const int lane = (int)lane_id(), warp = (int)warp_id();
  if (lane < kStages) mbar_init(smem_u32(&bars[warp][lane]), 1);
  if (threadIdx.x == 0) abort_s = 0u;
  fence_mbar_init();
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (launched early: lengths and operands from here on)
  if (blockIdx.x == 0) check_starts(plan.starts, plan.B, plan.T, (int)threadIdx.x, kThreads, &g_err_paged);
  int64_t mine;
  paged_total<kThreads>(plan, &sh, &mine);
  const PagedBorders border(sh.total, (int)gridDim.x);
  const int64_t p0 = border((int)blockIdx.x), p1 = border((int)blockIdx.x + 1);
  if (p0 < p1) paged_locate<kThreads>(plan, &sh, mine, p0);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const PagedPlace start = sh.at;
  PagedCut cut{0, 0, 0, 0, 0, 0, 0, 0};
  if (p0 >= p1) {
    if (threadIdx.x == 0 && !plan.whole) p.parts.cuts[blockIdx.x] = cut;
    return;
  }

  float* q_s = reinterpret_cast<float*>(smem);               // [R][qs]
  float* p_s = q_s + R * p.qs + warp * (kKeys + 1) * R;      // this warp's weights [key][row], then factors [row]
  uint8_t* ring0 = smem + (R * p.qs + kWarps * (kKeys + 1) * R) * 4;
  const int stage_bytes = kKeys * (p.ks + p.vs);
  uint8_t* ring = ring0 + warp * p.stages * stage_bytes;
  float* acc_s = reinterpret_cast<float*>(ring0);            // at a unit's end: [warp][R][dp]
  float2* ml_s = reinterpret_cast<float2*>(acc_s + kWarps * R * p.parts.dp);  // [warp][R]
  const int key = lane & 7, rg = lane >> 3;  // this lane's key, its rows rg * RPL ..
  // sums: DG lanes share a block of 4 rows and 4 keys, every DG-th piece of 4 columns each
  constexpr int DG = 64 / R;
  const int kg = (lane >> 2) & 1, dg = rg % (DG / 4) * 4 + (lane & 3);
  const float* q_r = q_s + rg / (DG / 4) * 4 * p.qs;
  const T* kc = static_cast<const T*>(p.k);
  const T* vc = static_cast<const T*>(p.v);

  int in = 0, out = 0;      // the ring's slots to fill and to work on next
  uint32_t out_phase = 0;
  PagedWalk w;
  w.begin(plan, start);
  for (bool more = w.seek(plan, p0, p1); more; more = w.next(plan) && w.seek(plan, p0, p1)) {
    const int hk = w.at.head / plan.gblocks, gb = w.at.head - hk * plan.gblocks;
    const int token0 = w.at.i * plan.nt;
    // the unit's queries, zero where there is no row
    fence_proxy_async_smem();  // (the rings held the shares of the unit before)
    __syncthreads();
    if (*abort_flag) break;
    for (int x = (int)threadIdx.x; x < R * p.qs; x += kThreads) {
      const int r = x / p.qs, d = x - r * p.qs, i = r / plan.gw, g = gb * plan.gw + r - i * plan.gw;
      float v = 0.f;
      if (d < p.DK && i < plan.nt && token0 + i < w.q.n && g < plan.G)
        v = to_f32(static_cast<const T*>(p.q)[((int64_t)(w.q.s0 + token0 + i) * p.H + (int64_t)hk * plan.G + g) * p.DK + d]);
      q_s[x] = v;
    }
    if (threadIdx.x == 0 && (plan.lens[w.at.b] > plan.max_keys || (TREE && w.q.n > (int64_t)p.words * 32)))
      atomicOr(&g_err_paged, kErrIndex);
    __syncthreads();
    int last[RPL];  // last key that each of this lane's rows sees
#pragma unroll
    for (int e = 0; e < RPL; ++e) {
      const int i = (rg * RPL + e) / plan.gw;
      last[e] = w.q.len - 1;
      if (plan.causal && w.q.last0 + token0 + i < last[e]) last[e] = w.q.last0 + token0 + i;
    }
    float m[RPL], l[RPL], acc[R][CPL];
#pragma unroll
    for (int e = 0; e < RPL; ++e) m[e] = -INFINITY, l[e] = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < CPL; ++c) acc[r][c] = 0.f;

    // row of the caches that holds this lane's key of tile j (every group of 8
    // lanes looks up the same 8), or -1
    auto lookup = [&](int j) -> int64_t {
      if (j >= w.j1) return -1;
      const int mk = j * 64 + warp * kKeys + key;
      if (mk >= w.q.len) return -1;
      const int at = (int)((uint32_t)mk / (uint32_t)p.page);
      const int page = p.table[(int64_t)w.at.b * p.max_pages + at];
      if (page >= 0 && page < p.pages) return ((int64_t)page * p.Hkv + hk) * p.page + (mk - at * p.page);
      atomicOr(&g_err_paged, kErrIndex);  // (its key and value are zeros)
      return -1;
    };
    // copies the 8 rows `row` names into the ring's next slot, zeros for -1
    auto fetch = [&](int64_t row) {
      uint8_t* kd = ring + in * stage_bytes;
      uint8_t* vd = kd + kKeys * p.ks;
      if (p.bulk) {
        // a lane a row: lanes 0 .. 7 the keys, 8 .. 15 the values
        const uint32_t kbytes = p.DK * (int)sizeof(T), vbytes = p.DV * (int)sizeof(T);
        const uint32_t here = __ballot_sync(0xffffffffu, row >= 0) & 0xffu, bar = smem_u32(&bars[warp][in]);
        for (uint32_t gone = here ^ 0xffu; gone != 0; gone &= gone - 1) {
          const int kk = __ffs((int)gone) - 1;
          for (uint32_t x = lane * 16; x < kbytes; x += 512) st_shared_v4(smem_u32(kd + kk * p.ks) + x, 0u, 0u, 0u, 0u);
          for (uint32_t x = lane * 16; x < vbytes; x += 512) st_shared_v4(smem_u32(vd + kk * p.vs) + x, 0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
        }
        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)__popc(here) * (kbytes + vbytes));
        __syncwarp();
        if (lane < 16 && row >= 0) {
          if (lane < 8)
            bulk_load(smem_u32(kd + key * p.ks), kc + row * p.DK, kbytes, bar);
          else
            bulk_load(smem_u32(vd + key * p.vs), vc + row * p.DV, vbytes, bar);
        }
      } else {
        for (int kk = 0; kk < kKeys; ++kk) {
          const int64_t src = __shfl_sync(0xffffffffu, row, kk);
          const T* kf = kc + (src < 0 ? 0 : src) * p.DK;
          const T* vf = vc + (src < 0 ? 0 : src) * p.DV;
          T* kr = reinterpret_cast<T*>(kd + kk * p.ks);
          T* vr = reinterpret_cast<T*>(vd + kk * p.vs);
          for (int d = lane; d < p.qs; d += 32) kr[d] = src >= 0 && d < p.DK ? kf[d] : T(0.f);
          for (int d = lane; d < p.DV; d += 32) vr[d] = src >= 0 ? vf[d] : T(0.f);
        }
      }
      if (++in == p.stages) in = 0;
    };

    __syncwarp();
    const int ahead = p.stages - 1;  // tiles on their way
    for (int s = 0; s < ahead && w.j0 + s < w.j1; ++s) fetch(lookup(w.j0 + s));
    int64_t next = lookup(w.j0 + ahead);  // of the next fetch: looked up a tile ahead
    for (int j = w.j0; j < w.j1; ++j) {
      if (j + ahead < w.j1) {
        fetch(next);
        next = lookup(j + p.stages);
      }
      if (p.bulk && !__all_sync(0xffffffffu, mbar_wait_asleep(smem_u32(&bars[warp][out]), out_phase, abort_flag,
                                                              &g_err_paged))) {
        // give up: let what is on its way land before shared memory goes
        for (int left = (j + p.stages < w.j1 ? j + p.stages : w.j1) - j; left > 0; --left) {
          mbar_drain(smem_u32(&bars[warp][out]), out_phase);
          if (++out == p.stages) out = 0, out_phase ^= 1u;
        }
        break;
      }
      __syncwarp();
      // whether this lane's rows see its key, where it is a new token's: fetched ahead of the sums
      [[maybe_unused]] uint32_t see[RPL];
      if constexpr (TREE) {
        const int at = j * 64 + warp * kKeys + key - w.q.last0;  // the key's number among the new ones
#pragma unroll
        for (int e = 0; e < RPL; ++e) {
          const int token = token0 + (rg * RPL + e) / plan.gw;
          see[e] = at < 0 ? 1u
                   : token < w.q.n && at >> 5 < p.words
                       ? __ldg(p.seen + (int64_t)(w.q.s0 + token) * p.words + (at >> 5)) >> (at & 31) & 1u
                       : 0u;
        }
      }
      const uint8_t* kb = ring + out * stage_bytes + kg * 4 * p.ks;
      const uint8_t* vb = ring + out * stage_bytes + kKeys * p.ks;
      float part[4][4];  // [row][key] over this lane's columns
#pragma unroll
      for (int e = 0; e < 4; ++e) part[e][0] = part[e][1] = part[e][2] = part[e][3] = 0.f;
#pragma unroll 2
      for (int d = dg * 4; d < p.qs; d += DG * 4) {
        float4 kv[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) kv[k] = lds4(reinterpret_cast<const T*>(kb + k * p.ks) + d);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 qv = *reinterpret_cast<const float4*>(q_r + e * p.qs + d);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            part[e][k] = fmaf(qv.x, kv[k].x, fmaf(qv.y, kv[k].y, fmaf(qv.z, kv[k].z, fmaf(qv.w, kv[k].w, part[e][k]))));
        }
      }
      __syncwarp();
      // the lanes of a block sum theirs up, each keeping half of what is left: a
      // key for each of four lanes, then rows
      float s[RPL];
      {
        const bool b0 = lane & 1, b1 = lane & 2, b3 = lane & 8, b4 = lane & 16;
        float two[4][2], one[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
          for (int k = 0; k < 2; ++k) two[e][k] = halve(b1, part[e][k], part[e][2 + k], 2);
          one[e] = halve(b0, two[e][0], two[e][1], 1);
        }
        if constexpr (RPL == 4) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[e] = one[e];
        } else if constexpr (RPL == 2) {
#pragma unroll
          for (int e = 0; e < 2; ++e) s[e] = halve(b3, one[e], one[2 + e], 8);
        } else {
          s[0] = halve(b3, halve(b4, one[0], one[2], 16), halve(b4, one[1], one[3], 16), 8);
        }
      }
      const int mk = j * 64 + warp * kKeys + key;
      bool grew = false;
      float f[RPL];
#pragma unroll
      for (int e = 0; e < RPL; ++e) {
        bool sees = mk <= last[e];
        if constexpr (TREE) sees = sees && see[e] != 0u;
        s[e] = sees ? s[e] * p.c1 : -INFINITY;
        float top = s[e];
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        f[e] = 1.f;
        if (top > m[e]) {
          f[e] = m[e] == -INFINITY ? 0.f : exp2f(m[e] - top);  // (what there is before the first key is zero)
          m[e] = top;
          grew = true;
        }
        const float wt = s[e] == -INFINITY ? 0.f : exp2f(s[e] - m[e]);
        l[e] = l[e] * f[e] + wt;
        p_s[key * R + rg * RPL + e] = wt;
        if (key == 0) p_s[kKeys * R + rg * RPL + e] = f[e];
      }
      grew = __any_sync(0xffffffffu, grew);
      __syncwarp();
      if (grew) {
#pragma unroll
        for (int r = 0; r < R; r += 4) {
          const float4 fr = *reinterpret_cast<const float4*>(p_s + kKeys * R + r);
#pragma unroll
          for (int c = 0; c < CPL; ++c) {
            acc[r][c] *= fr.x;
            acc[r + 1][c] *= fr.y;
            acc[r + 2][c] *= fr.z;
            acc[r + 3][c] *= fr.w;
          }
        }
      }
#pragma unroll
      for (int kk = 0; kk < kKeys; ++kk) {
        const T* vr = reinterpret_cast<const T*>(vb + kk * p.vs);
#pragma unroll
        for (int c = 0; c < CPL; c += 4) {
          const int col = (c / 4) * 128 + lane * 4;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          if (col < p.DV) v = lds4(vr + col);
#pragma unroll
          for (int r = 0; r < R; r += 4) {
            const float4 pr = *reinterpret_cast<const float4*>(p_s + kk * R + r);
            const float wr[4] = {pr.x, pr.y, pr.z, pr.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              acc[r + i][c] = fmaf(wr[i], v.x, acc[r + i][c]);
              acc[r + i][c + 1] = fmaf(wr[i], v.y, acc[r + i][c + 1]);
              acc[r + i][c + 2] = fmaf(wr[i], v.z, acc[r + i][c + 2]);
              acc[r + i][c + 3] = fmaf(wr[i], v.w, acc[r + i][c + 3]);
            }
          }
        }
      }
      __syncwarp();  // the slot and the weights may be written again
      if (++out == p.stages) out = 0, out_phase ^= 1u;
    }
    // ---- the unit's end: the warps' shares
#pragma unroll
    for (int e = 0; e < RPL; ++e)
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], o);
    __syncthreads();
    const int dp = p.parts.dp;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < CPL; c += 4) {
        const int col = (c / 4) * 128 + lane * 4;
        if (col < dp)
          *reinterpret_cast<float4*>(acc_s + (warp * R + r) * dp + col) =
              make_float4(acc[r][c], acc[r][c + 1], acc[r][c + 2], acc[r][c + 3]);
      }
    if (key == 0) {
#pragma unroll
      for (int e = 0; e < RPL; ++e) ml_s[warp * R + rg * RPL + e] = make_float2(m[e], l[e]);
    }
    __syncthreads();
    const bool whole = w.whole();
    for (int x = (int)threadIdx.x; x < R * dp; x += kThreads) {
      const int r = x / dp, col = x - r * dp, i = r / plan.gw, g = gb * plan.gw + r - i * plan.gw;
      if (i >= plan.nt || token0 + i >= w.q.n || g >= plan.G) continue;
      float top = -INFINITY;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) top = fmaxf(top, ml_s[v * R + r].x);
      const float ref = top == -INFINITY ? 0.f : top;
      float sum = 0.f, val = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) {
        const float2 ml = ml_s[v * R + r];
        if (ml.y == 0.f) continue;  // (no key: its output is zero)
        const float f = exp2f(ml.x - ref);
        sum += f * ml.y;
        val += f * acc_s[(v * R + r) * dp + col];
      }
      const int64_t t = w.q.s0 + token0 + i, h = (int64_t)hk * plan.G + g;
      if (whole) {
        if (col < p.DV) paged_store(static_cast<T*>(p.o) + (t * p.H + h) * p.DV + col, sum == 0.f ? 0.f : val / sum);
        if (col == 0 && p.lse != nullptr) p.lse[h * plan.T + t] = sum == 0.f ? INFINITY : (ref + log2f(sum)) * kLn2;
      } else {
        const int64_t slot = w.slot((int)blockIdx.x);
        reinterpret_cast<float*>(paged_part(p.parts, slot, false, r, col / 4))[col % 4] = val;
        if (col == 0) p.parts.ml[slot * p.parts.rows + r] = make_float2(ref, sum);
      }
    }
    if (threadIdx.x == 0) paged_note_part(plan, w, border, (int)blockIdx.x, &cut);
  }
  if (threadIdx.x == 0 && !plan.whole) p.parts.cuts[blockIdx.x] = cut;
}

constexpr int kSmemLimit = 232448 - 1024;  // (the plan's static part aside)

// Rows of a tile: four or eight where a sequence has no more to give (a
// decoding step of up to as many heads a key head), else 16, or 8 of wide values
// (128 registers of outputs a lane).  Tiles of 4, 8, 16 rows, f32: one
// sequence of 100,000 keys, 4 heads a key head 152, 193, 278 us; 16 sequences of
// 1,000 to 4,000 keys, 8 heads 73, 50, 63 us; chunks of 60 tokens on 2,000 keys
// 191, 133, 107 us.
int rows_of(const PagedProblem& pr) {
  const int64_t rows = pr.T * (pr.H / pr.Hkv);  // of a key head, all sequences
  return rows <= 4 * pr.B ? 4 : rows <= 8 * pr.B || pr.DV > 128 ? 8 : 16;
}
int dp_of(const PagedProblem& pr) { return (int)(pr.DV + 3) / 4 * 4; }

PagedPlan plan_of(const PagedProblem& pr) {
  const int R = rows_of(pr);
  PagedPlan p{};
  p.starts = pr.starts;
  p.lens = pr.lens;
  p.B = pr.B;
  p.T = pr.T;
  const int64_t most = pr.max_pages * pr.page;
  p.max_keys = most < 2147483647ll - 256 ? most : 2147483647ll - 256;  // (lengths are 32-bit)
  p.causal = pr.causal;
  p.G = (int)(pr.H / pr.Hkv);
  p.gw = p.G < R ? p.G : R;
  p.gblocks = (p.G + p.gw - 1) / p.gw;
  p.heads = (int)pr.Hkv * p.gblocks;
  p.nt = R / p.gw;
  p.tiles = 1;
  p.kt = 64;
  return p;
}

template <typename T, int R, int CPL, bool TREE>
cudaError_t launch_r(const PagedProblem& pr, int sms, cudaStream_t s) {
  SimtParams p;
  p.plan = plan_of(pr);
  p.parts = paged_parts(pr.workspace, R, dp_of(pr));
  p.table = pr.table;
  p.max_pages = pr.max_pages;
  p.pages = pr.pages;
  p.page = (int)pr.page;
  p.H = (int)pr.H;
  p.Hkv = (int)pr.Hkv;
  p.DK = (int)pr.DK;
  p.DV = (int)pr.DV;
  const int e = (int)sizeof(T);
  p.qs = (p.DK + 3) / 4 * 4;
  p.ks = (p.qs * e + 15) / 16 * 16 + 16;  // (16 more: eight keys' rows start in different banks)
  p.vs = (dp_of(pr) * e + 15) / 16 * 16;
  p.bulk = p.DK * e % 16 == 0 && p.DV * e % 16 == 0;
  p.c1 = pr.scale * kLog2e;
  p.seen = pr.seen;
  p.words = (int)pr.words;
  p.q = pr.q;
  p.k = pr.k;
  p.v = pr.v;
  p.o = pr.o;
  p.lse = pr.lse;
  const int fixed = (R * p.qs + kWarps * (kKeys + 1) * R) * 4, stage = kWarps * kKeys * (p.ks + p.vs);
  const int end = kWarps * R * (p.parts.dp + 2) * 4;  // the warps' shares, over the rings
  p.stages = (kSmemLimit - fixed) / stage;
  p.stages = p.stages > kStages ? kStages : p.stages < 1 ? 1 : p.stages;
  const int smem = fixed + (p.stages * stage > end ? p.stages * stage : end);
  const int grid = paged_grid(&p.plan, sms, kFewTiles);
  // (the limit is the kernel's, for all threads of the process: every call sets the same, whatever it needs itself)
  const auto kernel = paged_simt_kernel<T, R, CPL, TREE>;
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
  if (err != cudaSuccess) return err;
  err = launch_early(kernel, dim3((unsigned)grid), kThreads, (size_t)smem, s, p);
  if (err != cudaSuccess) return err;
  return launch_combine<T>(p.plan, p.parts, grid, p.DV, p.H, static_cast<T*>(pr.o), pr.lse, s);
}

template <typename T, bool TREE>
cudaError_t launch_m(const PagedProblem& pr, int sms, cudaStream_t s) {
  const int R = rows_of(pr);
  if (pr.DV > 128) return R == 4 ? launch_r<T, 4, 8, TREE>(pr, sms, s) : launch_r<T, 8, 8, TREE>(pr, sms, s);
  if (R == 16) return launch_r<T, 16, 4, TREE>(pr, sms, s);
  return R == 4 ? launch_r<T, 4, 4, TREE>(pr, sms, s) : launch_r<T, 8, 4, TREE>(pr, sms, s);
}

template <typename T>
cudaError_t launch_t(const PagedProblem& pr, int sms, cudaStream_t s) {
  return pr.seen != nullptr ? launch_m<T, true>(pr, sms, s) : launch_m<T, false>(pr, sms, s);
}

}  // namespace

size_t paged_simt_workspace_bytes(const PagedProblem& p) {
  return paged_workspace(plan_of(p), kFewTiles, 16, dp_of(p));
}

cudaError_t launch_paged_simt(const PagedProblem& p, cudaStream_t s) {
  const int sms = paged_sms();
  if (sms == 0) return cudaErrorInvalidValue;
  if (p.dtype == FAB_BF16) return launch_t<__nv_bfloat16>(p, sms, s);
  if (p.dtype == FAB_F16) return launch_t<__half>(p, sms, s);
  return launch_t<float>(p, sms, s);
}

uint32_t take_error_paged() {
  uint32_t v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_paged, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(g_err_paged, &z, sizeof(z));
  return v;
}

}  // namespace fab
