// fab_paged.cuh -- how the paged attention kernels share out their work, and
// how the pieces of a split row are joined.
//
// The lengths live on the device, so the kernels divide the work themselves.
// A tile is `nt` tokens times `gw` query heads of one key/value head (a row
// per pair); a unit is one tile or two (consecutive tokens) and walks its key
// tiles.  Units in order of (sequence, head, tokens) form one line, each as
// long as its work, and CTA c of G takes the piece from W c / G to W (c+1) / G
// of that line, so every CTA has the same work whatever the lengths are.  A
// unit's work is a start and an end and its key tiles, in quarters of what a
// key tile of a unit of two tiles takes: measured at 1.2 us for that, 0.9 us
// for one of a unit of one tile (whose streams wait for memory or for one
// another rather than for the tensor core) and 3 us for the start and the end,
// by a fit over the CTAs of a batch of mixed chunks at width 64.  The same figures
// serve width 128 and the CUDA cores, where they were not fitted but tried:
// starts and ends counted half, as they are, double: mixed chunks at width 128 98, 83 and 84
// us, 200 short decoding sequences 83, 77 and 79, 16 in f32 68, 62 and 64, mixed f32
// chunks 463, 437 and 400 (the one that another figure would serve).  A unit cut by
// a border leaves unnormalised partial results (output, maximum, sum) in the
// workspace, at most two to a CTA, which paged_combine_kernel joins.
#pragma once

#include <type_traits>

#include "fab_device.cuh"
#include "fab_internal.h"
#include "fab_launch.cuh"

namespace fab {

FAB_DEV int paged_lead(int width) { return width == 2 ? 10 : 6; }  // work of a start and an end,
FAB_DEV int paged_step(int width) { return width == 2 ? 4 : 3; }   // of a key tile
constexpr int kPagedMaxGrid = 304;  // CTAs that the workspace has room for

// What planning needs to know.
struct PagedPlan {
  const int32_t *starts, *lens;
  int64_t B, T, max_keys;  // max_keys: keys that a row of the table can hold
  int causal;
  int G, gw, gblocks;  // query heads of a key/value head, of a tile; tiles over them
  int heads;           // Hkv * gblocks
  int nt, tiles;       // tokens of a tile, tiles of a unit (1 or 2)
  int kt;              // keys of a key tile
  int snap;            // a unit of two tiles is not cut within so many key tiles of its ends
  int whole;           // 1: every unit counts the same and none is cut (then nothing is left to join)
};

struct PagedSeq {
  int s0, n;     // first new token, how many
  int last0;     // last key its first new token sees under a causal mask (may be negative)
  int len;       // keys
};

FAB_DEV PagedSeq paged_seq(const PagedPlan& p, int b) {
  PagedSeq q;
  // (clamped: starts and lengths out of range must not reach an address)
  const int64_t T = p.T, a = p.starts[b], e = p.starts[b + 1];
  const int64_t s0 = a < 0 ? 0 : a > T ? T : a, s1 = e < s0 ? s0 : e > T ? T : e;
  const int64_t len = p.lens[b];
  q.s0 = (int)s0;
  q.n = (int)(s1 - s0);
  q.last0 = (int)(len - q.n < -q.n - 1 ? -q.n - 1 : len - q.n);
  q.len = (int)(len < 0 ? 0 : len > p.max_keys ? p.max_keys : len);
  return q;
}

FAB_DEV int paged_units(const PagedPlan& p, const PagedSeq& q) {
  const int per = p.nt * p.tiles;
  return (q.n + per - 1) / per;
}
// Tiles of unit i (one where its tokens fit one tile), and its key tiles.
FAB_DEV int paged_width(const PagedPlan& p, const PagedSeq& q, int i) {
  return p.tiles == 2 && q.n - i * 2 * p.nt > p.nt ? 2 : 1;
}
FAB_DEV int paged_key_tiles(const PagedPlan& p, const PagedSeq& q, int i) {
  int end = q.len;
  if (p.causal) {
    const int per = p.nt * p.tiles, hi = (i + 1) * per < q.n ? (i + 1) * per : q.n;
    if (q.last0 + hi < end) end = q.last0 + hi;
  }
  return end > 0 ? (end + p.kt - 1) / p.kt : 1;
}

// Place on the line: unit i of head `head` of sequence b, which begins at u0.
struct PagedPlace {
  int b, head, i;
  int64_t u0;
};

struct PagedShared {
  int64_t sums[32];
  int64_t total;
  PagedPlace at;
};

// Length on the line of unit i.
FAB_DEV int paged_length(const PagedPlan& p, const PagedSeq& q, int i) {
  if (p.whole) return 1;
  const int width = paged_width(p, q, i);
  return paged_step(width) * paged_key_tiles(p, q, i) + paged_lead(width);
}

// Length on the line of one head of the sequence of each lane; whole warps.
FAB_DEV int64_t paged_head_length(const PagedPlan& p, const PagedSeq& q) {
  const int units = paged_units(p, q);
  int64_t len = 0;
  constexpr int kOwn = 12;  // units that a lane adds up by itself
  if (units <= kOwn) {
#pragma unroll 1
    for (int i = 0; i < units; ++i) len += paged_length(p, q, i);
  }
  // the lanes of a warp share the longer ones' units
  for (unsigned left = __ballot_sync(0xffffffffu, units > kOwn); left != 0; left &= left - 1) {
    const int src = __ffs((int)left) - 1;
    PagedSeq x;
    x.s0 = 0;
    x.n = __shfl_sync(0xffffffffu, q.n, src);
    x.last0 = __shfl_sync(0xffffffffu, q.last0, src);
    x.len = __shfl_sync(0xffffffffu, q.len, src);
    int64_t sum = 0;
#pragma unroll 1
    for (int i = (int)lane_id(), k = paged_units(p, x); i < k; i += 32) sum += paged_length(p, x, i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((int)lane_id() == src) len = sum;
  }
  return len;
}

// Where CTAs' pieces begin.
struct PagedBorders {
  int64_t q;
  uint32_t r, G;
  FAB_DEV PagedBorders(int64_t W, int grid) {
    G = (uint32_t)grid;
    q = W < (int64_t(1) << 32) ? (int64_t)((uint32_t)W / G) : W / grid;
    r = (uint32_t)(W - q * grid);
  }
  FAB_DEV int64_t operator()(int c) const { return q * c + (int64_t)(r * (uint32_t)c / G); }
};

// The line's length in s->total.  Called by the whole block (NT threads); `mine`
// gets the length of a head of sequence threadIdx.x.
template <int NT>
FAB_DEV void paged_total(const PagedPlan& p, PagedShared* s, int64_t* mine) {
  int64_t sum = 0;
  for (int64_t b0 = 0; b0 < p.B; b0 += NT) {
    const int64_t b = b0 + threadIdx.x;
    PagedSeq q{0, 0, 0, 0};
    if (b < p.B) q = paged_seq(p, (int)b);
    const int64_t one = paged_head_length(p, q);
    if (b0 == 0) *mine = one;
    sum += one * p.heads;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) s->sums[threadIdx.x >> 5] = sum;
  __syncthreads();
  int64_t w = 0;
  for (int i = 0; i < NT / 32; ++i) w += s->sums[i];
  if (threadIdx.x == 0) s->total = w;
  __syncthreads();
}

// The unit that holds `pos` (0 <= pos < s->total) in s->at.  Whole block.
template <int NT>
FAB_DEV void paged_locate(const PagedPlan& p, PagedShared* s, int64_t mine, int64_t pos) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t base = 0;
  for (int64_t b0 = 0; b0 < p.B; b0 += NT) {
    const int64_t b = b0 + threadIdx.x;
    int64_t one = mine;
    if (b0 > 0) {
      PagedSeq q{0, 0, 0, 0};
      if (b < p.B) q = paged_seq(p, (int)b);
      one = paged_head_length(p, q);
    }
    const int64_t all = one * p.heads;
    int64_t incl = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) s->sums[warp] = incl;
    __syncthreads();
    int64_t before = base;
    for (int i = 0; i < NT / 32; ++i) {
      if (i < warp) before += s->sums[i];
      base += s->sums[i];
    }
    const int64_t first = before + incl - all;
    const unsigned hit = __ballot_sync(0xffffffffu, all > 0 && pos >= first && pos < first + all);
    if (hit != 0) {  // in this warp: its lanes look for the unit together
      const int src = __ffs((int)hit) - 1;
      const int64_t f = __shfl_sync(0xffffffffu, first, src), head_len = __shfl_sync(0xffffffffu, one, src);
      const int bb = (int)(b0 + warp * 32 + src);
      const PagedSeq q = paged_seq(p, bb);
      int64_t d = pos - f;
      const int head = d < (int64_t(1) << 32) && head_len < (int64_t(1) << 32)
                           ? (int)((uint32_t)d / (uint32_t)head_len)
                           : (int)(d / head_len);
      int64_t u0 = f + head * head_len;
      for (int i0 = 0;; i0 += 32) {
        const int64_t len = i0 + lane < paged_units(p, q) ? paged_length(p, q, i0 + lane) : 0;
        int64_t end = len;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t up = __shfl_up_sync(0xffffffffu, end, o);
          if (lane >= o) end += up;
        }
        const unsigned in = __ballot_sync(0xffffffffu, pos < u0 + end);
        if (in != 0) {
          if (lane == __ffs((int)in) - 1) {
            s->at.b = bb;
            s->at.head = head;
            s->at.i = i0 + lane;
            s->at.u0 = u0 + end - len;
          }
          break;
        }
        if (i0 >= paged_units(p, q)) {  // only if the lengths changed under the kernel
          s->at = PagedPlace{bb, head, 0, u0};
          break;
        }
        u0 += __shfl_sync(0xffffffffu, end, 31);
      }
    }
    __syncthreads();
    if (base > pos) break;
  }
}

// Walks a CTA's piece of the line, unit by unit.
struct PagedWalk {
  PagedSeq q;
  PagedPlace at;
  int width, ntiles;   // of the present unit
  int j0, j1;          // its key tiles that lie in the piece
  int units;           // of a head of the sequence
  int snap;
  bool uncut;

  FAB_DEV void load(const PagedPlan& p) {
    width = paged_width(p, q, at.i);
    ntiles = paged_key_tiles(p, q, at.i);
    uncut = p.whole != 0;
    snap = p.snap;
  }
  FAB_DEV void begin(const PagedPlan& p, const PagedPlace& start) {
    at = start;
    q = paged_seq(p, at.b);
    units = paged_units(p, q);
    load(p);
  }
  // Key tiles of the present unit before `pos` on the line.  A border near an end of
  // a unit of two row tiles moves there: two parts written and joined cost more
  // than a few key tiles (width 128, two key tiles: a prompt of 4 x 2,048 tokens 132
  // -> 127 us, chunks of 500 to 900 tokens 35.7 -> 30.8; width 64, one: mixed chunks 55.1 ->
  // 54.4, with two 55.4).
  FAB_DEV int tiles_before(int64_t pos) const {
    if (uncut) return pos > at.u0 ? ntiles : 0;
    const int64_t d = pos - at.u0 - paged_lead(width);
    if (d <= 0) return 0;
    if (d >= (int64_t)paged_step(width) * ntiles) return ntiles;
    if (width == 1) return ((int)d + 2) / 3;
    const int t = ((int)d + 3) / 4;
    if (2 * t < ntiles) return t <= snap ? 0 : t;
    return ntiles - t <= snap ? ntiles : t;
  }
  // The part of the piece [p0, p1) that lies in the present unit.
  FAB_DEV bool piece(int64_t p0, int64_t p1) {
    if (at.u0 >= p1) return false;
    j0 = tiles_before(p0);
    j1 = tiles_before(p1);
    return true;
  }
  // The next unit (its j0, j1 are not set); false at the end of the line.
  FAB_DEV bool next(const PagedPlan& p) {
    at.u0 += uncut ? 1 : (int64_t)paged_step(width) * ntiles + paged_lead(width);
    if (++at.i == units) {
      at.i = 0;
      if (++at.head == p.heads) {
        at.head = 0;
        do {
          if (++at.b >= p.B) return false;
          q = paged_seq(p, at.b);
          units = paged_units(p, q);
        } while (units == 0);
      }
    }
    load(p);
    return true;
  }
  // From the present unit on, the first with key tiles in the piece; false past the piece.
  FAB_DEV bool seek(const PagedPlan& p, int64_t p0, int64_t p1) {
    for (;;) {
      if (!piece(p0, p1)) return false;
      if (j0 < j1) return true;
      if (!next(p)) return false;
    }
  }
  FAB_DEV bool whole() const { return j0 == 0 && j1 == ntiles; }
  // The piece's partial slot: 2c for a unit that began before it, else 2c + 1.
  FAB_DEV int slot(int c) const { return 2 * c + (j0 == 0 ? 1 : 0); }
};

// What a CTA leaves for the combine kernel: whether slot 2c holds a part of a
// unit that began before it, and the cut unit whose first part it holds.
struct PagedCut {
  int head_part;  // 1: slot 2c holds a part
  int last;       // the last CTA that holds a part of the unit in slot 2c + 1; 0: no such unit
  int s0, n;      // the unit: its sequence's tokens,
  int head, token0, rows;  // its head and tokens, how many rows
  int gaps;       // 1: pieces shorter than a key tile's work, some CTAs up to `last` may hold no part
};

// Partial results: outputs, and (maximum in log2 units, sum) pairs by row.  The
// outputs of a unit of more than 32 rows lie by 4 columns, then by row, as the writers'
// lanes are rows (units of two row tiles, mixed chunks: 53.7 -> 51.5 us; of one 51.2 -> 50.4);
// those of fewer rows row by row (one sequence of 131,000 keys 89.5 us, the other
// way 99.5).  On the CUDA cores, whose tiles have 16 rows at most, always so.
struct PagedParts {
  float* out;
  float2* ml;
  PagedCut* cuts;
  int rows, dp;  // rows of a slot, columns (a multiple of 4)
};
FAB_DEV float4* paged_part(const PagedParts& x, int64_t slot, bool by_columns, int row, int c4) {
  const int n4 = x.dp / 4;
  return reinterpret_cast<float4*>(x.out) + slot * (n4 * x.rows) + (by_columns ? c4 * x.rows + row : row * n4 + c4);
}
// Rows of a unit that belong to a token: `left` tokens of its sequence from its first on.
FAB_DEV int paged_live(int left, int gw, int rows) {
  const int64_t live = (int64_t)left * gw;
  return live < rows ? (int)live : rows;
}
FAB_DEV bool paged_by_columns(int live) { return live > 32; }
inline size_t paged_parts_bytes(int rows, int dp) {
  return (size_t)(2 * kPagedMaxGrid) * rows * (dp + 2) * sizeof(float) + kPagedMaxGrid * sizeof(PagedCut);
}
inline PagedParts paged_parts(void* workspace, int rows, int dp) {
  PagedParts x;
  x.out = static_cast<float*>(workspace);
  x.ml = reinterpret_cast<float2*>(x.out + (size_t)(2 * kPagedMaxGrid) * rows * dp);
  x.cuts = reinterpret_cast<PagedCut*>(x.ml + (size_t)(2 * kPagedMaxGrid) * rows);
  x.rows = rows;
  x.dp = dp;
  return x;
}

// Adds what the walk's present unit says to CTA c's note.
FAB_DEV void paged_note_part(const PagedPlan& p, const PagedWalk& w, const PagedBorders& border, int c, PagedCut* cut) {
  if (w.j0 > 0) cut->head_part = 1;
  if (w.j0 == 0 && w.j1 < w.ntiles) {
    int last = c + 1;
    while (last + 1 < (int)gridDim.x && w.tiles_before(border(last + 1)) < w.ntiles) ++last;
    cut->last = last;
    cut->s0 = w.q.s0;
    cut->n = w.q.n;
    cut->head = w.at.head;
    cut->token0 = w.at.i * p.nt * p.tiles;
    cut->rows = w.width * p.nt * p.gw;
    cut->gaps = border.q < 4;
  }
}

FAB_DEV void paged_store(float* p, float x) { *p = x; }
FAB_DEV void paged_store(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
FAB_DEV void paged_store(__half* p, float x) { *p = __float2half_rn(x); }

constexpr int kCombineThreads = 256;

// Joins the cut unit whose first part CTA blockIdx.x holds, if there is one (where
// units are few, `listed`: the blockIdx.x-th cut unit):
// out = sum 2^(m_i - M) out_i / sum 2^(m_i - M) l_i over its parts.  Where the parts lie by
// columns (16-bit types on the tensor cores, DV a multiple of 8) a thread takes 8 columns of a row and its neighbours the
// next rows; where they lie by rows, LPR lanes share a row, four columns at a time.
// blockIdx.y of gridDim.y shares the work.  U parts are fetched at once: eight where
// a unit has several, two, which leaves registers for six blocks an SM, where most
// have two (four in both: one sequence of 131,000 keys and 64 new tokens 107.4 -> 106.6 us
// with eight, 32 drafts of 8 to 64 tokens 63.7 -> 62.4 and mixed chunks 52.1 -> 51.3 with two).
// Launched while the attention kernel still runs; waits for it first.
template <typename T, int LPR, int U>
__global__ void __launch_bounds__(kCombineThreads, U == 2 ? 6 : 2) paged_combine_kernel(const PagedPlan p, const PagedParts parts,
                                                                        int ctas, int listed, int DV, int H, T* o, float* lse) {
  constexpr int RPB = kCombineThreads / LPR;  // rows a block takes at once
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int c = (int)blockIdx.x;
  if (U == 8 && listed) {  // (as many blocks as there can be units: most CTAs hold no unit's first part)
    __shared__ int found_s, counts_s[kCombineThreads / 32];
    const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
    if (threadIdx.x == 0) found_s = -1;
    int before = 0;
    for (int c0 = 0; c0 < ctas; c0 += kCombineThreads) {
      const int at = c0 + (int)threadIdx.x;
      const bool is = at < ctas && parts.cuts[at].last != 0;
      const uint32_t of_warp = __ballot_sync(0xffffffffu, is);
      __syncthreads();
      if (lane == 0) counts_s[warp] = __popc(of_warp);
      __syncthreads();
      int rank = before + __popc(of_warp & ((1u << lane) - 1u));
#pragma unroll
      for (int w = 0; w < kCombineThreads / 32; ++w) {
        if (w < warp) rank += counts_s[w];
        before += counts_s[w];
      }
      if (is && rank == (int)blockIdx.x) found_s = at;
    }
    __syncthreads();
    c = found_s;
    if (c < 0) return;
  }
  const PagedCut cut = parts.cuts[c];
  if (cut.last == 0) return;
  const int sub = (int)threadIdx.x % LPR;
  const int tile_rows = p.nt * p.gw;
  const int hk = cut.head / p.gblocks, gb = cut.head - hk * p.gblocks;
  const int live = paged_live(cut.n - cut.token0, p.gw, cut.rows);
  if (sizeof(T) == 2 && paged_by_columns(live)) {  // (f32's units have 16 rows at most)
    const int nc8 = DV / 8, items = (live + 31) / 32 * 32 * nc8;
    for (int x = (int)blockIdx.y * kCombineThreads + (int)threadIdx.x; x < items; x += (int)gridDim.y * kCombineThreads) {
      const int rblk = x / (32 * nc8), c8 = x / 32 - rblk * nc8, at = rblk * 32 + x % 32;
      if (at >= live) continue;
      const int tile = at >= tile_rows ? 1 : 0, r = at - tile * tile_rows, i = r / p.gw;
      const int token = cut.token0 + tile * p.nt + i, g = gb * p.gw + r - i * p.gw;
      if (token >= cut.n || g >= p.G) continue;
      const int row = tile * (parts.rows / 2) + r;
      float m = -INFINITY, l = 0.f, acc[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = 0.f;
      for (int k0 = c; k0 <= cut.last; k0 += U) {
        float2 ml[U];
        float4 v[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int k = k0 + u;
          ml[u] = make_float2(-INFINITY, 0.f);
          v[u][0] = v[u][1] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k <= cut.last && (k == c || !cut.gaps || parts.cuts[k].head_part)) {
            const int64_t slot = k == c ? 2 * k + 1 : 2 * k;
            ml[u] = parts.ml[slot * parts.rows + row];
            v[u][0] = *paged_part(parts, slot, true, row, c8 * 2);
            v[u][1] = *paged_part(parts, slot, true, row, c8 * 2 + 1);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (ml[u].y == 0.f) continue;  // nothing to add, whatever the row holds
          const float top = fmaxf(m, ml[u].x);
          const float a = m == -INFINITY ? 0.f : exp2f(m - top), b = exp2f(ml[u].x - top);
          const float add[8] = {v[u][0].x, v[u][0].y, v[u][0].z, v[u][0].w,
                                v[u][1].x, v[u][1].y, v[u][1].z, v[u][1].w};
          l = l * a + ml[u].y * b;
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] = acc[e] * a + add[e] * b;
          m = top;
        }
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int64_t t = cut.s0 + token, h = (int64_t)hk * p.G + g;
      constexpr bool f16 = std::is_same<T, __half>::value;
      *reinterpret_cast<uint4*>(o + (t * H + h) * DV + c8 * 8) =
          make_uint4(pack2<f16>(acc[0] * inv, acc[1] * inv), pack2<f16>(acc[2] * inv, acc[3] * inv),
                     pack2<f16>(acc[4] * inv, acc[5] * inv), pack2<f16>(acc[6] * inv, acc[7] * inv));
      if (lse != nullptr && c8 == 0) lse[h * p.T + t] = l == 0.f ? INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
    return;
  }
  for (int x = (int)blockIdx.y * RPB + (int)threadIdx.x / LPR; x < cut.rows; x += (int)gridDim.y * RPB) {
    const int tile = x >= tile_rows ? 1 : 0, r = x - tile * tile_rows, i = r / p.gw;
    const int token = cut.token0 + tile * p.nt + i, g = gb * p.gw + r - i * p.gw;
    if (token >= cut.n || g >= p.G) continue;
    const int row = tile * (parts.rows / 2) + r;
    const int64_t t = cut.s0 + token, h = (int64_t)hk * p.G + g;
    T* dst = o + (t * H + h) * DV;
    for (int c0 = sub * 4; c0 < parts.dp; c0 += LPR * 4) {
      float m = -INFINITY, l = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k0 = c; k0 <= cut.last; k0 += U) {
        float2 ml[U];
        float4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int k = k0 + u;
          ml[u] = make_float2(-INFINITY, 0.f);
          v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k <= cut.last && (k == c || !cut.gaps || parts.cuts[k].head_part)) {
            const int64_t at = (int64_t)(k == c ? 2 * k + 1 : 2 * k) * parts.rows + row;
            ml[u] = parts.ml[at];
            v[u] = *reinterpret_cast<const float4*>(parts.out + at * parts.dp + c0);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (ml[u].y == 0.f) continue;  // nothing to add, whatever the row holds
          const float top = fmaxf(m, ml[u].x);
          const float a = m == -INFINITY ? 0.f : exp2f(m - top), b = exp2f(ml[u].x - top);
          l = l * a + ml[u].y * b;
          acc.x = acc.x * a + v[u].x * b;
          acc.y = acc.y * a + v[u].y * b;
          acc.z = acc.z * a + v[u].z * b;
          acc.w = acc.w * a + v[u].w * b;
          m = top;
        }
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const float out[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c0 + e < DV) paged_store(dst + c0 + e, out[e]);
      if (lse != nullptr && c0 == 0) lse[h * p.T + t] = l == 0.f ? INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
  }
}

// Units of a call at most.
inline int64_t paged_most_units(const PagedPlan& p) { return (p.T / (p.nt * p.tiles) + p.B) * p.heads; }

// Sets plan.whole and returns the grid.  Short calls are not cut: a CTA then walks
// `few` key tiles more, but nothing is left to join and a launch is saved.
// Decoding: units of up to `few` key tiles, two to a CTA at most; chunks, whose
// parts are of whole 128-row tiles: up to 16 key tiles, one unit to a CTA.  Cut and whole,
// bf16, width 128: one sequence of 500 keys 12.6 and 11.5 us, of 1,000 15.6 and
// 14.8, of 2,000 18.2 and 22.4; 36 sequences of up to 500 (288 units) 25.8 and 20.8,
// 64 of up to 1,000 (512 units) 40.7 and 48.5; chunks of 50 to 400 tokens behind
// up to 500 keys 25.0 and 16.6, behind up to 2,000 29.7 and 26.4.  f32, 4 tiles at most:
// one sequence at width 64 of 128 keys 9.8 and 8.4, of 256 12.4 and 11.6, of 500 18.5 and 18.5;
// at width 128 with 32 heads of 200 keys 13.8 and 14.0, of 256 13.8 and 13.2, of 500 16.4 and
// 20.6; 4 sequences of 500 14.6 and 21.1; 16 of 200 18.2 and 14.4, of 500 24.8 and 21.2.
inline int paged_grid(PagedPlan* plan, int sms, int few) {
  const int64_t units = paged_most_units(*plan);
  const int64_t tiles = (plan->max_keys + plan->kt - 1) / plan->kt;                    // of a unit, at most
  const int most = sms < kPagedMaxGrid ? sms : kPagedMaxGrid;
  const bool chunks = plan->tiles == 2 && plan->T > plan->B * plan->nt;
  plan->whole = chunks ? tiles <= 16 && units <= most : tiles <= few && units <= 2 * most;
  if (units >= most) return most;
  const int64_t pieces = plan->whole ? units : 2 * units * (tiles < most ? tiles : most);  // that are worth a CTA
  return (int)(pieces < most ? pieces : most);
}

// SMs of the current device, 0 without one.
inline int paged_sms() {
  int dev = 0, sms = 0;
  const bool ok = cudaGetDevice(&dev) == cudaSuccess &&
                  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
  return ok ? sms : 0;
}

// Workspace of a call on the current device: none where no unit is cut.
inline size_t paged_workspace(PagedPlan plan, int few, int rows, int dp) {
  const int sms = paged_sms();
  plan.whole = 0;
  if (sms > 0) paged_grid(&plan, sms, few);
  return plan.whole ? 0 : paged_parts_bytes(rows, dp);
}

// Enqueues the combine kernel behind an attention kernel of `grid` CTAs.
template <typename T>
cudaError_t launch_combine(const PagedPlan& plan, const PagedParts& parts, int grid, int DV, int H, T* o, float* lse,
                           cudaStream_t s) {
  if (grid < 2 || plan.whole) return cudaSuccess;  // nothing is cut
  // (as many blocks as a unit of one row tile has use for, which one of two has too)
  const int rows = plan.nt * plan.gw;
  const int per = kCombineThreads / (parts.dp <= 64 ? 16 : 32);  // rows of a block at once
  const int64_t units = paged_most_units(plan);
  const bool pairs = units > grid;  // (most cut units then have two parts)
  // A block costs a place on an SM for 2 us even where its CTA holds no unit's first part.
  // Where units are far fewer than CTAs, blocks are launched for as many as there can be, and look
  // for theirs: one sequence of 131,000 keys and 64 new tokens 104.2 -> 102.2 us, of 500
  // keys and 7 new ones in f32 20.1 -> 18.4; not worth its look for one new token (86.9 ->
  // 87.8), nor for half as many units as CTAs (f32 chunks 21.3 -> 21.9).
  const int listed = !pairs && units * 4 <= grid && plan.T > plan.B ? 1 : 0;
  const dim3 g((unsigned)(listed ? units : grid - 1), (unsigned)((rows + per - 1) / per));
  const auto kernel = parts.dp <= 64 ? (pairs ? paged_combine_kernel<T, 16, 2> : paged_combine_kernel<T, 16, 8>)
                                     : (pairs ? paged_combine_kernel<T, 32, 2> : paged_combine_kernel<T, 32, 8>);
  return launch_early(kernel, g, kCombineThreads, 0, s, plan, parts, grid - 1, listed, DV, H, o, lse);
}

}  // namespace fab
