// fab_pages.cu -- drafts and pages of a paged key/value cache: who sees whom
// in a drafted tree, keeping the accepted path's rows, and which sequence
// holds which page (forked, grown, cut, freed, copied before it is written).
#include <limits.h>

#include "fab.h"
#include "fab_device.cuh"
#include "fab_internal.h"
#include "fab_launch.cuh"

namespace fab {
namespace {

__device__ uint32_t g_err_pages;

// ------------------------------------------------------------------ trees
//
//   seen(i) = {i} + seen(parent(i))
//
// A sequence's tokens are taken in blocks of 32, a word of `seen` each.  A warp
// first finds each token's ancestors in its own block, by doubling: five
// exchanges of (mask, first ancestor not yet in it) reach 32 steps back.  What
// is left of a path then takes one step per block instead of one per
// token: thread i walks from block to block and writes words as it goes.

constexpr int kTreeThreads = 128;
constexpr int kTreeWords = 8;  // words that a thread writes

__global__ void __launch_bounds__(kTreeThreads) draft_tree_kernel(const int32_t* starts, const int32_t* parents,
                                                                  int64_t B, int64_t T, int words, uint32_t* seen) {
  extern __shared__ int2 node[];  // of each token: its ancestors in its block, the first one before the block
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0 && blockIdx.y == 0)
    check_starts(starts, B, T, (int)threadIdx.x, kTreeThreads, &g_err_pages);
  const int64_t a = starts[blockIdx.x], z = starts[blockIdx.x + 1];
  const int64_t s0 = a < 0 ? 0 : a > T ? T : a, s1 = z < s0 ? s0 : z > T ? T : z;
  if (s1 - s0 > (int64_t)words * 32 && threadIdx.x == 0) atomicOr(&g_err_pages, kErrIndex);
  const int n = (int)(s1 - s0 < (int64_t)words * 32 ? s1 - s0 : (int64_t)words * 32);
  // this CTA's blocks are y, y + gridDim.y, ...; it needs all blocks up to its last one's
  const int blocks = (n + 31) / 32;
  if ((int)blockIdx.y >= blocks) return;
  const int top = (blocks - 1 - (int)blockIdx.y) / (int)gridDim.y * (int)gridDim.y + (int)blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int blk = warp; blk <= top; blk += kTreeThreads / 32) {
    const int i = blk * 32 + lane;
    int up = -1;
    if (i < n) {
      up = parents[s0 + i];
      if (up < -1 || up >= i) {  // (no ancestor then)
        up = -1;
        atomicOr(&g_err_pages, kErrIndex);
      }
    }
    uint32_t mask = 1u << lane;
#pragma unroll
    for (int step = 0; step < 5; ++step) {
      const bool in = up >= blk * 32;
      const uint32_t more = __shfl_sync(0xffffffffu, mask, in ? up & 31 : lane);
      const int next = __shfl_sync(0xffffffffu, up, in ? up & 31 : lane);
      if (in) mask |= more, up = next;
    }
    node[i] = make_int2((int)mask, up);
  }
  __syncthreads();
  const int groups = (words + kTreeWords - 1) / kTreeWords;
  const int per = 32 * groups;  // threads of a block of tokens
  const int mine = (blocks - 1 - (int)blockIdx.y) / (int)gridDim.y + 1;
  for (int x = (int)threadIdx.x; x < mine * per; x += kTreeThreads) {
    const int blk = x / per * (int)gridDim.y + (int)blockIdx.y, y = x % per;
    const int i = blk * 32 + y / groups, w0 = y % groups * kTreeWords;
    if (i >= n) continue;
    uint32_t out[kTreeWords];
    int at = i;
    int2 d = node[at];
    auto step = [&]() {
      at = d.y;
      if (at >= 0) d = node[at];
    };
    while (at >= 0 && at >> 5 >= w0 + kTreeWords) step();
#pragma unroll
    for (int w = kTreeWords - 1; w >= 0; --w) {
      out[w] = 0u;
      if (at >= 0 && at >> 5 == w0 + w) {
        out[w] = (uint32_t)d.x;
        step();
      }
    }
    uint32_t* to = seen + (s0 + i) * words + w0;
    if (words % 4 == 0) {  // (rows start at 16 bytes)
#pragma unroll
      for (int w = 0; w < kTreeWords; w += 4)
        if (w0 + w < words) *reinterpret_cast<uint4*>(to + w) = make_uint4(out[w], out[w + 1], out[w + 2], out[w + 3]);
    } else {
#pragma unroll
      for (int w = 0; w < kTreeWords; ++w)
        if (w0 + w < words) to[w] = out[w];
    }
  }
}

// ------------------------------------------------------------------ the accepted path
//
// Row j of a path lies at or behind row j of its destination, paths ascend, and
// no two paths share a row: rows are moved in order, a batch read whole before it
// is written, by one warp for each (layer, head, keys or values), and nothing is
// overwritten before it has been read.

constexpr int kMoveThreads = 256;
constexpr int kMoves = 64;  // rows of a path listed at once

template <typename V>
__global__ void __launch_bounds__(kMoveThreads) paged_accept_kernel(const CacheProblem p, int kv, int vv) {
  __shared__ int64_t from_s[kMoves], to_s[kMoves];  // rows, as if of head 0
  __shared__ int count_s, next_s;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0 && blockIdx.y == 0)
    check_starts(p.starts, p.B, p.T, (int)threadIdx.x, kMoveThreads, &g_err_pages);
  const int64_t b = blockIdx.x;
  const int64_t s0 = p.starts[b], n = (int64_t)p.starts[b + 1] - s0, len = p.lens[b], last = n > 0 ? p.last[b] : -1;
  const int64_t past = len - n;
  const bool bad = s0 < 0 || n < 0 || s0 + n > p.T || past < 0 || len > p.max_pages * p.page || last < -1 ||
                   last >= n || last >= 32 * p.words;
  if (bad) {
    if (threadIdx.x == 0) {
      atomicOr(&g_err_pages, kErrIndex);
      if (blockIdx.y == 0) p.lens_out[b] = (int32_t)len;
    }
    return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t* row = p.seen + (s0 + (last < 0 ? 0 : last)) * p.words;
  const int words = (int)(last >> 5) + 1;  // (none for -1)
  // items: (layer, head) of keys and of values, the warps' shares alternate between the two
  const int64_t items = p.layers * p.Hkv;
  const int64_t i0 = items * blockIdx.y / gridDim.y, i1 = items * (blockIdx.y + 1) / gridDim.y;
  const bool values = warp & 1;
  const int64_t sub = warp >> 1, subs = kMoveThreads / 64;
  const int64_t w0 = i0 + (i1 - i0) * sub / subs, w1 = i0 + (i1 - i0) * (sub + 1) / subs;
  const uint32_t nv = values ? vv : kv;  // vectors of a row
  V* const base = static_cast<V*>(values ? p.v : p.k);
  const int64_t ld = (values ? p.ldv : p.ldk) / (int64_t)((values ? p.DV : p.DK) / nv);  // vectors between layers
  // a batch is whole rows, as many as U vectors a lane hold; this lane's of them
  constexpr int U = 8;
  const uint32_t rows = 32 * U / nv;
  uint32_t ru[U], cu[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    ru[u] = (uint32_t)(u * 32 + lane) / nv;
    cu[u] = (uint32_t)(u * 32 + lane) - ru[u] * nv;
  }
  int64_t taken = 0;  // rows of the path before the list
  for (int word = 0; word < words;) {
    // warp 0 lists the next rows that move, 32 candidates at a time
    if (warp == 0) {
      int count = 0;
      for (; word < words && count <= kMoves - 32; ++word) {
        uint32_t bits = __ldg(row + word);
        if (word == words - 1 && (last & 31) != 31) bits &= (2u << (last & 31)) - 1u;
        const int64_t to = past + taken + __popc(bits & ((1u << lane) - 1u)), from = past + word * 32 + lane;
        const bool moves = (bits >> lane & 1u) && to != from;
        const uint32_t moving = __ballot_sync(0xffffffffu, moves);
        if (moves) {
          const int32_t a = p.table[b * p.max_pages + from / p.page], z = p.table[b * p.max_pages + to / p.page];
          const int at = count + __popc(moving & ((1u << lane) - 1u));
          const bool ok = a >= 0 && a < p.pages && z >= 0 && z < p.pages;
          if (!ok) atomicOr(&g_err_pages, kErrIndex);  // (the row stays where it is)
          from_s[at] = ok ? ((int64_t)a * p.Hkv) * p.page + from % p.page : -1;
          to_s[at] = ok ? ((int64_t)z * p.Hkv) * p.page + to % p.page : -1;
        }
        count += __popc(moving);
        taken += __popc(bits);
      }
      if (lane == 0) {
        count_s = count;
        next_s = word;
      }
    }
    __syncthreads();
    const uint32_t m = (uint32_t)count_s;
    word = next_s;
    if (m > 0) {
      const uint32_t total = (uint32_t)(w1 - w0) * m;
      for (uint32_t r0 = 0; r0 < total; r0 += rows) {
        V v[U];
        int64_t dst[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t r = r0 + ru[u];
          dst[u] = -1;
          if (ru[u] < rows && r < total) {
            const uint32_t item = (uint32_t)w0 + r / m, mv = r % m;
            const uint32_t layer = item / (uint32_t)p.Hkv, head = item - layer * (uint32_t)p.Hkv;
            const int64_t from = from_s[mv], at = layer * ld + (int64_t)head * p.page * nv + cu[u];
            if (from >= 0) {
              v[u] = base[at + from * nv];
              dst[u] = at + to_s[mv] * nv;
            }
          }
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (dst[u] >= 0) base[dst[u]] = v[u];
        __syncwarp();
      }
    }
    __syncthreads();
  }
  if (blockIdx.y == 0 && threadIdx.x == 0) p.lens_out[b] = (int32_t)(past + taken);
}

// ------------------------------------------------------------------ pages
//
// Three kernels.  `release` drops and adds references as rows lose and gain
// entries, `plan` (which alone sees all rows) settles who keeps a page that
// several rows would go on writing, and hands out the free pages in order of
// (row, entry), `fill` writes the table and copies what has to be copied.

struct ReserveRow {
  int first;   // the first entry that gets a fresh page
  int rank;    // its place among all fresh ones
};
struct ReserveCopy {
  int from, rows;  // page, rows of it
  int rank;        // the fresh page's place
  int pad;
};
struct ReserveSpace {
  int32_t* carried;     // [B][max_pages], of rows that continue another one
  int32_t* free_pages;  // the free ones, lowest first
  ReserveRow* rows;     // [B]
  ReserveCopy* copies;  // [B]
  int32_t* counts;      // free pages, copies
};
ReserveSpace reserve_space(const CacheProblem& p, size_t* bytes) {
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t was = at;
    at += (n + 255) / 256 * 256;
    return static_cast<char*>(p.workspace) + was;
  };
  ReserveSpace x;
  x.copies = reinterpret_cast<ReserveCopy*>(take((size_t)p.B * sizeof(ReserveCopy)));
  x.rows = reinterpret_cast<ReserveRow*>(take((size_t)p.B * sizeof(ReserveRow)));
  x.counts = reinterpret_cast<int32_t*>(take(2 * sizeof(int32_t)));
  x.free_pages = reinterpret_cast<int32_t*>(take((size_t)p.pages * sizeof(int32_t)));
  x.carried = reinterpret_cast<int32_t*>(take((size_t)(p.B * p.max_pages) * sizeof(int32_t)));
  if (bytes) *bytes = at;
  return x;
}

// What a row's numbers say.
struct RowPlan {
  int64_t source;   // the row it continues, -1: none
  int first, end;   // entries carried over, entries it will have
  int part;         // rows of its last carried page that it goes on behind, 0: it does not
  bool bad;
};
FAB_DEV RowPlan row_plan(const CacheProblem& p, int64_t b) {
  RowPlan r;
  const int64_t room = p.max_pages * p.page;
  int64_t src = p.source != nullptr ? p.source[b] : b, len = p.lens[b], kept = p.kept[b];
  r.bad = src < -1 || src >= p.B || len < 0 || len > room || kept < 0 || kept > room;
  if (src >= p.B || src < 0) src = -1;
  len = len < 0 ? 0 : len > room ? room : len;
  kept = src < 0 || kept < 0 ? 0 : kept > len ? len : kept;
  r.source = src;
  r.first = (int)((kept + p.page - 1) / p.page);
  r.end = (int)((len + p.page - 1) / p.page);
  r.part = len > kept ? (int)(kept % p.page) : 0;
  return r;
}
FAB_DEV bool page_ok(const CacheProblem& p, int32_t page) { return page >= 0 && page < p.pages; }

constexpr int kReserveThreads = 256;
constexpr int kReserveSlots = 4 * kReserveThreads;  // entries of a row that a CTA looks at

__global__ void __launch_bounds__(kReserveThreads) reserve_release_kernel(const CacheProblem p, const ReserveSpace ws,
                                                                          int chunks) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t b = blockIdx.x / (unsigned)chunks;
  const int64_t s0 = (int64_t)(blockIdx.x % (unsigned)chunks) * kReserveSlots;
  const RowPlan r = row_plan(p, b);
  bool bad = r.bad;
  const int32_t* own = p.table + b * p.max_pages;
  const int32_t* from = p.table + r.source * p.max_pages;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int64_t s = s0 + u * kReserveThreads + (int)threadIdx.x;
    if (s >= p.max_pages) break;
    // (the page that the row goes on writing is dropped here, and settled by `plan`)
    const bool stays = s < r.first && !(r.part > 0 && s == r.first - 1);
    const int32_t had = own[s];
    if (had >= p.pages) bad = true;
    if (r.source == b) {
      if (!stays && page_ok(p, had)) atomicSub(p.refs + had, 1);
      if (s < r.first && !page_ok(p, had)) bad = true;
    } else {
      if (page_ok(p, had)) atomicSub(p.refs + had, 1);
      if (s < r.first) {
        const int32_t page = from[s];
        ws.carried[b * p.max_pages + s] = page_ok(p, page) ? page : -1;
        if (!page_ok(p, page))
          bad = true;
        else if (stays)
          atomicAdd(p.refs + page, 1);
      }
    }
  }
  if (bad) atomicOr(&g_err_pages, kErrIndex);
}

constexpr int kPlanThreads = 1024;

// Sum over the block of one value a thread, and what the threads before this one
// add up to.
FAB_DEV int64_t block_scan(int64_t v, int64_t* before, int64_t* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int64_t base = 0, all = 0;
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) base += sums[w];
    all += sums[w];
  }
  *before = base + incl - v;
  return all;
}

__global__ void __launch_bounds__(kPlanThreads) reserve_plan_kernel(const CacheProblem p, const ReserveSpace ws) {
  __shared__ int64_t sums[kPlanThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // the page that row b goes on writing, or -1
  auto wanted = [&](const RowPlan& r) -> int32_t {
    if (r.part == 0) return -1;
    const int32_t page = p.table[r.source * p.max_pages + r.first - 1];
    return page_ok(p, page) ? page : -1;
  };
  // Of the rows that would go on writing a page which no other row holds (its
  // references have all been dropped) the first keeps it.
  for (int64_t b = threadIdx.x; b < p.B; b += kPlanThreads) {
    const int32_t page = wanted(row_plan(p, b));
    if (page >= 0 && __ldcg(p.refs + page) <= 0) atomicMin(p.refs + page, INT_MIN + (int)b);
  }
  __syncthreads();
  int64_t need = 0, copies = 0;  // of the rows before
  for (int64_t b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    const int64_t b = b0 + threadIdx.x;
    RowPlan r{-1, 0, 0, 0, false};
    int32_t page = -1;
    bool keeps = false;
    if (b < p.B) {
      r = row_plan(p, b);
      page = wanted(r);
      keeps = page >= 0 && __ldcg(p.refs + page) == INT_MIN + (int)b;
    }
    // (a row whose page is not there gets a fresh one, and nothing is copied)
    const int first = r.first - (r.part > 0 && !keeps ? 1 : 0);
    const bool copy = page >= 0 && !keeps;
    int64_t before, at;
    const int64_t all = block_scan(r.end - first, &before, sums);
    const int64_t many = block_scan(copy ? 1 : 0, &at, sums);
    if (b < p.B) ws.rows[b] = ReserveRow{first, (int)(need + before)};
    if (copy) ws.copies[copies + at] = ReserveCopy{page, r.part, (int)(need + before), 0};
    need += all;
    copies += many;
  }
  __syncthreads();
  for (int64_t b = threadIdx.x; b < p.B; b += kPlanThreads) {
    const int32_t page = wanted(row_plan(p, b));
    if (page >= 0 && __ldcg(p.refs + page) == INT_MIN + (int)b) __stcg(p.refs + page, 1);
  }
  __syncthreads();
  // the free pages, in order
  int64_t free = 0;
  bool bad = false;
  for (int64_t x0 = 0; x0 < p.pages; x0 += 4 * kPlanThreads) {
    const int64_t x = x0 + threadIdx.x * 4;
    uint32_t is = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int32_t held = x + u < p.pages ? __ldcg(p.refs + x + u) : 1;
      if (held == 0) is |= 1u << u;
      bad |= held < 0;  // (more entries named it than its references say)
    }
    int64_t before;
    const int64_t all = block_scan(__popc(is), &before, sums);
    int64_t at = free + before;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (is >> u & 1u) ws.free_pages[at++] = (int32_t)(x + u);
    free += all;
  }
  if (bad) atomicOr(&g_err_pages, kErrIndex);
  if (threadIdx.x == 0) {
    ws.counts[0] = (int32_t)free;
    ws.counts[1] = (int32_t)copies;
    const int64_t left = free - need;
    *p.spare = (int32_t)(left < INT_MIN ? INT_MIN : left);
  }
}

// Blocks below `table_blocks` write the table, the others copy.
template <typename V>
__global__ void __launch_bounds__(kReserveThreads) reserve_fill_kernel(const CacheProblem p, const ReserveSpace ws,
                                                                       int chunks, int64_t table_blocks, int kv, int vv) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int32_t free = ws.counts[0];
  if (blockIdx.x < table_blocks) {
    const int64_t b = blockIdx.x / (unsigned)chunks;
    const int64_t s0 = (int64_t)(blockIdx.x % (unsigned)chunks) * kReserveSlots;
    const RowPlan r = row_plan(p, b);
    const ReserveRow x = ws.rows[b];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t s = s0 + u * kReserveThreads + (int)threadIdx.x;
      if (s >= p.max_pages) break;
      int32_t* entry = p.table + b * p.max_pages + s;
      if (s < x.first) {
        if (r.source != b) *entry = ws.carried[b * p.max_pages + s];
      } else if (s < r.end) {
        const int64_t rank = (int64_t)x.rank + (s - x.first);
        const int32_t page = rank < free ? ws.free_pages[rank] : -1;
        *entry = page;
        if (page >= 0) p.refs[page] = 1;
      } else {
        *entry = -1;
      }
    }
    return;
  }
  // units: (copy, layer, keys or values, head), a warp each
  const int lane = threadIdx.x & 31;
  const int64_t per = p.layers * 2 * p.Hkv, units = ws.counts[1] * per;
  const int64_t warps = (int64_t)(gridDim.x - table_blocks) * (kReserveThreads / 32);
  for (int64_t x = (int64_t)(blockIdx.x - table_blocks) * (kReserveThreads / 32) + (threadIdx.x >> 5); x < units;
       x += warps) {
    const int64_t c = x / per;
    int64_t y = x - c * per;
    const int64_t layer = y / (2 * p.Hkv);
    y -= layer * 2 * p.Hkv;
    const bool values = y >= p.Hkv;
    const int64_t head = values ? y - p.Hkv : y;
    const ReserveCopy copy = ws.copies[c];
    if (copy.rank >= free) continue;
    const int nv = values ? vv : kv;
    const int64_t ld = (values ? p.ldv : p.ldk) / (int64_t)((values ? p.DV : p.DK) / nv);
    V* const base = static_cast<V*>(values ? p.v : p.k) + layer * ld;
    const V* src = base + ((int64_t)copy.from * p.Hkv + head) * p.page * nv;
    V* dst = base + ((int64_t)ws.free_pages[copy.rank] * p.Hkv + head) * p.page * nv;
    const int64_t count = (int64_t)copy.rows * nv;
    constexpr int U = 8;
    for (int64_t i0 = lane; i0 < count; i0 += 32 * U) {
      V v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u * 32 < count) v[u] = src[i0 + u * 32];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u * 32 < count) dst[i0 + u * 32] = v[u];
    }
  }
}

// Bytes of the pieces in which rows of a cache are moved: 16 where every row
// of every layer starts at 16 bytes, else an element.
int piece_bytes(const CacheProblem& p, int64_t e) {
  const bool whole = p.DK * e % 16 == 0 && p.DV * e % 16 == 0 && p.ldk * e % 16 == 0 && p.ldv * e % 16 == 0;
  return whole ? 16 : (int)e;
}

}  // namespace

cudaError_t launch_draft_tree(const int32_t* starts, const int32_t* parents, int64_t B, int64_t T, int64_t words,
                              uint32_t* seen, cudaStream_t s) {
  // CTAs of a sequence: about two an SM in all, at most one for each block of 32 tokens
  int64_t per = (304 + B - 1) / B;
  if (per > words) per = words;
  const size_t smem = (size_t)words * 32 * sizeof(int2);
  cudaError_t err = cudaFuncSetAttribute(draft_tree_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         FAB_DRAFT_MAX_WORDS * 32 * (int)sizeof(int2));
  if (err != cudaSuccess) return err;
  return launch_early(draft_tree_kernel, dim3((unsigned)B, (unsigned)per), kTreeThreads, smem, s, starts, parents, B, T,
                      (int)words, seen);
}

cudaError_t launch_paged_accept(const CacheProblem& p, cudaStream_t s) {
  const int64_t items = p.layers * p.Hkv;
  // CTAs of a sequence: about eight an SM in all, four items at least to a CTA
  int64_t per = (1216 + p.B - 1) / p.B;
  if (per > (items + 3) / 4) per = (items + 3) / 4;
  if (per > 65535) per = 65535;
  const dim3 grid((unsigned)p.B, (unsigned)per);
  const int64_t e = p.dtype == FAB_F32 ? 4 : 2;
  const int piece = piece_bytes(p, e), kv = (int)(p.DK * e / piece), vv = (int)(p.DV * e / piece);
  if (piece == 16) return launch_early(paged_accept_kernel<uint4>, grid, kMoveThreads, 0, s, p, kv, vv);
  if (piece == 4) return launch_early(paged_accept_kernel<uint32_t>, grid, kMoveThreads, 0, s, p, kv, vv);
  return launch_early(paged_accept_kernel<uint16_t>, grid, kMoveThreads, 0, s, p, kv, vv);
}

size_t paged_reserve_workspace_bytes(const CacheProblem& p) {
  size_t bytes = 0;
  reserve_space(p, &bytes);
  return bytes;
}

cudaError_t launch_paged_reserve(const CacheProblem& p, cudaStream_t s) {
  const ReserveSpace ws = reserve_space(p, nullptr);
  const int chunks = (int)((p.max_pages + kReserveSlots - 1) / kReserveSlots);
  const int64_t table_blocks = p.B * chunks;
  cudaError_t err = launch_early(reserve_release_kernel, dim3((unsigned)table_blocks), kReserveThreads, 0, s, p, ws, chunks);
  if (err != cudaSuccess) return err;
  err = launch_early(reserve_plan_kernel, dim3(1), kPlanThreads, 0, s, p, ws);
  if (err != cudaSuccess) return err;
  const int64_t e = p.dtype == FAB_F32 ? 4 : 2;
  const int piece = piece_bytes(p, e), kv = (int)(p.DK * e / piece), vv = (int)(p.DV * e / piece);
  const int64_t warps = p.B * p.layers * 2 * p.Hkv;  // units of copying, at most
  const int64_t blocks = (warps + kReserveThreads / 32 - 1) / (kReserveThreads / 32);
  const dim3 grid((unsigned)(table_blocks + (blocks < 1216 ? blocks : 1216)));
  if (piece == 16)
    return launch_early(reserve_fill_kernel<uint4>, grid, kReserveThreads, 0, s, p, ws, chunks, table_blocks, kv, vv);
  if (piece == 4)
    return launch_early(reserve_fill_kernel<uint32_t>, grid, kReserveThreads, 0, s, p, ws, chunks, table_blocks, kv, vv);
  return launch_early(reserve_fill_kernel<uint16_t>, grid, kReserveThreads, 0, s, p, ws, chunks, table_blocks, kv, vv);
}

uint32_t take_error_pages() {
  uint32_t v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_pages, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(g_err_pages, &z, sizeof(z));
  return v;
}

}  // namespace fab
