// fab_pages.cu -- drafts and pages of a paged key/value cache: who sees whom
// in a drafted tree, keeping the accepted path's rows, and which sequence
// holds which page (forked, grown, cut, freed, copied before it is written).
#include <limits.h>
#include <stddef.h>

#include <type_traits>

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
// token: a thread walks from block to block and writes words as it goes, eight of a
// row.  Bound by the chain of start, predecessor, exchanges, walk and store: one
// draft of 8 tokens 2.2 us, 256 of 20 to 500 tokens (4.4 MB) 5.0, where the host takes 10 to 12.

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
// is written, by one warp for each item (keys or values, layer, head) of a
// sequence, and nothing is overwritten before it has been read.
//
// How many rows move is known on the device only, and differs: the items of all
// sequences form one line, each as long as its rows, and every warp takes an equal
// piece of it (the items that begin there).  Each CTA lays the line out for itself.
// Bound by that chain (lengths, bits, pages, copy, store: 6.7 us for one layer) and the
// scattered rows: 64 drafts in 32 layers of 8 heads of width 128, 52 MB, 15.6 us, 5.9 TB/s
// behind the chain.  Two CTAs an SM; three took 15.5, and 9.1 for 8.2 us in 8 layers.

constexpr int kMoveThreads = 256;
constexpr int kMoveWarps = kMoveThreads / 32;
constexpr int kMoveCtas = 2;  // CTAs of an SM
constexpr int kMoves = 64;    // rows of a path listed at once
constexpr int kMoveBuffer = 8192;  // bytes of rows that a warp has on their way

// How rows of a cache are moved: in pieces of 16 bytes where every row of every
// layer starts at 16 bytes, else of an element.  Index 0: keys, 1: values.
struct Pieces {
  int row[2];        // pieces of a row
  int64_t layer[2];  // from one layer to the next
  int bytes;
};
Pieces pieces_of(const CacheProblem& p) {
  const int64_t e = p.dtype == FAB_F32 ? 4 : 2;
  const bool whole = p.DK * e % 16 == 0 && p.DV * e % 16 == 0 && p.ldk * e % 16 == 0 && p.ldv * e % 16 == 0;
  Pieces x;
  x.bytes = whole ? 16 : (int)e;
  x.row[0] = (int)(p.DK * e / x.bytes);
  x.row[1] = (int)(p.DV * e / x.bytes);
  x.layer[0] = p.ldk * e / x.bytes;
  x.layer[1] = p.ldv * e / x.bytes;
  return x;
}

// What a sequence keeps.
struct PathPlan {
  int64_t past;        // rows before the new tokens
  const uint32_t* row; // who the path's last token sees, itself included
  int words;           // words of it up to that token's (0: nothing is kept)
  uint32_t last_mask;  // of the last one
  bool bad;
};
FAB_DEV PathPlan path_plan(const CacheProblem& p, int64_t b) {
  const int64_t s0 = p.starts[b], n = (int64_t)p.starts[b + 1] - s0, len = p.lens[b], told = p.last[b];
  const int64_t last = n > 0 ? told : -1;
  PathPlan x;
  x.past = len - n;
  x.bad = s0 < 0 || n < 0 || s0 + n > p.T || x.past < 0 || len > p.max_pages * p.page || last < -1 || last >= n ||
          last >= 32 * p.words;
  x.words = x.bad || last < 0 ? 0 : (int)(last >> 5) + 1;
  x.row = p.seen + (x.words > 0 ? s0 + last : 0) * p.words;
  x.last_mask = (last & 31) == 31 ? 0xffffffffu : (2u << (last & 31)) - 1u;
  return x;
}
FAB_DEV uint32_t path_word(const PathPlan& x, int w) {
  const uint32_t bits = __ldg(x.row + w);
  return w == x.words - 1 ? bits & x.last_mask : bits;
}

// a / b for a >= 0, b > 0 (a 64-bit division is some hundred instructions)
FAB_DEV int64_t ratio(int64_t a, int64_t b) {
  return ((uint64_t)(a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Copies `rows` rows of a cache from src to dst (a lane's own; null: none), one
// warp.  Rows of whole aligned 16-byte pieces go through shared memory by bulk
// copies, a lane a row: 256 B cost a lane two instructions, where copies through
// registers have the whole warp work on two rows (64 drafts in 32 layers, 52 MB: 15.6
// us, through registers 17.0, both with the rows shared out evenly; a CTA a sequence and
// an equal share of the items, through registers, 21.7).
struct BulkMover {
  uint32_t buf, bar;  // kMoveBuffer bytes, a barrier
  uint32_t phase;
  volatile uint32_t* abort_flag;
  FAB_DEV int most(uint32_t row_bytes) const {
    const int n = kMoveBuffer / (int)row_bytes;
    return n < 32 ? n : 32;
  }
  FAB_DEV bool operator()(const uint8_t* src, uint8_t* dst, uint32_t row_bytes) {
    const uint32_t mine = buf + lane_id() * row_bytes;
    bulk_wait_read_all();  // (the rows before have left the buffer)
    const uint32_t there = (uint32_t)__popc(__ballot_sync(0xffffffffu, src != nullptr));
    if (lane_id() == 0) mbar_arrive_expect_tx(bar, there * row_bytes);
    __syncwarp();
    if (src != nullptr) bulk_load(mine, src, row_bytes, bar);
    if (!__all_sync(0xffffffffu, mbar_wait_asleep(bar, phase, abort_flag, &g_err_pages))) {
      mbar_drain(bar, phase);  // (what is on its way lands before shared memory goes)
      return false;
    }
    phase ^= 1u;
    if (src != nullptr) bulk_store(dst, mine, row_bytes);
    bulk_commit_group();
    return true;
  }
  FAB_DEV void finish() { bulk_wait_all(); }
};
template <typename V>
struct PieceMover {
  FAB_DEV int most(uint32_t) const { return 32; }
  FAB_DEV bool operator()(const uint8_t* src, uint8_t* dst, uint32_t row_bytes) {
    const int n = (int)(row_bytes / sizeof(V)), lane = (int)lane_id();
    // four rows at a time, each at most 256 pieces
    for (int r0 = 0; r0 < 32; r0 += 4) {
      V v[4][8];
      uint64_t to[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const V* from = reinterpret_cast<const V*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(src), r0 + r));
        to[r] = from != nullptr ? __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(dst), r0 + r) : 0;
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (from != nullptr && u * 32 + lane < n) v[r][u] = from[u * 32 + lane];
      }
      __syncwarp();
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (to[r] != 0 && u * 32 + lane < n) reinterpret_cast<V*>(to[r])[u * 32 + lane] = v[r][u];
      __syncwarp();
    }
    return true;
  }
  FAB_DEV void finish() {}
};

// V: uint4 (bulk copies) or an element.
template <typename V>
__global__ void __launch_bounds__(kMoveThreads, kMoveCtas) paged_accept_kernel(const CacheProblem p, const Pieces pc) {
  constexpr bool kBulk = sizeof(V) == 16;
  extern __shared__ __align__(128) uint8_t buf_s[];
  __shared__ int64_t from_s[kMoveWarps][kMoves], to_s[kMoveWarps][kMoves];  // rows, as if of head 0
  __shared__ int64_t ends_s[kMoveThreads];  // rows that move, of the sequences up to this one
  __shared__ int64_t sums_s[kMoveWarps];
  __shared__ uint64_t bars[kMoveWarps];
  __shared__ uint32_t abort_s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) abort_s = 0u;
  typename std::conditional<kBulk, BulkMover, PieceMover<V>>::type mover;
  if constexpr (kBulk) {
    if (lane == 0) mbar_init(smem_u32(&bars[warp]), 1);
    fence_mbar_init();
    mover = BulkMover{smem_u32(buf_s) + warp * kMoveBuffer, smem_u32(&bars[warp]), 0u, &abort_s};
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0) check_starts(p.starts, p.B, p.T, (int)threadIdx.x, kMoveThreads, &g_err_pages);
  const int64_t items = p.layers * p.Hkv;  // of keys, and as many of values

  // ends_s of the sequences from b0 on; returns how many rows of theirs move
  auto lay_out = [&](int64_t b0, bool tell) -> int64_t {
    const int64_t b = b0 + threadIdx.x;
    int64_t moves = 0;
    if (b < p.B) {
      const PathPlan x = path_plan(p, b);
      int64_t count = 0, stay = 0;  // rows of the path, those of them that are in place
      for (int w = 0; w < x.words; ++w) {
        const uint32_t bits = path_word(x, w);
        if (stay == w * 32) stay += bits == 0xffffffffu ? 32 : __ffs((int)~bits) - 1;
        count += __popc(bits);
      }
      moves = count - stay;
      if (tell) {
        if (x.bad) atomicOr(&g_err_pages, kErrIndex);
        p.lens_out[b] = x.bad ? p.lens[b] : (int32_t)(x.past + count);
      }
    }
    int64_t incl = moves;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    __syncthreads();
    if (lane == 31) sums_s[warp] = incl;
    __syncthreads();
    int64_t base = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kMoveWarps; ++w) {
      if (w < warp) base += sums_s[w];
      all += sums_s[w];
    }
    ends_s[threadIdx.x] = base + incl;
    __syncthreads();
    return all;
  };
  int64_t total = 0;
  for (int64_t b0 = 0; b0 < p.B; b0 += kMoveThreads) total += lay_out(b0, blockIdx.x == 0);

  // this warp's piece of the line
  const int64_t line = total * 2 * items, all_warps = (int64_t)gridDim.x * kMoveWarps;
  const int64_t me = (int64_t)blockIdx.x * kMoveWarps + warp;
  const int64_t q = ratio(line, all_warps), r = line - q * all_warps;
  const int64_t p0 = q * me + ratio(r * me, all_warps), p1 = q * (me + 1) + ratio(r * (me + 1), all_warps);

  // sequence b's items (keys', then values') whose place on the line (from a on, `moves` each) is in the piece
  auto work = [&](int64_t b, int64_t a, int64_t moves) -> bool {
    const int64_t x0 = p0 <= a ? 0 : ratio(p0 - a + moves - 1, moves), x1 = p1 <= a ? 0 : ratio(p1 - a + moves - 1, moves);
    const int64_t i0 = x0, i1 = x1 < 2 * items ? x1 : 2 * items;
    if (i0 >= i1) return true;
    const PathPlan x = path_plan(p, b);
    const int32_t* table = p.table + b * p.max_pages;
    int64_t taken = 0;  // rows of the path before the list
    for (int word = 0; word < x.words;) {
      int count = 0;
      for (; word < x.words && count <= kMoves - 32; ++word) {
        const uint32_t bits = path_word(x, word);
        const int64_t to = x.past + taken + __popc(bits & ((1u << lane) - 1u)), from = x.past + word * 32 + lane;
        const bool moves_now = (bits >> lane & 1u) && to != from;
        const uint32_t moving = __ballot_sync(0xffffffffu, moves_now);
        if (moves_now) {
          const uint32_t page = (uint32_t)p.page, pa = (uint32_t)from / page, pz = (uint32_t)to / page;
          const int32_t ta = table[pa], tz = table[pz];
          const int at = count + __popc(moving & ((1u << lane) - 1u));
          const bool ok = ta >= 0 && ta < p.pages && tz >= 0 && tz < p.pages;
          if (!ok) atomicOr(&g_err_pages, kErrIndex);  // (the row stays where it is)
          from_s[warp][at] = ok ? (int64_t)ta * p.Hkv * p.page + ((uint32_t)from - pa * page) : -1;
          to_s[warp][at] = ok ? (int64_t)tz * p.Hkv * p.page + ((uint32_t)to - pz * page) : -1;
        }
        count += __popc(moving);
        taken += __popc(bits);
      }
      __syncwarp();
      for (int kind = 0; kind < 2; ++kind) {
        const int64_t k0 = i0 - kind * items > 0 ? i0 - kind * items : 0, k = i1 - kind * items, k1 = k < items ? k : items;
        if (k0 >= k1 || count == 0) continue;
        const uint32_t rb = (uint32_t)pc.row[kind] * sizeof(V), rows = (uint32_t)(k1 - k0) * count;
        uint8_t* const base = static_cast<uint8_t*>(kind ? p.v : p.k);
        const uint32_t step = (uint32_t)mover.most(rb);
        // a lane a row, in order of (item, move)
        for (uint32_t r0 = 0; r0 < rows; r0 += step) {
          const uint32_t y = r0 + lane;
          const uint8_t* src = nullptr;
          uint8_t* dst = nullptr;
          if (lane < (int)step && y < rows) {
            const uint32_t it = y / (uint32_t)count, mv = y - it * count, item = (uint32_t)k0 + it;
            const uint32_t layer = item / (uint32_t)p.Hkv, head = item - layer * (uint32_t)p.Hkv;
            uint8_t* const at = base + (layer * pc.layer[kind] * (int64_t)sizeof(V) + (int64_t)head * p.page * rb);
            const int64_t from = from_s[warp][mv];
            if (from >= 0) {
              src = at + from * rb;
              dst = at + to_s[warp][mv] * rb;
            }
          }
          if (!mover(src, dst, rb)) return false;
        }
      }
      __syncwarp();
    }
    return true;
  };
  int64_t before = 0;  // rows of the sequences before ends_s
  bool ok = true;
  for (int64_t b0 = 0; b0 < p.B; b0 += kMoveThreads) {
    const int64_t here = p.B > kMoveThreads ? lay_out(b0, false) : total;
    if (ok && p0 < p1 && p0 < (before + here) * 2 * items && p1 > before * 2 * items) {
      // the first sequence that reaches into the piece, and on from there
      int lo = 0, hi = kMoveThreads - 1;
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if ((before + ends_s[mid]) * 2 * items > p0) hi = mid; else lo = mid + 1;
      }
      for (int i = lo; ok && i < kMoveThreads && b0 + i < p.B; ++i) {
        const int64_t first = i > 0 ? ends_s[i - 1] : 0, moves = ends_s[i] - first;
        if ((before + first) * 2 * items >= p1) break;
        if (moves > 0) ok = work(b0 + i, (before + first) * 2 * items, moves);
      }
    }
    before += here;
  }
  mover.finish();
}

// ------------------------------------------------------------------ pages
//
// Two kernels.  `plan`, one cluster of CTAs, drops and adds references as rows
// lose and gain entries, settles who keeps a page that several rows would go on
// writing, finds the free pages and hands them out in order of (row, entry): steps
// that each need all of the one before, with the cluster's barrier between them.
// Each CTA has a share of the rows and a share of the pages.  `copy` copies what has
// to be copied.  Planning is bound by the five steps, each two or three accesses long, and
// the barriers: 256 rows over a pool of 131,072 pages 18.9 us with the copy's empty
// launch, 16 rows of a small pool 11 (as three kernels, the plan's a single CTA, 87 and more).

struct ReserveCopy {
  int from, rows;  // page, rows of it
  int rank;        // the fresh page's place
  int pad;
};
struct ReserveRow {
  int first;  // the first entry that gets a fresh page
  int rank;   // its place among all fresh ones
  int kept;   // the page that it goes on writing and keeps, or -1
  int pad;
};
static_assert(sizeof(ReserveRow) == 16, "read as one piece");
constexpr int kPlanCtas = 8;  // the largest cluster that every GPU runs
constexpr int kPlanThreads = 1024;
// What the shares of a CTA come to.
struct PlanTotals {
  int64_t need;     // fresh pages of its rows
  int copies;       // and copies (written in one with the next)
  uint32_t misfit;  // references without entries or the reverse, weighted
  int64_t free;     // free ones of its pages
};
struct ReserveSpace {
  int32_t* carried;     // [B][max_pages], of rows that continue another one
  int32_t* free_pages;  // the free ones, lowest first
  ReserveRow* rows;     // [B]
  ReserveCopy* copies;  // [B]
  int64_t* counts;      // free pages, copies
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
  x.counts = reinterpret_cast<int64_t*>(take(2 * sizeof(int64_t)));
  x.free_pages = reinterpret_cast<int32_t*>(take((size_t)p.pages * sizeof(int32_t)));
  x.carried = reinterpret_cast<int32_t*>(take((size_t)(p.B * p.max_pages) * sizeof(int32_t)));
  if (bytes) *bytes = at;
  return x;
}

// What a row's numbers say.
struct RowPlan {
  int source;       // the row it continues, -1: none
  int first, end;   // entries carried over, entries it will have
  int part;         // rows of its last carried page that it goes on behind, 0: it does not
};
FAB_DEV RowPlan row_plan(const CacheProblem& p, int64_t b, bool* bad) {
  const int64_t room = p.max_pages * p.page;
  int64_t src = p.source != nullptr ? p.source[b] : b, len = p.lens[b], kept = p.kept[b];
  *bad |= src < -1 || src >= p.B || len < 0 || len > room || kept < 0 || kept > room;
  if (src >= p.B || src < 0) src = -1;
  len = len < 0 ? 0 : len > room ? room : len;
  kept = src < 0 || kept < 0 ? 0 : kept > len ? len : kept;
  RowPlan r;
  r.source = (int)src;
  const uint32_t page = (uint32_t)p.page, k = (uint32_t)kept, n = (uint32_t)len;  // (below 2^31, all three)
  r.first = (int)((k + page - 1) / page);
  r.end = (int)((n + page - 1) / page);
  r.part = len > kept ? (int)(k % page) : 0;
  return r;
}
FAB_DEV bool page_ok(const CacheProblem& p, int32_t page) { return page >= 0 && page < p.pages; }

// A page's weight in the sums that show whether references fit the table: odd, so that one
// page's misfit always shows, and otherwise spread over 32 bits, so that those of several cancel
// by chance alone, once in 2^32.  (The bits of the golden ratio and of the root of 2.)
FAB_DEV uint32_t weight(uint32_t page) {
  const uint32_t x = page * 0x9E3779B9u;
  return ((x ^ x >> 15) * 0x6A09E667u) | 1u;
}

// Sum over the block of one value a thread, and what the threads before this one
// add up to.
FAB_DEV int block_scan(int v, int* before, int* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int of_warps = sums[lane];  // (32 warps: each sums them up by itself)
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, of_warps, o);
    if (lane >= o) of_warps += up;
  }
  const int base = __shfl_sync(0xffffffffu, of_warps, warp > 0 ? warp - 1 : 0);
  *before = (warp > 0 ? base : 0) + incl - v;
  return __shfl_sync(0xffffffffu, of_warps, 31);
}

// The sum alone.
FAB_DEV int block_sum(int v, int* sums) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, sums[threadIdx.x & 31]);
}

// The sums of two.
FAB_DEV int2 block_sums(int v, int w, int2* sums) {
  const int2 of_warp = make_int2(__reduce_add_sync(0xffffffffu, v), __reduce_add_sync(0xffffffffu, w));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = of_warp;
  __syncthreads();
  const int2 x = sums[threadIdx.x & 31];
  return make_int2(__reduce_add_sync(0xffffffffu, x.x), __reduce_add_sync(0xffffffffu, x.y));
}

constexpr int kPlanRows = 1024;        // rows of a CTA's share held in shared memory at once
constexpr int kPlanSlots = 128;        // entries that a warp looks at
constexpr int kPlanPages = 16 * kPlanThreads;  // pages that a CTA looks at at once

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads)
    reserve_plan_kernel(const CacheProblem p, const ReserveSpace ws) {
  static_assert(kPlanThreads == 1024, "block_scan is for 32 warps");
  __shared__ RowPlan rows_s[kPlanRows];
  __shared__ PlanTotals totals_s[kPlanCtas];
  __shared__ int sums[32];
  __shared__ int2 sums2[32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cta = (int)blockIdx.x;
  const int64_t b0 = p.B * cta / kPlanCtas, b1 = p.B * (cta + 1) / kPlanCtas;
  const int segs = (int)((p.max_pages + kPlanSlots - 1) / kPlanSlots);  // of a row, a warp each
  bool bad = false;
  int held = -1;  // rows_s holds this part of the share
  // calls f(count of rows in rows_s, the first of them) for each part of the share
  auto each_part = [&](auto f) {
    int part = 0;
    for (int64_t r0 = b0; r0 < b1; r0 += kPlanRows, ++part) {
      const int n = (int)(b1 - r0 < kPlanRows ? b1 - r0 : kPlanRows);
      if (held != part) {
        __syncthreads();
        if ((int)threadIdx.x < n) rows_s[threadIdx.x] = row_plan(p, r0 + threadIdx.x, &bad);
        __syncthreads();
        held = part;
      }
      f(n, r0);
    }
  };
  // What a thread knows of its row (of a share of more rows than threads: of the last part).
  int32_t page = -1;   // the page that the row goes on writing, -1: none
  bool own = false;    // and keeps
  // the same for a row of another part
  auto wanted = [&](const RowPlan& r) -> int32_t {
    if (r.part == 0) return -1;
    const int32_t x = p.table[(int64_t)r.source * p.max_pages + r.first - 1];
    return page_ok(p, x) ? x : -1;
  };
  auto keeps = [&](int32_t x, int64_t b) { return x >= 0 && __ldcg(p.refs + x) == INT_MIN + (int)b; };
  const bool parts = b1 - b0 > kPlanRows;
  // The references that step 1 leaves, less the entries that hold on to their page, both
  // weighted by page: 0 where they fit.
  uint32_t misfit = 0;
  // 1. Entries that go and come.  (A page that a row goes on writing is dropped.)
  each_part([&](int n, int64_t r0) {
    if ((int)threadIdx.x < n) page = wanted(rows_s[threadIdx.x]);
    for (int x = warp; x < n * segs; x += kPlanThreads / 32) {
      const int i = x / segs;
      const int64_t b = r0 + i;
      const RowPlan r = rows_s[i];
      const int32_t* row = p.table + b * p.max_pages;
      const int32_t* from = p.table + (int64_t)(r.source < 0 ? 0 : r.source) * p.max_pages;
      const int64_t s0 = (int64_t)(x - i * segs) * kPlanSlots + lane;
      int32_t had[4], get[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t s = s0 + u * 32;
        had[u] = s < p.max_pages ? row[s] : -1;
        get[u] = r.source != b && s < r.first ? from[s] : -1;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t s = s0 + u * 32;
        const bool carried = s < r.first, stays = carried && !(r.part > 0 && s == r.first - 1);
        if (had[u] >= p.pages) bad = true;
        if (r.source == b) {
          if (!stays && page_ok(p, had[u])) atomicSub(p.refs + had[u], 1);
          if (stays && page_ok(p, had[u])) misfit -= weight((uint32_t)had[u]);
          if (carried && had[u] < 0) bad = true;
        } else {
          if (page_ok(p, had[u])) atomicSub(p.refs + had[u], 1);
          if (carried) {
            const bool ok = page_ok(p, get[u]);
            ws.carried[b * p.max_pages + s] = ok ? get[u] : -1;
            if (!ok)
              bad = true;
            else if (stays)
              atomicAdd(p.refs + get[u], 1), misfit -= weight((uint32_t)get[u]);
          }
        }
      }
    }
  });
  cluster_sync();
  // 2. Of the rows that would go on writing a page which no other row holds (its
  // references have all been dropped) the first keeps it: the lowest mark stays.
  // (a count below zero that is no mark: more entries named the page than its references say)
  auto odd = [](int32_t c) { return c < 0 && c > INT_MIN / 2; };
  each_part([&](int n, int64_t r0) {
    if ((int)threadIdx.x < n) {
      if (parts) page = wanted(rows_s[threadIdx.x]);
      const int32_t count = page >= 0 ? __ldcg(p.refs + page) : 1;
      if (count <= 0) atomicMin(p.refs + page, INT_MIN + (int)(r0 + threadIdx.x));
      bad |= odd(count);  // (the first to leave its mark sees what was there before)
    }
  });
  cluster_sync();
  // 3. How many pages of the CTA's share are free, the fresh pages and copies of its rows.
  const int64_t g0 = (p.pages + 3) / 4 * cta / kPlanCtas * 4;
  const int64_t g = (p.pages + 3) / 4 * (cta + 1) / kPlanCtas * 4, g1 = g < p.pages ? g : p.pages;
  // Of the 512 pages from x on that a warp looks at, 128 at a time: bit 4 k + u of
  // this lane's says that page x + 128 k + 4 lane + u is free.
  auto look = [&](int64_t x) -> uint32_t {
    int4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t at = x + k * 128 + lane * 4;
      v[k] = make_int4(INT_MIN, INT_MIN, INT_MIN, INT_MIN);  // (as if kept: no page there)
      if (at + 4 <= g1) {
        v[k] = __ldcg(reinterpret_cast<const int4*>(p.refs + at));
      } else {
        if (at < g1) v[k].x = __ldcg(p.refs + at);
        if (at + 1 < g1) v[k].y = __ldcg(p.refs + at + 1);
        if (at + 2 < g1) v[k].z = __ldcg(p.refs + at + 2);
      }
    }
    uint32_t bits = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int32_t c[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (odd(c[u])) bad = true;
        misfit += (uint32_t)max(c[u], 0) * weight((uint32_t)x + k * 128 + lane * 4 + u);
      }
      bits |= ((v[k].x == 0 ? 1u : 0u) | (v[k].y == 0 ? 2u : 0u) | (v[k].z == 0 ? 4u : 0u) | (v[k].w == 0 ? 8u : 0u))
              << (4 * k);
    }
    return bits;
  };
  // a row's fresh entries; a row whose page is not there gets a fresh one, and nothing is copied
  auto fresh_of = [&](const RowPlan& r) { return r.end - r.first + (r.part > 0 && !own ? 1 : 0); };
  int64_t need = 0, copies = 0;
  uint32_t mine = look(g0 + warp * 512);  // the last part's bits of this thread
  each_part([&](int n, int64_t r0) {
    int fresh = 0;
    if ((int)threadIdx.x < n) {
      if (parts) page = wanted(rows_s[threadIdx.x]);
      own = keeps(page, r0 + threadIdx.x);
      fresh = fresh_of(rows_s[threadIdx.x]);
    }
    need += block_sum(fresh, sums);
    copies += __syncthreads_count((int)threadIdx.x < n && page >= 0 && !own);  // (of this part's rows alone)
  });
  int unused = __popc(mine);  // pages (of a thread, below 2^31 / 1024)
  for (int64_t x0 = g0 + kPlanPages; x0 < g1; x0 += kPlanPages) {
    mine = look(x0 + warp * 512);
    unused += __popc(mine);
  }
  const int2 of_pages = block_sums(unused, (int)misfit, sums2);
  if (threadIdx.x < kPlanCtas) {  // to every CTA of the cluster
    const uint32_t to = cluster_addr(smem_u32(totals_s + cta), threadIdx.x);
    st_cluster(to + offsetof(PlanTotals, need), need);
    st_cluster(to + offsetof(PlanTotals, copies), (int64_t)(uint32_t)of_pages.y << 32 | copies);
    st_cluster(to + offsetof(PlanTotals, free), of_pages.x);
  }
  cluster_sync();
  // 4. Ranks of the rows, the list of the free pages.
  int64_t need0 = 0, copies0 = 0, free0 = 0, all_need = 0, all_copies = 0, all_free = 0;
  uint32_t unfit = 0;
#pragma unroll
  for (int c = 0; c < kPlanCtas; ++c) {
    const PlanTotals t = totals_s[c];
    if (c < cta) need0 += t.need, copies0 += t.copies, free0 += t.free;
    all_need += t.need, all_copies += t.copies, all_free += t.free;
    unfit += t.misfit;
  }
  // What a row holds on to has a reference left, or the counts were too low: the page
  // would be handed out, or another row would write it.  Looked for only where the sums say
  // that something does not fit (256 rows: the look at each entry's count 4.2 us, the sums 0.9).
  if (unfit != 0u)
    each_part([&](int n, int64_t r0) {
      for (int x = warp; x < n * segs; x += kPlanThreads / 32) {
        const int i = x / segs;
        const RowPlan r = rows_s[i];
        const int stay = r.first - (r.part > 0 ? 1 : 0);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int s = (x - i * segs) * kPlanSlots + u * 32 + lane;
          if (s >= stay) break;
          const int32_t held = p.table[(int64_t)r.source * p.max_pages + s];  // (a row of no source holds nothing)
          if (page_ok(p, held) && __ldcg(p.refs + held) <= 0) bad = true;
        }
      }
    });
  each_part([&](int n, int64_t r0) {
    int fresh = 0;
    RowPlan r{-1, 0, 0, 0};
    if ((int)threadIdx.x < n) {
      r = rows_s[threadIdx.x];
      if (parts) {
        page = wanted(r);
        own = keeps(page, r0 + threadIdx.x);
      }
      fresh = fresh_of(r);
    }
    const bool copy = (int)threadIdx.x < n && page >= 0 && !own;
    int before, at;
    const int all = block_scan(fresh, &before, sums), many = block_scan(copy ? 1 : 0, &at, sums);
    if ((int)threadIdx.x < n)
      ws.rows[r0 + threadIdx.x] = ReserveRow{r.end - fresh, (int)(need0 + before), own ? page : -1, 0};
    if (copy) ws.copies[copies0 + at] = ReserveCopy{page, r.part, (int)(need0 + before), 0};
    need0 += all;
    copies0 += many;
  });
  const bool again = g1 - g0 > kPlanPages;  // (the bits of more than one part are looked at again)
  for (int64_t x0 = g0; x0 < g1 && free0 < all_need; x0 += kPlanPages) {
    if (again) mine = look(x0 + warp * 512);
    // in order of page: the warp's four pieces of 128, in each the lanes in turn
    int before;
    const int of_part = block_scan(__popc(mine), &before, sums);
    int64_t at = free0 + __shfl_sync(0xffffffffu, before, 0);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t bits = mine >> (4 * k) & 15u;
      int ahead = 0, of_piece = 0;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t m = __ballot_sync(0xffffffffu, bits >> u & 1u);
        ahead += __popc(m & ((1u << lane) - 1u));
        of_piece += __popc(m);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (bits >> u & 1u) {
          if (at + ahead < all_need) ws.free_pages[at + ahead] = (int32_t)(x0 + warp * 512 + k * 128 + lane * 4 + u);
          ++ahead;
        }
      at += of_piece;
    }
    free0 += of_part;
  }
  if (cta == 0 && threadIdx.x == 0) {
    ws.counts[0] = all_free;
    ws.counts[1] = all_copies;
    const int64_t left = all_free - all_need;
    *p.spare = (int32_t)(left < INT_MIN ? INT_MIN : left);
  }
  cluster_sync();
  // 5. The table, and the references of what was handed out and kept.
  each_part([&](int n, int64_t r0) {
    for (int x = warp; x < n * segs; x += kPlanThreads / 32) {
      const int i = x / segs;
      const int64_t b = r0 + i;
      const RowPlan r = rows_s[i];
      const int4 y = __ldcg(reinterpret_cast<const int4*>(ws.rows + b));
      const int64_t s0 = (int64_t)(x - i * segs) * kPlanSlots + lane;
      if (s0 == 0 && y.z >= 0) p.refs[y.z] = 1;
      int32_t* row = p.table + b * p.max_pages;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t s = s0 + u * 32;
        if (s >= p.max_pages) break;
        if (s < y.x) {
          if (r.source != b) row[s] = __ldcg(ws.carried + b * p.max_pages + s);
        } else if (s < r.end) {
          const int64_t rank = (int64_t)y.y + (s - y.x);
          const int32_t given = rank < all_free ? __ldcg(ws.free_pages + rank) : -1;
          row[s] = given;
          if (given >= 0) p.refs[given] = 1;
        } else {
          row[s] = -1;
        }
      }
    }
  });
  if (bad) atomicOr(&g_err_pages, kErrIndex);
}

constexpr int kCopyThreads = 256;

// Units: (copy, layer, keys or values, head), a warp each.  Bound by HBM: 16 prompts
// forked into 8 beams, 32 layers of 8 heads of width 128 (411 MB written, 59 MB read
// once and then from the L2, for which the copies give way: 100 -> 96 us): 90 us, 75
// of them the copy's, 6.3 TB/s.  Rings of bulk copies in place of the registers took 100 to 109.
template <typename V>
__global__ void __launch_bounds__(kCopyThreads) reserve_copy_kernel(const CacheProblem p, const ReserveSpace ws,
                                                                    const Pieces pc) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t free = ws.counts[0];
  const int lane = threadIdx.x & 31;
  const int64_t per = p.layers * 2 * p.Hkv, units = ws.counts[1] * per;
  const int64_t warps = (int64_t)gridDim.x * (kCopyThreads / 32);
  for (int64_t x = (int64_t)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); x < units; x += warps) {
    const int64_t c = ratio(x, per);
    const int y = (int)(x - c * per), hkv = (int)p.Hkv, layer = y / (2 * hkv), z = y - layer * 2 * hkv;
    const int kind = z >= hkv ? 1 : 0, head = z - kind * hkv;
    const ReserveCopy copy = ws.copies[c];
    if (copy.rank >= free) continue;
    const int nv = pc.row[kind];
    V* const base = static_cast<V*>(kind ? p.v : p.k) + layer * pc.layer[kind];
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
        if (i0 + u * 32 < count) __stcs(dst + i0 + u * 32, v[u]);
    }
  }
}

}  // namespace

cudaError_t launch_draft_tree(const int32_t* starts, const int32_t* parents, int64_t B, int64_t T, int64_t words,
                              uint32_t* seen, cudaStream_t s) {
  // CTAs of a sequence: about two an SM in all, at most one for each block of 32 tokens
  int64_t per = (304 + B - 1) / B;
  if (per > words) per = words;
  const size_t smem = (size_t)words * 32 * sizeof(int2);
  if (smem > 48 * 1024) {  // (what a kernel has without asking)
    const cudaError_t err = cudaFuncSetAttribute(draft_tree_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 FAB_DRAFT_MAX_WORDS * 32 * (int)sizeof(int2));
    if (err != cudaSuccess) return err;
  }
  return launch_early(draft_tree_kernel, dim3((unsigned)B, (unsigned)per), kTreeThreads, smem, s, starts, parents, B, T,
                      (int)words, seen);
}

cudaError_t launch_paged_accept(const CacheProblem& p, cudaStream_t s) {
  // as many CTAs as run at once, at most one for every eight items
  const int64_t items = p.B * 2 * p.layers * p.Hkv, most = kMoveCtas * 152;
  const int64_t ctas = (items + kMoveWarps - 1) / kMoveWarps;
  const dim3 grid((unsigned)(ctas < most ? ctas : most));
  const Pieces pc = pieces_of(p);
  if (pc.bytes == 16) {
    constexpr int smem = kMoveWarps * kMoveBuffer;
    const cudaError_t err =
        cudaFuncSetAttribute(paged_accept_kernel<uint4>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    return launch_early(paged_accept_kernel<uint4>, grid, kMoveThreads, smem, s, p, pc);
  }
  if (pc.bytes == 4) return launch_early(paged_accept_kernel<uint32_t>, grid, kMoveThreads, 0, s, p, pc);
  return launch_early(paged_accept_kernel<uint16_t>, grid, kMoveThreads, 0, s, p, pc);
}

size_t paged_reserve_workspace_bytes(const CacheProblem& p) {
  size_t bytes = 0;
  reserve_space(p, &bytes);
  return bytes;
}

cudaError_t launch_paged_reserve(const CacheProblem& p, cudaStream_t s) {
  const ReserveSpace ws = reserve_space(p, nullptr);
  const cudaError_t err = launch_early(reserve_plan_kernel, dim3(kPlanCtas), kPlanThreads, 0, s, p, ws);
  if (err != cudaSuccess) return err;
  const Pieces pc = pieces_of(p);
  const int64_t warps = p.B * p.layers * 2 * p.Hkv;  // units of copying, at most
  const int64_t blocks = (warps + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
  // Blocks of the copy.  Rows that continue others will copy much (16 prompts forked into 8 beams in 32
  // layers: 89.1 us with 4,864 blocks, 96.2 with 1,216), rows that go on by themselves
  // seldom anything (256 of them, 32 layers: 16.8 and 13.1 us).
  const int64_t most = p.source != nullptr ? 4864 : 1216;
  const dim3 grid((unsigned)(blocks < most ? blocks : most));
  if (pc.bytes == 16) return launch_early(reserve_copy_kernel<uint4>, grid, kCopyThreads, 0, s, p, ws, pc);
  if (pc.bytes == 4) return launch_early(reserve_copy_kernel<uint32_t>, grid, kCopyThreads, 0, s, p, ws, pc);
  return launch_early(reserve_copy_kernel<uint16_t>, grid, kCopyThreads, 0, s, p, ws, pc);
}

uint32_t take_error_pages() {
  uint32_t v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_pages, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(g_err_pages, &z, sizeof(z));
  return v;
}

}  // namespace fab
