// fab_paged_tc.cu -- attention of new tokens over a paged key/value cache, on
// tcgen05: bf16 or f16, DK and DV multiples of 8 up to 128, pages of a
// multiple of 8 rows.
//
//   token i of the n new ones of sequence b, head h:
//   s_m = scale q . k_m over m <= lens[b] - n + i (causal) or m < lens[b],
//   o = sum softmax(s)_m v_m,  lse = log sum exp(s_m)
//
// Tiles.  A row of a tile is a (token, query head) pair of one key/value head:
// 128 / group tokens times the group's heads, so a page of keys is read once
// for the whole group and a single token still fills as many rows as it has
// heads.  Two streams of four softmax warps each own a score tile S_s and an
// output O_s in tensor memory (thread = row, all 128 keys of a tile), and the
// tensor core alternates between them: while one stream's softmax runs, the
// other's products do.  A unit of two row tiles gives each stream a row tile
// and lets both use every key tile; a unit of one (a decoding step, a short
// chunk) gives the streams alternate key tiles of the same rows, joined at
// the end.  Work is cut evenly over the SMs by fab_paged.cuh whatever the
// lengths are.
//
// Keys and values stream through TMA rings; each box holds min(page, 128)
// rows of one page, fetched by the lane that looked its page up.  Past the
// last key, scores are masked by index and value rows are zeroed in shared
// memory, so nothing of a cache's unused rows reaches a product.
//
// The running maximum is raised only when a tile exceeds it by more than 8
// (log2): weights then stay below 2^8 and the output is rescaled rarely; the
// sum and the output share the stale maximum, so the result is exact.  f16
// weights are kept 2^7 larger, which moves their smallest step 2^7 down.
// Weights are rounded to the input type for the second product, which takes
// both operands in 16 bits; their sum is not.  Against 64 bits the result is then
// off by 1.3 to 1.4 times what one rounding of an f32 result gives (64 decoding
// sequences, bf16: 0.0022 of its size for 0.0017).  A third product, of what
// the rounding left, would cost chunks half as many products again.
//
// Bounds and measured times (bf16, 32 heads on 8, width 128).  Decoding: memory;
// 64 sequences of 64 to 4,095 keys 98 us, 5.7 TB/s; one of 131,000 keys 89 us,
// 6.0 TB/s.  Chunks: the tensor core; two of 2,048 tokens behind 14,336 keys
// 645 to 690 us as the power cap allows, 1.5 to 1.6 PFLOP/s (the pipe is 78%
// active; a plain library product of bf16 sustains 1.69).  At width 64 the
// exponentials: the 16,384 of a 128 x 128 tile take 1,024 cycles, its products
// about 630; chunks of 2,048 tokens behind 6,000 keys 216 us, 1.1 PFLOP/s.
// Short calls: the chain of start, plan, page number, copy, product, softmax,
// product and store, 10.0 us for one sequence of 500 keys of width 64.
//
// Warps (384 threads): 0 = query and key loads, 1 = matrix instructions, 2 =
// value loads, 3 = the units in order and the note for the combine kernel (and
// tensor memory); 4-7 and 8-11 = the two softmax streams.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "fab.h"
#include "fab_device.cuh"
#include "fab_internal.h"
#include "fab_paged.cuh"

namespace fab {
namespace {

__device__ uint32_t g_err_paged_tc;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.f;  // log2 units
constexpr int kThreads = 384;

constexpr int kUnits = 4;  // units described ahead
constexpr int kFewTiles = 8;  // key tiles of a unit that one CTA walks (paged_grid)

// A unit's part of a CTA's piece of the line, for every warp.
struct UnitPart {
  int more;       // 0: the piece is over
  int width;      // row tiles
  int j0, j1;     // key tiles
  int s0, n;      // its sequence's new tokens,
  int last0, len; // last key the first of them sees (causal), keys
  int b;          // the sequence
  int token0;     // first token of the unit
  int hk, g0;     // key/value head, first query head of it
  int slot;       // partial slot, or -1: the unit is whole
  int pad[3];
};
static_assert(sizeof(UnitPart) == 64, "");

template <int DP>
struct PCfg {
  static constexpr int ATOMS = DP / 64;
  static constexpr uint32_t ATOM = 128 * 128;  // 128 rows of 128 swizzled bytes
  static constexpr uint32_t TILE = ATOMS * ATOM;
  static constexpr int NQ = DP == 128 ? 2 : 4, NK = NQ, NV = DP == 128 ? 3 : 4;  // ring slots
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_K = NQ * TILE;
  static constexpr uint32_t OFF_V = OFF_K + NK * TILE;
  static constexpr uint32_t OFF_BAR = OFF_V + NV * TILE;
  static constexpr uint32_t OFF_MISC = OFF_BAR + 52 * 8;
  static constexpr uint32_t OFF_UNIT = OFF_MISC + 16;       // kUnits descriptions of units
  static constexpr uint32_t OFF_ML = OFF_UNIT + kUnits * 64;  // 128 (maximum, sum) pairs; the plan's scratch before
  static constexpr uint32_t USED = OFF_ML + 128 * 8;
  static constexpr uint32_t SMEM = USED > 118784 ? USED : 118784;  // one CTA owns the SM's tensor memory
  // Score tiles in tensor memory: one a stream, and at width 64, where the
  // outputs leave room, a third: the streams then take turns with all three, and
  // a stream's next S is there when its softmax comes for it.
  static constexpr int NB = DP == 128 ? 2 : 3;
  static constexpr uint32_t TM_S = 0;         // + 128 * buffer
  static constexpr uint32_t TM_O = NB * 128;  // + DP * stream
  static_assert(TM_O + 2 * DP <= 512, "tensor memory budget");
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(sizeof(PagedShared) <= 1024, "plan scratch");
};

enum : int {
  B_KF = 0,   // + slot: K landed
  B_KE = 4,   // + slot: K free
  B_VF = 8,   // + slot: V landed
  B_VE = 12,  // + slot: V free
  B_QF = 16,  // + slot: Q landed
  B_QE = 20,  // + slot: Q free
  B_S = 24,   // + buffer: S landed
  B_P = 27,   // + 2 buffer + half: P's keys of that half written (and O rescaled where it had to be);
              // with three buffers only + 1, for both
  B_PV = 33,  // + buffer: O += P V finished (three buffers only)
  B_O = 36,   // + stream: the unit's last product of the stream finished
  B_ML = 38,  // one-tile units: stream 1's maxima and sums are in shared memory
  B_MD = 39,  // one-tile units: stream 0 has read stream 1's output
  B_FIN = 40,
  B_DF = 41,  // + slot: a unit is described
  B_DE = 45,  // + slot: every warp is done with it
  B_COUNT = 49
};

struct TcParams {
  PagedPlan plan;
  PagedParts parts;
  const int32_t* table;
  int64_t max_pages, pages;
  int page, box;  // rows of a page, of a TMA box
  int H, DV;
  float scale;
  void* o;
  float* lse;
};

FAB_DEV void reg_dealloc() { asm volatile("setmaxnreg.dec.sync.aligned.u32 96;"); }
FAB_DEV void reg_alloc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 200;"); }

template <int DP, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TcParams p) {
  using C = PCfg<DP>;
  using T = typename std::conditional<F16, __half, __nv_bfloat16>::type;
  extern __shared__ uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // swizzled tiles need a 1024-byte-aligned base
    asm volatile("griddepcontrol.wait;" ::: "memory");  // (the call before may still be reading its notes)
    if (threadIdx.x == 0) {
      atomicOr(&g_err_paged_tc, kErrSmemAlign);
      if (!p.plan.whole) p.parts.cuts[blockIdx.x] = PagedCut{0, 0, 0, 0, 0, 0, 0, 0};  // nothing to join
    }
    return;
  }
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + C::OFF_BAR + 8u * (uint32_t)i; };
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC + 4);
  int* copied = reinterpret_cast<int*>(smem + C::OFF_MISC + 8);  // where the load warps' rings ended: keys and Q, values
  UnitPart* units = reinterpret_cast<UnitPart*>(smem + C::OFF_UNIT);
  float2* ml_s = reinterpret_cast<float2*>(smem + C::OFF_ML);
  PagedShared* sh = reinterpret_cast<PagedShared*>(smem + C::OFF_ML);
  uint32_t* err = &g_err_paged_tc;
  const int warp = (int)warp_id(), lane = (int)lane_id();
  const PagedPlan& plan = p.plan;

  if (threadIdx.x == 0) {
    *abort_flag = 0u;
    for (int s = 0; s < 4; ++s) {
      mbar_init(bar(B_KF + s), 1);
      mbar_init(bar(B_KE + s), 1);
      mbar_init(bar(B_VF + s), 1);
      mbar_init(bar(B_VE + s), 1);
      mbar_init(bar(B_QF + s), 1);
      mbar_init(bar(B_QE + s), 1);
      mbar_init(bar(B_DF + s), 1);
      mbar_init(bar(B_DE + s), 3 + 8);
    }
    mbar_init(bar(B_O), 1);
    mbar_init(bar(B_O + 1), 1);
    for (int s = 0; s < 3; ++s) {
      mbar_init(bar(B_S + s), 1);
      mbar_init(bar(B_P + 2 * s), 4);
      mbar_init(bar(B_P + 2 * s + 1), 4);
      mbar_init(bar(B_PV + s), 1);
    }
    mbar_init(bar(B_ML), 128);
    mbar_init(bar(B_MD), 128);
    mbar_init(bar(B_FIN), 1);
    fence_mbar_init();
    prefetch_tensormap(&tmQ);
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (launched early: lengths and operands from here on)
  if (warp == 3) {  // (after the wait: a kernel before that is not done yet may still want tensor memory)
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  if (blockIdx.x == 0) check_starts(plan.starts, plan.B, plan.T, (int)threadIdx.x, kThreads, err);
  int64_t mine;
  paged_total<kThreads>(plan, sh, &mine);
  const int64_t W = sh->total;
  const PagedBorders border(W, (int)gridDim.x);
  const int64_t p0 = border((int)blockIdx.x), p1 = border((int)blockIdx.x + 1);
  if (p0 < p1) paged_locate<kThreads>(plan, sh, mine, p0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tm = *tmem_holder;
  const bool any = p0 < p1;

  if (warp < 4) {
    reg_dealloc();
    if (warp == 3) {
      // ------------------------------------------------------------ the units
      if (lane == 0) {
        PagedCut cut{0, 0, 0, 0, 0, 0, 0, 0};
        PagedWalk w;
        bool more = any;
        if (any) {
          w.begin(plan, sh->at);
          more = w.seek(plan, p0, p1);
        }
        uint32_t slot = 0, phase = 1;
        while (mbar_wait_asleep(bar(B_DE + slot), phase, abort_flag, err)) {
          UnitPart* u = units + slot;
          u->more = more;
          if (more) {
            const int hk = w.at.head / plan.gblocks;
            u->width = w.width;
            u->j0 = w.j0;
            u->j1 = w.j1;
            u->s0 = w.q.s0;
            u->n = w.q.n;
            u->last0 = w.q.last0;
            u->len = w.q.len;
            u->b = w.at.b;
            u->token0 = w.at.i * plan.nt * 2;
            u->hk = hk;
            u->g0 = (w.at.head - hk * plan.gblocks) * plan.gw;
            u->slot = w.whole() ? -1 : w.slot((int)blockIdx.x);
          }
          mbar_arrive(bar(B_DF + slot));
          if (!more) break;
          paged_note_part(plan, w, border, (int)blockIdx.x, &cut);
          if (++slot == kUnits) slot = 0, phase ^= 1;
          more = w.next(plan) && w.seek(plan, p0, p1);
        }
        if (!plan.whole) p.parts.cuts[blockIdx.x] = cut;
      }
      __syncwarp();
    } else if (warp != 1) {
      // ------------------------------------------------------------ loads
      // Warp 0: a unit's Q (once the S products of the unit that had its slot
      // are done) and its keys; warp 2: its values.  Lane i fetches box i of a
      // tile; its page number is looked up a tile ahead.
      const bool keys = warp == 0;
      const int full = keys ? B_KF : B_VF, empty = keys ? B_KE : B_VE, slots = keys ? C::NK : C::NV;
      const uint32_t ring = sbase + (keys ? C::OFF_K : C::OFF_V);
      const CUtensorMap* map = keys ? &tmK : &tmV;
      int slot = 0, phase = 1, qslot = 0, qphase = 1, us = 0, up = 0;
      bool ok = true;
      // (the warp goes on or gives up as one: its lanes meet at __syncwarp below)
      auto wait = [&](int i, int parity) {
        return ok = __all_sync(0xffffffffu, mbar_wait_asleep(bar(i), parity, abort_flag, err));
      };
      for (;;) {
        if (!wait(B_DF + us, up)) break;
        const UnitPart& u = units[us];
        if (!u.more) break;
        const int j0 = u.j0, j1 = u.j1, len = u.len, hk = u.hk;
        const int32_t* table = p.table + (int64_t)u.b * p.max_pages;
        // page of box `lane` of key tile j, and its first row there
        auto lookup = [&](int j, int& row) {
          const uint32_t m = (uint32_t)j * 128u + (uint32_t)(lane * p.box);
          const uint32_t at = m / (uint32_t)p.page;
          row = (int)(m - at * (uint32_t)p.page);
          if (lane * p.box >= 128 || m >= (uint32_t)len) return 0;
          const int page = __ldg(table + at);
          // (out of range: the copy fills zeros, the call is reported)
          if (page < 0 || page >= p.pages) atomicOr(err, kErrIndex);
          return page;
        };
        int row, page = lookup(j0, row);
        if (keys) {
          if (lane == 0 && plan.lens[u.b] > plan.max_keys) atomicOr(err, kErrIndex);
          for (int s = 0; s < u.width; ++s) {
            if (!wait(B_QE + qslot, qphase)) break;
            if (lane == 0) {
              mbar_arrive_expect_tx(bar(B_QF + qslot), (uint32_t)(64 * 2 * plan.gw * plan.nt * C::ATOMS));
              for (int a = 0; a < C::ATOMS; ++a)
                tma_load_3d(sbase + C::OFF_Q + qslot * C::TILE + a * C::ATOM, &tmQ, bar(B_QF + qslot), a * 64,
                            hk * plan.G + u.g0, u.s0 + u.token0 + s * plan.nt);
            }
            if (++qslot == C::NQ) qslot = 0, qphase ^= 1;
          }
          if (!ok) break;
        }
        for (int j = j0; j < j1; ++j) {
          if (!wait(empty + slot, phase)) break;
          const int held = len - j * 128;  // keys of the tile and beyond
          const int boxes = held <= 0 ? 0 : held >= 128 ? 128 / p.box : (held + p.box - 1) / p.box;
          fence_proxy_async_smem();
          if (lane == 0) mbar_arrive_expect_tx(bar(full + slot), (uint32_t)(boxes * p.box * 128 * C::ATOMS));
          __syncwarp();
          if (lane < boxes) {
            const uint32_t dst = ring + slot * C::TILE + lane * p.box * 128;
#pragma unroll
            for (int a = 0; a < C::ATOMS; ++a)
              tma_load_4d(dst + a * C::ATOM, map, bar(full + slot), a * 64, row, hk, page);
          }
          if (++slot == slots) slot = 0, phase ^= 1;
          if (j + 1 < j1) page = lookup(j + 1, row);
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_DE + us));
        if (++us == kUnits) us = 0, up ^= 1;
      }
      if (lane == 0) copied[keys ? 0 : 1] = slot | phase << 4 | qslot << 8 | qphase << 12;  // (see the end)
    } else {
      // ------------------------------------------------------------ products
      // One elected lane does it all: the compiler then knows that a single lane
      // issues the matrix instructions (9 cycles each; from a lane chosen by its
      // number 47, of the 64 that they run for).  A stream's next S is issued
      // right behind the O += P V that frees its columns: a thread's matrix
      // instructions run in the order of their issue.  A slot of K's or V's ring
      // and of Q is freed by a commit behind the last product that reads it.
      if (elect_one()) {
        // (bit 13: A, the queries, negated, for a scale below zero)
        const uint32_t ID_S = idesc_16(128, 128, false, false, F16) | (p.scale < 0.f ? 1u << 13 : 0u);
        constexpr uint32_t ID_PV = idesc_16(128, DP, false, true, F16);
        constexpr uint32_t HI = sdesc_hi_sw128(1024);
        constexpr uint32_t SLOT = C::TILE >> 4;  // a slot, in a descriptor's units
        const uint32_t q_lo = sdesc_lo(sbase + C::OFF_Q, 16), k_lo = sdesc_lo(sbase + C::OFF_K, 16);
        const uint32_t v_lo = sdesc_lo(sbase + C::OFF_V, C::ATOM);
        auto wait = [&](int i, uint32_t parity) { return mbar_wait_asleep(bar(i), parity, abort_flag, err); };
        constexpr int NB = C::NB;
        auto s_product = [&](uint32_t buf, uint32_t a_lo, uint32_t b_lo) {
#pragma unroll
          for (int kk = 0; kk < DP / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * C::ATOM + (kk & 3) * 32) >> 4;
            mma_ss_one(tm + C::TM_S + buf * 128, a_lo + off, b_lo + off, HI, ID_S, kk > 0);
          }
          mma_commit_one(bar(B_S + buf));
        };
        // O_s += P V (more = 0: O_s = P V), P in a buffer; with `early` the first 64
        // keys as soon as their weights are there.
        uint32_t pphase = 0;  // bit 2 buffer + half
        auto pv_product = [&](uint32_t s, uint32_t buf, uint32_t b_lo, uint32_t keys, uint32_t more, bool early) -> bool {
          const uint32_t d = tm + C::TM_O + s * DP, a = tm + C::TM_S + buf * 128;
          auto half = [&](uint32_t h) {
            if (!wait(B_P + 2 * buf + h, (pphase >> (2 * buf + h)) & 1u)) return false;
            tc_fence_after();
            return true;
          };
          if (!half(early ? 0 : 1)) return false;
          if (keys == 128) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_ts_one(d, a + kk * 8, b_lo + kk * 128, HI, ID_PV, kk > 0 ? 1u : more);
            if (early && !half(1)) return false;
#pragma unroll
            for (int kk = 4; kk < 8; ++kk) mma_ts_one(d, a + kk * 8, b_lo + kk * 128, HI, ID_PV, 1u);
          } else {
            if (early && !half(1)) return false;
            for (uint32_t kk = 0; kk * 16 < keys; ++kk)
              mma_ts_one(d, a + kk * 8, b_lo + kk * 128, HI, ID_PV, kk > 0 ? 1u : more);
          }
          pphase ^= 3u << (2 * buf);
          if (NB == 3) mma_commit_one(bar(B_PV + buf));
          return true;
        };
        // The last keys' tile: products run over whole steps of 16 keys (one at
        // least), with the rows from the last key to the steps' end zeroed.
        auto end_keys = [&](uint32_t slot, uint32_t last) -> uint32_t {
          const uint32_t keys = last == 0 ? 16u : (last + 15u) / 16u * 16u;
          if (last < 128u) {
            const uint32_t row0 = sbase + C::OFF_V + slot * C::TILE;
            for (uint32_t x = last * 8u; x < keys * 8u; ++x) {
              st_shared_v4(row0 + x * 16u, 0u, 0u, 0u, 0u);
              if (C::ATOMS == 2) st_shared_v4(row0 + C::ATOM + x * 16u, 0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
          }
          return keys;
        };
        auto last_of = [&](const UnitPart& x) {  // keys from the part's last key tile on, 128 at most
          const int held = x.len - (x.j1 - 1) * 128;
          return held < 0 ? 0u : held > 128 ? 128u : (uint32_t)held;
        };
        uint32_t kslot = 0, kphase = 0, vslot = 0, vphase = 0, qn = 0;
        bool ok = true;
        auto next_k = [&]() {
          if (++kslot == C::NK) kslot = 0, kphase ^= 1;
        };
        auto next_v = [&]() {
          if (++vslot == C::NV) vslot = 0, vphase ^= 1;
        };
        uint32_t sbuf = 0, pbuf = 0;  // three buffers: the next S's and the next P's
        auto next_buf = [&](uint32_t& b) {
          if (++b == 3) b = 0;
        };
        // A unit of two row tiles: per key tile O_0, S_0, O_1, S_1, so that each
        // stream's softmax runs beside the other's products.
        auto two_tiles = [&](const UnitPart& x) -> bool {
          const uint32_t tiles = (uint32_t)(x.j1 - x.j0), last = last_of(x);
          const uint32_t q0 = qn % C::NQ, q1 = (qn + 1) % C::NQ;
          const uint32_t a0 = q_lo + q0 * SLOT, a1 = q_lo + q1 * SLOT;
          if (!wait(B_QF + q0, (qn / C::NQ) & 1u) || !wait(B_QF + q1, ((qn + 1) / C::NQ) & 1u)) return false;
          qn += 2;
          if constexpr (NB == 3) {
            const uint32_t steps = 2 * tiles;
            uint32_t si = 0;
            auto next_s = [&]() -> bool {
              if (!(si & 1u)) {
                if (!wait(B_KF + kslot, kphase)) return false;
                tc_fence_after();
              }
              s_product(sbuf, si & 1u ? a1 : a0, k_lo + kslot * SLOT);
              next_buf(sbuf);
              if (si & 1u) {
                mma_commit_one(bar(B_KE + kslot));
                next_k();
              }
              if (++si == steps) {
                mma_commit_one(bar(B_QE + q0));
                mma_commit_one(bar(B_QE + q1));
              }
              return true;
            };
            while (si < steps && si < 3)
              if (!next_s()) return false;
            uint32_t keys = 128;
            for (uint32_t i = 0; i < steps; ++i) {
              if (!(i & 1u)) {
                if (!wait(B_VF + vslot, vphase)) return false;
                if (i + 2 == steps) keys = end_keys(vslot, last);
              }
              if (!pv_product(i & 1u, pbuf, v_lo + vslot * SLOT, keys, i >= 2 ? 1u : 0u, false)) return false;
              next_buf(pbuf);
              if (i + 2 >= steps) mma_commit_one(bar(B_O + (i & 1u)));
              if (i & 1u) {
                mma_commit_one(bar(B_VE + vslot));
                next_v();
              }
              if (si < steps && !next_s()) return false;
            }
            return true;
          }
          if (!wait(B_KF + kslot, kphase)) return false;
          tc_fence_after();
          s_product(0, a0, k_lo + kslot * SLOT);
          s_product(1, a1, k_lo + kslot * SLOT);
          mma_commit_one(bar(B_KE + kslot));
          next_k();
          uint32_t more = 0;
          for (uint32_t t = 1; t < tiles; ++t) {
            if (!wait(B_KF + kslot, kphase) || !wait(B_VF + vslot, vphase)) return false;
            const uint32_t kb = k_lo + kslot * SLOT, vb = v_lo + vslot * SLOT;
            if (!pv_product(0, 0, vb, 128, more, true)) return false;
            s_product(0, a0, kb);
            if (!pv_product(1, 1, vb, 128, more, true)) return false;
            mma_commit_one(bar(B_VE + vslot));
            s_product(1, a1, kb);
            mma_commit_one(bar(B_KE + kslot));
            more = 1;
            next_k();
            next_v();
          }
          mma_commit_one(bar(B_QE + q0));
          mma_commit_one(bar(B_QE + q1));
          if (!wait(B_VF + vslot, vphase)) return false;
          const uint32_t vb = v_lo + vslot * SLOT, keys = end_keys(vslot, last);
          if (!pv_product(0, 0, vb, keys, more, true)) return false;
          mma_commit_one(bar(B_O));
          if (!pv_product(1, 1, vb, keys, more, true)) return false;
          mma_commit_one(bar(B_O + 1));
          mma_commit_one(bar(B_VE + vslot));
          next_v();
          return true;
        };
        // Units of one row tile: key tile i is stream i & 1's.  The S products
        // run two tiles ahead (unit sd, tile si), into the next such unit too
        // where its operands have landed, so that a unit's end leaves work to do.
        uint32_t us = 0, up = 0;                      // the unit at work
        uint32_t sd = 0, sdp = 0, si = 0, ahead = 0;  // the S products' unit; units between the two
        uint32_t busy = 0;                            // streams (three buffers: buffers) with an S or a P
        auto s_ahead = [&]() -> bool {
          while (!((busy >> (NB == 3 ? sbuf : si & 1u)) & 1u)) {
            // another unit's description and operands are waited for only when
            // nothing else is left to do
            const bool patient = busy != 0 && ahead != 0;
            if (patient && !mbar_test(bar(B_DF + sd), sdp)) return true;
            if (!wait(B_DF + sd, sdp)) return false;
            const UnitPart& u = units[sd];
            if (!u.more || u.width == 2) return true;
            const uint32_t qs = qn % C::NQ, qp = (qn / C::NQ) & 1u;
            if (patient && !((si > 0 || mbar_test(bar(B_QF + qs), qp)) && mbar_test(bar(B_KF + kslot), kphase)))
              return true;
            if (si == 0 && !wait(B_QF + qs, qp)) return false;
            if (!wait(B_KF + kslot, kphase)) return false;
            tc_fence_after();
            const uint32_t buf = NB == 3 ? sbuf : si & 1u;
            s_product(buf, q_lo + qs * SLOT, k_lo + kslot * SLOT);
            next_buf(sbuf);
            mma_commit_one(bar(B_KE + kslot));
            next_k();
            busy |= 1u << buf;
            if ((int)++si == u.j1 - u.j0) {
              mma_commit_one(bar(B_QE + qs));
              ++qn;
              si = 0;
              ++ahead;
              if (++sd == kUnits) sd = 0, sdp ^= 1u;
            }
          }
          return true;
        };
        auto one_tile = [&](const UnitPart& x) -> bool {
          const uint32_t tiles = (uint32_t)(x.j1 - x.j0), last = last_of(x);
          for (uint32_t i = 0; i < tiles; ++i) {
            const uint32_t s = i & 1u;
            if (!s_ahead() || !wait(B_VF + vslot, vphase)) return false;
            const uint32_t keys = i + 1 == tiles ? end_keys(vslot, last) : 128u;
            const uint32_t buf = NB == 3 ? pbuf : s;
            if (!pv_product(s, buf, v_lo + vslot * SLOT, keys, i < 2 ? 0u : 1u, false)) return false;
            next_buf(pbuf);
            mma_commit_one(bar(B_VE + vslot));
            if (i + 2 >= tiles) mma_commit_one(bar(B_O + s));
            next_v();
            busy &= ~(1u << buf);
          }
          --ahead;
          return true;
        };
        while (ok && wait(B_DF + us, up)) {
          const UnitPart& u = units[us];
          if (!u.more) break;
          if (u.width == 2) {
            ok = two_tiles(u);
            if (++sd == kUnits) sd = 0, sdp ^= 1u;
          } else {
            ok = one_tile(u);
          }
          if (!ok) break;
          mbar_arrive(bar(B_DE + us));
          if (++us == kUnits) us = 0, up ^= 1u;
        }
        mma_commit_one(bar(B_FIN));
        mbar_drain(bar(B_FIN), 0);
      }
      __syncwarp();
    }
  } else {
    reg_alloc();
    // -------------------------------------------------------------- softmax
    const int s = (warp - 4) >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tO = tm + lane_off + C::TM_O + s * DP;
    // weights 2^(s c1 - m) (the S products carry the scale's sign); a scale of
    // zero is taken as one too small to tell the scores apart (0 times a masked
    // score would be NaN)
    const float c1 = fmaxf(fabsf(p.scale) * kLog2e, 1e-37f);
    constexpr float kBias = F16 ? 7.f : 0.f;
    const int i_row = r / plan.gw, g_row = r - i_row * plan.gw;
    uint32_t sphase = 0, ophase = 0, mphase = 0;
    uint32_t steps = 0;  // three buffers: steps of the units before
    uint32_t us = 0, up = 0;
    bool ok = true;
    auto next_unit = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_DE + us));
      if (++us == kUnits) us = 0, up ^= 1u;
    };
    for (;;) {
      if (!(ok = __all_sync(0xffffffffu, mbar_wait_asleep(bar(B_DF + us), up, abort_flag, err)))) break;
      const UnitPart& u = units[us];
      if (!u.more) break;
      {
        const bool wide = u.width == 2;
        const int n = u.j1 - u.j0;
        const int token = u.token0 + (wide ? s * plan.nt : 0) + i_row;
        const bool row_ok = i_row < plan.nt && token < u.n && u.g0 + g_row < plan.G;
        const bool active = __any_sync(0xffffffffu, row_ok);
        int last = u.len - 1;  // last key the row sees
        if (plan.causal && u.last0 + token < last) last = u.last0 + token;
        if (!row_ok) last = -1;
        last -= u.j0 * 128;  // counted from the part's first key
        float m_run = -INFINITY, l = 0.f;
        for (int t = wide ? 0 : s; t < n; t += wide ? 1 : 2) {
          const uint32_t step = steps + (wide ? 2 * t + s : t);
          const uint32_t buf = C::NB == 3 ? step % 3u : (uint32_t)s;
          const uint32_t tS = tm + lane_off + C::TM_S + buf * 128;
          if (C::NB == 3) sphase = (step / 3u) & 1u;
          if (!ok || !(ok = __all_sync(0xffffffffu, mbar_wait_asleep(bar(B_S + buf), sphase, abort_flag, err)))) break;
          sphase ^= 1;
          if (active) {
            tc_fence_after();
            const int k0 = t * 128;
            uint32_t x[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, x[c]);
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld_wait(x[c]);
            auto sv = [&](int e) -> uint32_t& { return x[e >> 5][e & 31]; };
            if (__any_sync(0xffffffffu, row_ok && k0 + 127 > last)) {
              const int lim = last - k0;
#pragma unroll
              for (int e = 0; e < 128; ++e)
                if (e > lim) sv(e) = 0xff800000u;  // -inf
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 128; e += 8)
#pragma unroll
              for (int c = 0; c < 4; ++c)
                mx[c] = max3(mx[c], __uint_as_float(sv(e + 2 * c)), __uint_as_float(sv(e + 2 * c + 1)));
            const float tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c1;
            float alpha = 1.f;
            bool need = false;
            if (tmax > m_run + kRescaleThreshold || (m_run == -INFINITY && tmax > -INFINITY)) {
              need = row_ok && m_run != -INFINITY;
              alpha = need ? exp2f(m_run - tmax) : 1.f;
              m_run = tmax;
            }
            if (__any_sync(0xffffffffu, need)) {
              // two buffers: every product into O_s was issued before this S, so it
              // is done; three: the last one is waited for
              if (C::NB == 3)
                ok = __all_sync(0xffffffffu, mbar_wait_asleep(bar(B_PV + (step - 2) % 3u), ((step - 2) / 3u) & 1u,
                                                              abort_flag, err));
              tc_fence_after();
#pragma unroll 1
              for (int c0 = 0; c0 < DP; c0 += 32) {
                uint32_t o[32];
                tmem_ld32(tO + c0, o);
                tmem_ld_wait(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st32(tO + c0, o);
              }
              l *= alpha;
            }
            const float ref = m_run == -INFINITY ? 0.f : m_run - kBias;
            const uint64_t c12 = pair_f32(c1, c1), ref2 = pair_f32(-ref, -ref);
            uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t pk[32];
#pragma unroll
              for (int c = 0; c < 32; ++c) {
                const int e = h * 64 + 2 * c;
                const float2 y =
                    split_f32(fma_f32x2(pair_f32(__uint_as_float(sv(e)), __uint_as_float(sv(e + 1))), c12, ref2));
                const float a = ex2_approx(y.x), b = ex2_approx(y.y);
                sum[c & 3] = add_f32x2(sum[c & 3], pair_f32(a, b));
                pk[c] = pack2<F16>(a, b);
              }
              tmem_st32(tS + h * 32, pk);
              if (C::NB == 2 || h == 1) {  // (three buffers: nothing waits for the first half alone)
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_P + 2 * buf + h));
              }
            }
            const float2 total = split_f32(add_f32x2(add_f32x2(sum[0], sum[1]), add_f32x2(sum[2], sum[3])));
            l += total.x + total.y;
          } else if (lane < 2 && (C::NB == 2 || lane == 1)) {
            mbar_arrive(bar(B_P + 2 * buf + lane));
          }
        }
        if (!ok) break;
        steps += wide ? 2 * n : n;
        // ---- the unit's end: O / l and the log-sum-exp, or partial results
        const float ref = m_run == -INFINITY ? 0.f : m_run - kBias;
        const bool ran = wide || s < n;  // the stream had a key tile
        if (ran) {
          if (!(ok = __all_sync(0xffffffffu, mbar_wait_asleep(bar(B_O + s), ophase, abort_flag, err)))) break;
          ophase ^= 1;
        }
        float f0 = 1.f, f1 = 0.f, lt = l, mt = ref;  // the row is f0 O_0 + f1 O_1
        if (!wide) {
          if (s == 1) {
            // hand over to stream 0, which has the same rows in the same lanes
            ml_s[r] = make_float2(ref, l);
            tc_fence_after();
            tc_fence_before();
            mbar_arrive(bar(B_ML));
            if (!(ok = __all_sync(0xffffffffu, mbar_wait_asleep(bar(B_MD), mphase, abort_flag, err)))) break;
            mphase ^= 1;
            next_unit();
            continue;
          }
          if (!(ok = __all_sync(0xffffffffu, mbar_wait_asleep(bar(B_ML), mphase, abort_flag, err)))) break;
          mphase ^= 1;
          const float2 other = ml_s[r];
          if (other.y != 0.f) {
            if (l == 0.f) {
              mt = other.x;
              f0 = 0.f;
              f1 = 1.f;
            } else {
              mt = fmaxf(ref, other.x);
              f0 = exp2f(ref - mt);
              f1 = exp2f(other.x - mt);
            }
            lt = (f0 == 0.f ? 0.f : f0 * l) + f1 * other.y;
          }
        }
        if (active) {
          tc_fence_after();
          const bool two = !wide && n > 1;
          const int64_t tok = u.s0 + token, head = (int64_t)u.hk * plan.G + u.g0 + g_row;
          const bool whole = u.slot < 0;
          const float inv = lt == 0.f ? 0.f : whole ? 1.f / lt : 1.f;
          const float a0 = l == 0.f ? 0.f : f0 * inv, a1 = f1 * inv;
          T* o = static_cast<T*>(p.o) + (tok * p.H + head) * p.DV;
          const int prow = (wide ? s * 128 : 0) + r;
          float4* part = paged_part(p.parts, u.slot, u.width, prow, 0);
          const int next4 = wide ? 256 : 1;  // from 4 columns to the next
#pragma unroll 1
          for (int c0 = 0; c0 < DP; c0 += 32) {
            uint32_t x[32];
            tmem_ld32(tO + c0, x);
            tmem_ld_wait(x);
            // (a factor of zero drops what the columns hold, NaN too)
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = a0 == 0.f ? 0u : __float_as_uint(__uint_as_float(x[e]) * a0);
            if (two) {
              uint32_t y[32];
              tmem_ld32(tO + DP + c0, y);
              tmem_ld_wait(y);
              if (a1 != 0.f) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  x[e] = __float_as_uint(fmaf(__uint_as_float(y[e]), a1, __uint_as_float(x[e])));
              }
            }
            if (!row_ok) continue;
            if (whole) {
#pragma unroll
              for (int e = 0; e < 32; e += 8)
                if (c0 + e < p.DV)
                  *reinterpret_cast<uint4*>(o + c0 + e) =
                      make_uint4(pack2<F16>(__uint_as_float(x[e]), __uint_as_float(x[e + 1])),
                                 pack2<F16>(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])),
                                 pack2<F16>(__uint_as_float(x[e + 4]), __uint_as_float(x[e + 5])),
                                 pack2<F16>(__uint_as_float(x[e + 6]), __uint_as_float(x[e + 7])));
            } else {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                part[(c0 + e) / 4 * next4] = make_float4(__uint_as_float(x[e]), __uint_as_float(x[e + 1]),
                                                         __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
            }
          }
          if (row_ok) {
            if (!whole)
              p.parts.ml[(int64_t)u.slot * 256 + prow] = make_float2(mt, lt);
            else if (p.lse != nullptr)
              p.lse[head * plan.T + tok] = lt == 0.f ? INFINITY : (mt + log2f(lt)) * kLn2;
          }
          tc_fence_before();
        }
        if (!wide) mbar_arrive(bar(B_MD));
      }
      next_unit();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tm, 512);
  }
  // Where a wait ran out, copies may still be in flight that no warp has waited
  // for: they land before shared memory goes.
  if (*abort_flag != 0u && threadIdx.x == 0) {
    auto drain = [&](int first, int slots, int slot, int phase) {
      for (int s = 0; s < slots; ++s) mbar_drain(bar(first + s), s < slot ? phase ^ 1 : phase);
    };
    drain(B_KF, C::NK, copied[0] & 15, copied[0] >> 4 & 1);
    drain(B_QF, C::NQ, copied[0] >> 8 & 15, copied[0] >> 12 & 1);
    drain(B_VF, C::NV, copied[1] & 15, copied[1] >> 4 & 1);
  }
}

int gcd(int a, int b) { return b == 0 ? a : gcd(b, a % b); }

bool make_map(CUtensorMap* map, bool f16, int rank, const void* base, const cuuint64_t* dims, const cuuint64_t* strides,
              const cuuint32_t* box) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return false;
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank,
             const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int padded_width(const PagedProblem& pr) { return (pr.DK > pr.DV ? pr.DK : pr.DV) <= 64 ? 64 : 128; }

PagedPlan plan_of(const PagedProblem& pr) {
  PagedPlan p{};
  p.starts = pr.starts;
  p.lens = pr.lens;
  p.B = pr.B;
  p.T = pr.T;
  const int64_t most = pr.max_pages * pr.page;
  p.max_keys = most < 2147483647ll - 256 ? most : 2147483647ll - 256;  // (lengths are 32-bit)
  p.causal = pr.causal;
  p.G = (int)(pr.H / pr.Hkv);
  p.gw = p.G < 128 ? p.G : 128;
  p.gblocks = (p.G + p.gw - 1) / p.gw;
  p.heads = (int)pr.Hkv * p.gblocks;
  p.nt = 128 / p.gw;
  p.tiles = 2;
  p.kt = 128;
  p.snap = padded_width(pr) / 64;
  return p;
}

template <int DP, bool F16>
cudaError_t launch_d(const PagedProblem& pr, int sms, cudaStream_t s) {
  using C = PCfg<DP>;
  using T = typename std::conditional<F16, __half, __nv_bfloat16>::type;
  TcParams p;
  p.plan = plan_of(pr);
  p.parts = paged_parts(pr.workspace, 256, DP);
  p.table = pr.table;
  p.max_pages = pr.max_pages;
  p.pages = pr.pages;
  p.page = (int)pr.page;
  p.box = gcd((int)pr.page, 128);
  p.H = (int)pr.H;
  p.DV = (int)pr.DV;
  p.scale = pr.scale;
  p.o = pr.o;
  p.lse = pr.lse;
  CUtensorMap mq, mk, mv;
  {
    const cuuint64_t dims[3] = {(cuuint64_t)pr.DK, (cuuint64_t)pr.H, (cuuint64_t)pr.T};
    const cuuint64_t str[2] = {(cuuint64_t)pr.DK * 2, (cuuint64_t)(pr.H * pr.DK) * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)p.plan.gw, (cuuint32_t)p.plan.nt};
    if (!make_map(&mq, F16, 3, pr.q, dims, str, box)) return cudaErrorInvalidValue;
  }
  for (int v = 0; v < 2; ++v) {
    const cuuint64_t D = (cuuint64_t)(v ? pr.DV : pr.DK);
    const cuuint64_t dims[4] = {D, (cuuint64_t)pr.page, (cuuint64_t)pr.Hkv, (cuuint64_t)pr.pages};
    const cuuint64_t str[3] = {D * 2, (cuuint64_t)pr.page * D * 2, (cuuint64_t)(pr.Hkv * pr.page) * D * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)p.box, 1, 1};
    if (!make_map(v ? &mv : &mk, F16, 4, v ? pr.v : pr.k, dims, str, box)) return cudaErrorInvalidValue;
  }
  const int grid = paged_grid(&p.plan, sms, kFewTiles);
  cudaError_t err =
      cudaFuncSetAttribute(paged_tc_kernel<DP, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (err != cudaSuccess) return err;
  err = launch_early(paged_tc_kernel<DP, F16>, dim3((unsigned)grid), kThreads, C::SMEM, s, mq, mk, mv, p);
  if (err != cudaSuccess) return err;
  return launch_combine<T>(p.plan, p.parts, grid, (int)pr.DV, (int)pr.H, static_cast<T*>(pr.o), pr.lse, s);
}

}  // namespace

bool paged_tc_supported(const PagedProblem& p) {
  if (p.dtype != FAB_BF16 && p.dtype != FAB_F16) return false;
  // rows of whole 16-byte pieces, boxes of whole swizzle groups of 8 rows (the
  // same calls on the CUDA cores: 64 decoding sequences 230 us for 98, one of
  // 500 keys 13.1 for 11.5, mixed chunks at width 64 2,348 for 52.2)
  if (p.DK % 8 != 0 || p.DV % 8 != 0 || p.DK > 128 || p.DV > 128 || p.page % 8 != 0) return false;
  // what a tensor map can describe
  const int64_t D = p.DK > p.DV ? p.DK : p.DV, lim = int64_t(1) << 40;
  return p.Hkv * p.page * D * 2 < lim && p.H * p.DK * 2 < lim && p.H < (1ll << 31);
}

size_t paged_tc_workspace_bytes(const PagedProblem& p) {
  return paged_workspace(plan_of(p), kFewTiles, 256, padded_width(p));
}

cudaError_t launch_paged_tc(const PagedProblem& p, cudaStream_t s) {
  const int sms = paged_sms();
  if (sms == 0) return cudaErrorInvalidValue;
  if (padded_width(p) == 128)
    return p.dtype == FAB_F16 ? launch_d<128, true>(p, sms, s) : launch_d<128, false>(p, sms, s);
  return p.dtype == FAB_F16 ? launch_d<64, true>(p, sms, s) : launch_d<64, false>(p, sms, s);
}

uint32_t take_error_paged_tc() {
  uint32_t v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_paged_tc, sizeof(v)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(g_err_paged_tc, &z, sizeof(z));
  return v;
}

}  // namespace fab
